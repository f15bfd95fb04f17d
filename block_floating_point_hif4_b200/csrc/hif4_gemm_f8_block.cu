// hif4_gemm_f8_block.cu — matrix product of FP8 operands with one FP32 scale
// per block of 128:
//   y[m][n] = bias[n] + sum_u sa[u][m] sb[u, n] sum_{k in block u} a[m][k] b[n][k]
// with 1 x 128 blocks on a and 128 x 128 or 1 x 128 blocks on b.
//
// FP32 scales cannot enter the tensor core (its block scales are powers of
// two), so each 128-deep product goes to a TMEM accumulator of its own
// (tcgen05 kind::f8f6f4, FP32 accumulation), and the promotion warps read it
// back and add  scale * P  into FP32 totals held in registers: one FMA per
// output element and 128 of K.
//
// Roles (256 threads): warp 0 issues the TMA loads (128-byte swizzled operand
// tiles into a ring, scale vectors into a ring of their own), warp 1 the MMAs
// into two alternating accumulators; warps 4-7 promote.  The tile is 128 rows
// of one operand (P) by BN rows of the other (Q).  SWAP exchanges the roles of
// a and b: for few rows of a, the weight fills the MMA's 128 rows and the
// tokens its narrow side, so that the tensor core and the TMA box do no work
// for rows that do not exist.
//
// When there are too few tiles for the GPU, a cluster of S CTAs shares a tile:
// each takes a contiguous part of K, leaves its FP32 totals in its shared
// memory, and after a cluster barrier each adds up its share of the tile over
// the CTAs in rank order (distributed shared memory).  The order of the sum is
// fixed and no workspace is needed.
//
// Every mbarrier wait is bounded (4 s); a role that gives up sets the block's
// abort flag, the producer lets its copies land, the MMA thread drains its
// MMAs before TMEM is freed, every thread still meets the cluster barriers,
// and HIF4_FLAG_TIMEOUT is raised.
#include "hif4_f8.cuh"
#include "hif4_pdl.cuh"
#include "hif4_sm100.cuh"

namespace hif4 {

bool make_tensor_map_u8_2d_sw128(CUtensorMap *map, const void *base, uint64_t inner, uint64_t outer,
                                 uint64_t row_stride_bytes, uint32_t box_inner, uint32_t box_outer);

namespace gemm8b {

constexpr int BP = 128;                         // rows of a tile (MMA M)
constexpr int KU = 128;                         // K elements (bytes) per unit and per stage
constexpr int SLOTS = 8;                        // scale ring
constexpr int GROUP = 16;                       // raster: P tiles per group
constexpr uint64_t TIMEOUT_NS = 4000000000ull;

template <int BN>
struct Cfg {
    static constexpr int EPI_WARPS = 4;
    static constexpr int THREADS = 128 + 32 * EPI_WARPS;
    static constexpr int ACC = BN;              // totals per promotion thread
    static constexpr int CTAS = BN <= 32 ? 3 : BN <= 64 ? 2 : 1;      // per SM
    static constexpr int STAGES = BN <= 32 ? 3 : BN <= 64 ? 4 : 5;
    static constexpr int CH = BN >= 128 ? 32 : 16;                    // columns per TMEM read
    static constexpr int P_BYTES = BP * KU;
    static constexpr int Q_BYTES = BN * KU;
    static constexpr int RING = STAGES * (P_BYTES + Q_BYTES);
    static constexpr int TMEM_COLS = 2 * BN < 32 ? 32 : 2 * BN;
    static constexpr int PITCH = BP + 1;        // of the staged totals: conflict-free along either axis
    static constexpr int BARS = 2 * STAGES + 4 + 1 + SLOTS;
    static constexpr size_t SMEM = (size_t)RING + SLOTS * (BP + BN) * 4 + BARS * 8 + 64 + 1024;
    static_assert(SLOTS >= STAGES + 3, "a scale slot is rewritten only after its unit's promotion");
    static_assert(BN * PITCH * 4 <= RING, "the staged totals reuse the operand ring");
};

struct Args {
    int P, Q;                                   // rows of the two operands
    int num_p, num_q, num_u, num_tiles;
    int split;                                  // CTAs per tile (the cluster)
    const float *p_vec, *q_vec;                 // scale vectors [num_u][ld] (null: block scales)
    int64_t p_ld, q_ld;
    const float *blk;                           // 128 x 128 block scales [row block][num_u ..]
    int64_t blk_ld;
    const uint16_t *bias;                       // BF16 [N], nullable
    void *y;
    int64_t ldy;
    uint32_t out_f32;
    uint32_t idesc;
    uint32_t *status;
    uint32_t withhold;
    uint64_t timeout_ns;
};

__device__ __forceinline__ void fma2(float &d0, float &d1, float a0, float a1, float b0, float b1)
{
    asm("{\n\t.reg .b64 pa, pb, pd;\n\t"
        "mov.b64 pa, {%2, %3};\n\tmov.b64 pb, {%4, %5};\n\tmov.b64 pd, {%0, %1};\n\t"
        "fma.rn.f32x2 pd, pa, pb, pd;\n\tmov.b64 {%0, %1}, pd;\n\t}"
        : "+f"(d0), "+f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

template <int N>
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&r)[N])
{
    if constexpr (N == 32)
        sm100::tmem_ld_32x32b_x32(addr, r);
    else
        sm100::tmem_ld_32x32b_x16(addr, r);
}

// Waits for the TMEM reads in flight; r may be used only after it.
template <int N>
__device__ __forceinline__ void tmem_landed(uint32_t (&r)[N])
{
    sm100::tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ float peer_ld(uint32_t local, uint32_t rank)
{
    uint32_t a;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(local), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ void tile_coords(int t, const Args &g, int &pb, int &qb)
{
    const int per_group = GROUP * g.num_q;
    const int gi = t / per_group;
    const int first = gi * GROUP;
    const int gp = min(g.num_p - first, GROUP);
    const int r = t - gi * per_group;
    pb = first + r % gp;
    qb = r / gp;
}

// acc[0..N) += r c[0..N) p[0..N); COLS: column factors from shared memory, else r alone.
template <int N, bool COLS>
__device__ __forceinline__ void promote(float *acc, const uint32_t (&p)[N], float r, const float *c)
{
#pragma unroll
    for (int j = 0; j < N; j += 4) {
        float f[4] = {r, r, r, r};
        if (COLS) {
            const float4 w = *reinterpret_cast<const float4 *>(c + j);
            f[0] = w.x * r; f[1] = w.y * r; f[2] = w.z * r; f[3] = w.w * r;
        }
#pragma unroll
        for (int i = 0; i < 4; i += 2)
            fma2(acc[j + i], acc[j + i + 1], bits_f(p[j + i]), bits_f(p[j + i + 1]), f[i], f[i + 1]);
    }
}

__device__ __forceinline__ void store_one(const Args &g, int64_t m, int n, float v)
{
    if (g.out_f32) {
        static_cast<float *>(g.y)[m * g.ldy + n] = v;
    } else {
        const __nv_bfloat16 h = __float2bfloat16_rn(v);
        static_cast<uint16_t *>(g.y)[m * g.ldy + n] = *reinterpret_cast<const uint16_t *>(&h);
    }
}

__device__ __forceinline__ float bias_of(const Args &g, int n)
{
    return g.bias ? bits_f((uint32_t)__ldg(g.bias + n) << 16) : 0.0f;
}

template <int BN, bool SWAP, bool VECB>
__global__ void __launch_bounds__(Cfg<BN>::THREADS, Cfg<BN>::CTAS)
k_gemm_f8_block(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ, Args g)
{
    using namespace sm100;
    using C = Cfg<BN>;
    constexpr bool PVEC = !SWAP || VECB;        // P / Q carry scale vectors
    constexpr bool QVEC = SWAP || VECB;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sP = smem;
    uint8_t *sQ = sP + C::STAGES * C::P_BYTES;
    float *sPv = reinterpret_cast<float *>(smem + C::RING);               // [SLOTS][BP]
    float *sQv = sPv + SLOTS * BP;                                        // [SLOTS][BN]
    uint64_t *full = reinterpret_cast<uint64_t *>(sQv + SLOTS * BN);
    uint64_t *empty = full + C::STAGES;
    uint64_t *tfull = empty + C::STAGES;
    uint64_t *tempty = tfull + 2;
    uint64_t *drain = tempty + 2;
    uint64_t *sfull = drain + 1;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(sfull + SLOTS);
    volatile uint32_t *abort_flag = tmem_holder + 1;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&tfull[a], 1);
            mbar_init(&tempty[a], C::EPI_WARPS);
        }
        for (int s = 0; s < SLOTS; ++s) mbar_init(&sfull[s], 1);
        mbar_init(drain, 1);
        *abort_flag = 0u;
        fence_barrier_init();
        prefetch_tensormap(&tmP);
        prefetch_tensormap(&tmQ);
    }
    if (warp == 1) {
        tmem_alloc(tmem_holder, C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    pdl_enter();

    const int split = g.split;
    const int rank = split > 1 ? (int)cluster_rank() : 0;
    const int t0 = blockIdx.x / split, tstep = gridDim.x / split;
    const int u0 = (int)((int64_t)g.num_u * rank / split), u1 = (int)((int64_t)g.num_u * (rank + 1) / split);

    if (warp < 4) {
        if (warp == 0 && lane == 0) {
            // ---------------------------------------------------- producer
            uint32_t stage = 0, phase = 0, issued = 0, ug = 0;
            bool ok = true;
            for (int t = t0; ok && t < g.num_tiles; t += tstep) {
                int pb, qb;
                tile_coords(t, g, pb, qb);
                const uint32_t pv = (uint32_t)min(BP, (g.P - pb * BP + 3) & ~3) * 4;
                const uint32_t qv = (uint32_t)min(BN, (g.Q - qb * BN + 3) & ~3) * 4;
                for (int u = u0; u < u1; ++u, ++ug) {
                    if (!mbar_wait_bounded(&empty[stage], phase ^ 1u, abort_flag, g.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&full[stage], C::P_BYTES + C::Q_BYTES);
                    if (!(g.withhold && blockIdx.x == 0 && ug == 0))      // else its wait can only run out
                        tma_load_2d(sP + stage * C::P_BYTES, &tmP, u * KU, pb * BP, &full[stage]);
                    tma_load_2d(sQ + stage * C::Q_BYTES, &tmQ, u * KU, qb * BN, &full[stage]);
                    // the slot's previous unit lies at least STAGES + 3 back: this stage's last MMAs were
                    // issued after every warp had released the accumulator of the unit two before them,
                    // and with it had done the promotion of the unit before that
                    const uint32_t slot = ug % SLOTS;
                    mbar_arrive_expect_tx(&sfull[slot], (PVEC ? pv : 0u) + (QVEC ? qv : 0u));
                    if (PVEC)
                        bulk_load(sPv + slot * BP, g.p_vec + u * g.p_ld + (int64_t)pb * BP, pv, &sfull[slot]);
                    if (QVEC)
                        bulk_load(sQv + slot * BN, g.q_vec + u * g.q_ld + (int64_t)qb * BN, qv, &sfull[slot]);
                    ++issued;
                    if (++stage == C::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok) {
                // let our own copies land before the block leaves
                for (uint32_t i = 0; i < C::STAGES && i < issued; ++i) {
                    const uint32_t s = (stage + C::STAGES - 1 - i) % C::STAGES;
                    const uint32_t ph = (s < stage) ? phase : (phase ^ 1u);
                    mbar_wait_bounded(&full[s], ph, nullptr, 100000000ull);
                }
                for (uint32_t i = 0; i < C::STAGES && i < issued; ++i) {
                    const uint32_t u = ug - 1 - i;
                    mbar_wait_bounded(&sfull[u % SLOTS], (u / SLOTS) & 1u, nullptr, 100000000ull);
                }
            }
        } else if (warp == 1 && lane == 0) {
            // ---------------------------------------------------- MMA issuer
            uint32_t stage = 0, phase = 0, ug = 0;
            bool ok = true;
            for (int t = t0; ok && t < g.num_tiles; t += tstep) {
                for (int u = u0; u < u1; ++u, ++ug) {
                    const uint32_t b = ug & 1u;
                    if (!mbar_wait_bounded(&tempty[b], ((ug >> 1) & 1u) ^ 1u, abort_flag, g.timeout_ns) ||
                        !mbar_wait_bounded(&full[stage], phase, abort_flag, g.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t p0 = smem_addr(sP + stage * C::P_BYTES);
                    const uint32_t q0 = smem_addr(sQ + stage * C::Q_BYTES);
#pragma unroll
                    for (int k = 0; k < KU / 32; ++k)
                        mma_f8f6f4(tmem_base + b * BN, smem_desc_sw128(p0 + k * 32), smem_desc_sw128(q0 + k * 32),
                                   g.idesc, (uint32_t)k);
                    mma_commit(&empty[stage]);
                    mma_commit(&tfull[b]);
                    if (++stage == C::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // no MMA may still be running when TMEM is released
            mma_commit(drain);
            mbar_wait_bounded(drain, 0, nullptr, 100000000ull);
        }
        __syncwarp();
        if (split > 1) {
            cluster_sync();
            cluster_sync();
        }
    } else {
        // ------------------------------------------------------- promotion
        const int q4 = warp & 3;                         // TMEM lane quarter
        const int prow = q4 * 32 + lane;                 // this thread's row of the tile
        uint32_t ug = 0;
        bool ok = true;
        for (int t = t0; ok && t < g.num_tiles; t += tstep) {
            int pb, qb;
            tile_coords(t, g, pb, qb);
            float acc[C::ACC];
#pragma unroll
            for (int j = 0; j < C::ACC; ++j) acc[j] = 0.0f;
            // block scales: of the tile's 128 rows of b (SWAP: P; BN <= 128 columns lie in one block)
            const float *blk = VECB ? nullptr : g.blk + (SWAP ? pb : (qb * BN) / 128) * g.blk_ld;
            float bs = VECB || u0 >= u1 ? 1.0f : __ldg(blk + u0);
            for (int u = u0; u < u1; ++u, ++ug) {
                const float bcur = bs;
                if (!VECB && u + 1 < u1) bs = __ldg(blk + u + 1);
                const uint32_t slot = ug % SLOTS, b = ug & 1u;
                if (!mbar_wait_bounded(&sfull[slot], (ug / SLOTS) & 1u, abort_flag, g.timeout_ns)) {
                    ok = false;
                    break;
                }
                float r = PVEC ? sPv[slot * BP + prow] : 1.0f;
                if (!VECB) r *= bcur;
                const float *cv = sQv + slot * BN;
                if (!mbar_wait_bounded(&tfull[b], (ug >> 1) & 1u, abort_flag, g.timeout_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t ta = tmem_base + ((uint32_t)(q4 * 32) << 16) + b * BN;
                uint32_t d0[C::CH], d1[C::CH];
                tmem_load<C::CH>(ta, d0);
                tmem_landed<C::CH>(d0);
#pragma unroll
                for (int c = 0; c < C::ACC; c += 2 * C::CH) {
                    const bool two = c + C::CH < C::ACC, more = c + 2 * C::CH < C::ACC;
                    if (two) tmem_load<C::CH>(ta + c + C::CH, d1);
                    if (!two) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&tempty[b]);
                    }
                    promote<C::CH, QVEC>(acc + c, d0, r, cv + c);
                    if (two) {
                        tmem_landed<C::CH>(d1);
                        if (more) {
                            tmem_load<C::CH>(ta + c + 2 * C::CH, d0);
                        } else {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&tempty[b]);
                        }
                        promote<C::CH, QVEC>(acc + c + C::CH, d1, r, cv + c + C::CH);
                        if (more) tmem_landed<C::CH>(d0);
                    }
                }
            }
            if (!ok) break;
            const int p = pb * BP + prow;
            const int q0 = qb * BN;
            if (split > 1) {
                // the last unit's MMAs have completed: nothing reads or writes the ring any more
                float *st = reinterpret_cast<float *>(smem);
#pragma unroll
                for (int j = 0; j < C::ACC; ++j) st[j * C::PITCH + prow] = acc[j];
            } else if (SWAP) {
                const float bv = p < g.P ? bias_of(g, p) : 0.0f;
#pragma unroll
                for (int j = 0; j < C::ACC; ++j)
                    if (p < g.P && q0 + j < g.Q) store_one(g, q0 + j, p, acc[j] + bv);
            } else if (p < g.P) {
                if (g.bias) {
#pragma unroll
                    for (int j = 0; j < C::ACC; ++j)
                        if (q0 + j < g.Q) acc[j] += bias_of(g, q0 + j);
                }
                if (q0 + C::ACC <= g.Q) {
#pragma unroll
                    for (int j = 0; j < C::ACC; j += 8) {
                        float o[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) o[i] = acc[j + i];
                        if (g.out_f32)
                            f8::store8<false>(g.y, (int64_t)p * g.ldy + q0 + j, o, 8);
                        else
                            f8::store8<true>(g.y, (int64_t)p * g.ldy + q0 + j, o, 8);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < C::ACC; ++j)
                        if (q0 + j < g.Q) store_one(g, p, q0 + j, acc[j]);
                }
            }
        }
        __syncwarp();
        if (split > 1) {
            cluster_sync();
            if (ok && t0 < g.num_tiles) {
                int pb, qb;
                tile_coords(t0, g, pb, qb);
                const uint32_t st = smem_addr(smem);
                const int share = BP * BN / split;
                for (int i = (int)threadIdx.x - 128; i < share; i += 32 * C::EPI_WARPS) {
                    const int e = rank * share + i;
                    // consecutive lanes along n, the contiguous axis of y
                    const int r = SWAP ? e % BP : e / BN, c = SWAP ? e / BP : e % BN;
                    float s = 0.0f;
                    for (int k = 0; k < split; ++k) s += peer_ld(st + (c * C::PITCH + r) * 4, (uint32_t)k);
                    const int pp = pb * BP + r, qq = qb * BN + c;
                    if (pp < g.P && qq < g.Q)
                        store_one(g, SWAP ? qq : pp, SWAP ? pp : qq, s + bias_of(g, SWAP ? pp : qq));
                }
            }
            cluster_sync();
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem_base, C::TMEM_COLS);
    if (threadIdx.x == 0 && *abort_flag) status_or(g.status, HIF4_FLAG_TIMEOUT);
}

struct Call {
    const uint8_t *a, *b;
    int64_t M, N, K, lda, ldb;
    const float *sa, *sb;
    int64_t lds_a, lds_b;
    bool a_e5m2, b_e5m2;
};

template <int BN, bool SWAP, bool VECB>
hif4_status launch(const Call &c, Args g, cudaStream_t stream)
{
    using CF = Cfg<BN>;
    const uint8_t *p = SWAP ? c.b : c.a, *q = SWAP ? c.a : c.b;
    g.P = (int)(SWAP ? c.N : c.M);
    g.Q = (int)(SWAP ? c.M : c.N);
    g.num_p = (g.P + BP - 1) / BP;
    g.num_q = (g.Q + BN - 1) / BN;
    g.num_u = (int)f8::blocks_of(c.K);
    if ((int64_t)g.num_p * g.num_q > INT32_MAX / 8) return HIF4_ERR_UNSUPPORTED;
    g.num_tiles = g.num_p * g.num_q;
    g.p_vec = SWAP ? (VECB ? c.sb : nullptr) : c.sa;
    g.p_ld = SWAP ? c.lds_b : c.lds_a;
    g.q_vec = SWAP ? c.sa : (VECB ? c.sb : nullptr);
    g.q_ld = SWAP ? c.lds_a : c.lds_b;
    g.blk = VECB ? nullptr : c.sb;
    g.blk_ld = c.lds_b;
    g.idesc = sm100::idesc_f8_f32(BP, BN, SWAP ? c.b_e5m2 : c.a_e5m2, SWAP ? c.a_e5m2 : c.b_e5m2);

    CUtensorMap tmP, tmQ;
    if (!make_tensor_map_u8_2d_sw128(&tmP, p, (uint64_t)c.K, (uint64_t)g.P, (uint64_t)(SWAP ? c.ldb : c.lda), KU,
                                     BP) ||
        !make_tensor_map_u8_2d_sw128(&tmQ, q, (uint64_t)c.K, (uint64_t)g.Q, (uint64_t)(SWAP ? c.lda : c.ldb), KU,
                                     BN))
        return HIF4_ERR_UNSUPPORTED;            // the driver's encoder refused the layout
    auto k = k_gemm_f8_block<BN, SWAP, VECB>;
    // cheap enough to set on every call, and then right on every device
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)CF::SMEM);
    if (e != cudaSuccess) return cuda_failed(e);

    const int slots = sm_count() * CF::CTAS;
    int split = 1;
    while (split < 8 && (int64_t)g.num_tiles * split * 2 <= slots && g.num_u >= split * 2 * 4) split *= 2;
    g.split = split;
    int64_t grid = (int64_t)g.num_tiles * split;
    if (split == 1 && grid > slots) grid = slots;

    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(CF::THREADS);
    cfg.dynamicSmemBytes = CF::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = split > 1 ? 2 : 1;
    const cudaError_t le = cudaLaunchKernelEx(&cfg, k, tmP, tmQ, g);
    if (le != cudaSuccess) {
        (void)cudaGetLastError();
        return cuda_failed(le);
    }
    return launch_status();
}

template <bool VECB>
hif4_status dispatch(const Call &c, const Args &g, cudaStream_t s)
{
    if (c.M <= 16) return launch<16, true, VECB>(c, g, s);
    if (c.M <= 32) return launch<32, true, VECB>(c, g, s);
    if (c.M <= 64) return launch<64, true, VECB>(c, g, s);
    return launch<128, false, VECB>(c, g, s);
}

} // namespace gemm8b
} // namespace hif4

using namespace hif4;

extern "C" hif4_status hif4_gemm_f8_block(const uint8_t *a, hif4_f8_format a_fmt, int64_t M, int64_t K, int64_t lda,
                                          const float *sa, int64_t lds_a, const uint8_t *b, hif4_f8_format b_fmt,
                                          int64_t N, int64_t ldb, const float *sb, int64_t lds_b,
                                          int32_t b_block_rows, const void *bias, void *y, int64_t ldy,
                                          uint32_t flags, uint32_t *status, hif4_stream_t stream)
{
    using namespace gemm8b;
    if (M < 0 || N < 0 || K < 0 || !f8::valid_fmt(a_fmt) || !f8::valid_fmt(b_fmt)) return HIF4_ERR_INVALID_ARG;
    if (b_block_rows != 1 && b_block_rows != 128) return HIF4_ERR_INVALID_ARG;
    if (flags & ~(uint32_t)HIF4_LINEAR_OUT_F32) return HIF4_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return HIF4_OK;
    if (K == 0) return HIF4_ERR_SHAPE;
    if (!a || !b || !sa || !sb || !y) return HIF4_ERR_INVALID_ARG;
    const bool vecb = b_block_rows == 1;
    const int64_t units = f8::blocks_of(K);
    if (lda < K || ldb < K || ldy < N || lds_a < M || lds_b < (vecb ? N : units)) return HIF4_ERR_SHAPE;
    const int64_t ysz = (flags & HIF4_LINEAR_OUT_F32) ? 4 : 2;
    if (!aligned16(a) || !aligned16(b) || !aligned16(y) || !aligned16(sa) || lda % 16 || ldb % 16 || lds_a % 4 ||
        (ldy * ysz) % 16 || (bias && !aligned_to(bias, 2)))
        return HIF4_ERR_ALIGNMENT;
    if (vecb ? (!aligned16(sb) || lds_b % 4) : !aligned_to(sb, 4)) return HIF4_ERR_ALIGNMENT;
    if (M > INT32_MAX / 2 || N > INT32_MAX / 2 || K > INT32_MAX / 2) return HIF4_ERR_UNSUPPORTED;

    Args g{};
    g.bias = static_cast<const uint16_t *>(bias);
    g.y = y;
    g.ldy = ldy;
    g.out_f32 = (flags & HIF4_LINEAR_OUT_F32) ? 1u : 0u;
    g.status = status;
    g.withhold = wait_test_withhold();
    g.timeout_ns = wait_limit_ns(TIMEOUT_NS);
    const Call c{a, b, M, N, K, lda, ldb, sa, sb, lds_a, lds_b, a_fmt == HIF4_E5M2, b_fmt == HIF4_E5M2};
    return vecb ? dispatch<true>(c, g, reinterpret_cast<cudaStream_t>(stream))
                : dispatch<false>(c, g, reinterpret_cast<cudaStream_t>(stream));
}
