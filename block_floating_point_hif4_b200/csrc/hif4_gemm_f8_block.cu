// hif4_gemm_f8_block.cu — matrix product of FP8 operands with one FP32 scale
// per block of 128:
//   y[m][n] = bias[n] + sum_u sa[u][m] sb[u, n] sum_{k in block u} a[m][k] b[n][k]
// with 1 x 128 blocks on a and 128 x 128 or 1 x 128 blocks on b.
//
// FP32 scales cannot enter the tensor core (its block scales are powers of
// two), so each 128-deep product ("unit") goes to a TMEM accumulator of its own
// (tcgen05 kind::f8f6f4, FP32 accumulation), and promotion warps read it back
// and add  scale * P  into FP32 totals held in registers: one FMA per output
// element and unit, and a multiplication where b has a scale per row, for its
// product with a's.  There a thread holds four rows of a quarter of the columns
// (16x256b reads) and not one row (32x32b): a scale read from shared memory
// serves four rows, else those reads take longer than the MMAs (5120 x 5120 x
// 14391 on a cool card: 592 us with one row per thread, 489 with four, 440 in a
// trial copy without the scales' reads and products; a call, with the clock that
// the power cap leaves, takes 571 with four).
//
// Roles: warp 0 issues the TMA loads (128-byte swizzled operand tiles into a
// ring), warps 1 and 2 the MMAs into two alternating accumulators, warp 3 the
// copies of the scale vectors (a ring of their own, four units to a slot);
// warps 4 and up promote.  A tile is 128 rows of one operand (P) by BN rows of
// the other (Q).
//   SWAP (BN 16, 32; up to 32 rows of a): the weight is P, so that it fills the
//     MMA's 128 rows, and the tokens are Q.  Up to two CTAs per SM stream the
//     weight: 1 x 13824 x 5120 in 16.0 us, 4.4 TB/s, 5 of them before the first
//     block starts or after the last has ended.
//   128 x 128 tiles: short products of more rows.
//   PAIR: 256 x 256 or 256 x 192 tiles of a cluster of two CTAs (tcgen05
//     cta_group::2).  Each CTA loads 128 rows of P and half of Q's, 32 KB a unit
//     for the larger tile instead of the 48 KB of a 128 x 256 tile: an SM takes
//     in about 61 bytes a cycle, and a unit is 512 cycles of MMA.
//
// When there are too few tiles for the GPU, a cluster of S CTAs shares a tile:
// each takes a contiguous part of K, leaves its FP32 totals in its shared
// memory, and after a cluster barrier each adds up its share of the tile over
// the CTAs in rank order (distributed shared memory).  The order of the sum is
// fixed and no workspace is needed.
//
// What bounds the large products, measured at 57600 x 13824 x 5120 in cycles of
// the SM clock: a unit takes 930 cycles, whether in one launch (1.60 GHz, 3850 us)
// or sustained (1.37 GHz, 4570 us), where its MMAs need 512.  The MMA warps wait
// 1300 of the 1910 cycles between two units of theirs for a free accumulator and 85
// for operands; a promotion warp waits 200 of 960 cycles for MMAs (trial copy with
// clocks).  Without the promotion's FMAs a unit takes 650 cycles, without its TMEM
// reads as well 644: the FMAs and the hand-off of the two accumulators are the
// bound, and the 1 kW power cap then sets the clock.  Half of the operands' bytes
// changes nothing (925).  A 128 x 256 tile of one CTA measured 3 to 8 % slower.
//
// A unit's MMAs announce their completion once, on the barrier of the stage
// they read (in both CTAs of a pair): it hands the stage back to the producer
// and the accumulator to the promotion warps.
//
// Every mbarrier wait is bounded (4 s); a role that gives up sets the block's
// abort flag, the MMA warps drain their MMAs, the producers wait until those
// warps have left and then for every copy and every completion still under way
// (in a pair some of them arrive from the other CTA), every thread still meets
// the cluster barriers, and HIF4_FLAG_TIMEOUT is raised.
#include <mutex>

#include <cuda_fp16.h>

#include "hif4_f8.cuh"
#include "hif4_pdl.cuh"
#include "hif4_sm100_f8.cuh"

namespace hif4 {

bool make_tensor_map_u8_2d_sw128(CUtensorMap *map, const void *base, uint64_t inner, uint64_t outer,
                                 uint64_t row_stride_bytes, uint32_t box_inner, uint32_t box_outer);

namespace gemm8b {

constexpr int BP = 128;                         // rows of a CTA's tile (MMA M, of each CTA)
constexpr int KU = 128;                         // K elements (bytes) per unit and per stage
constexpr int SG = 4;                           // units per slot of the scale ring
constexpr int SLOTS = 2;
constexpr int ST_BYTES = 2048;                 // a promotion warp's staging of its stores: 32 rows of 64 bytes
constexpr int GROUP = 16;                       // raster: P tiles per group
constexpr float FLT_TOP = 3.402823466e38f;
constexpr uint64_t TIMEOUT_NS = 4000000000ull;
constexpr uint64_t DRAIN_NS = 20000000ull;

// BN: columns of the tile.  PAIR: two CTAs share a tile of 256 rows (each holds 128 of them and half of
// Q's rows).
template <int BN, bool VECB, bool PAIR, bool SWAP>
struct Cfg {
    static constexpr int EPI_WGS = BN >= 128 ? 2 : 1;                 // promotion warpgroups
    static constexpr bool SPLITS = !PAIR && BN <= 128;                // may share K over a cluster
    static constexpr int EPI_WARPS = 4 * EPI_WGS;
    static constexpr int THREADS = 128 + 32 * EPI_WARPS;
    static constexpr int ACC = BN / EPI_WGS;    // totals per promotion thread
    static constexpr int CTAS = BN <= 32 ? 2 : 1;                // per SM
    static constexpr int STAGES = PAIR ? (BN > 192 ? 6 : 7) : 5;
    static constexpr int CH = 16;                // values per thread and TMEM read
    static constexpr int NCH = ACC / CH;
    static constexpr bool FRAG = VECB && !SWAP; // a thread's totals are those of 4 rows, not of one
    // registers: the promotion warps take what the producer's warpgroup gives back; the shares add up to
    // what the launch brings along, 384 threads x 168, or less (192 columns with a scale per row of b: 69 us
    // with 96 and 200, 74 with 72 and 216, 512 x 5120 x 13824; 256 columns: 589 and 577, 5120 x 5120 x 14391)
    static constexpr int REG_LOW = BN < 192 ? 0 : VECB && BN == 192 ? 96 : 72;
    static constexpr int REG_HIGH = BN < 192 ? 0 : VECB && BN == 192 ? 200 : 216;
    static constexpr int P_BYTES = BP * KU;
    static constexpr int Q_BYTES = BN * KU / (PAIR ? 2 : 1);
    static constexpr int RING = STAGES * (P_BYTES + Q_BYTES);
    static constexpr int TMEM_COLS = BN > 128 ? 512 : 2 * BN;         // a power of two
    static constexpr bool TWO_BLOCKS = BN == 192;                     // a thread's columns lie in up to two blocks of b
    static constexpr int BARS = 2 * STAGES + 2 + 2 + 2 * SLOTS;
    static constexpr bool PVEC = !SWAP || VECB, QVEC = SWAP || VECB;  // P / Q carry scale vectors
    static constexpr int PV = PVEC ? SLOTS * SG * BP : 0, QV = QVEC ? SLOTS * SG * BN : 0;
    static constexpr int STORE = SWAP ? 0 : EPI_WARPS * ST_BYTES;
    static constexpr size_t SMEM = (size_t)RING + STORE + (PV + QV) * 4 + BARS * 8 + 64 + 1024;
    static_assert(!SPLITS || (SWAP ? BN * (BP + 4) : BP * (BN + 4)) * 4 <= RING,
                  "the staged totals reuse the operand ring");
    static_assert(SMEM <= 227 * 1024, "shared memory of one CTA");
};

struct Args {
    int P, Q;                                   // rows of the two operands
    int K;
    const uint8_t *p_codes, *q_codes;           // the operands again, for sum_again()
    int64_t p_codes_ld, q_codes_ld;
    uint32_t p_e5m2, q_e5m2;
    int num_p, num_q, num_u, num_tiles;
    int split;                                  // CTAs that share a tile's K (the cluster)
    const float *p_vec, *q_vec;                 // scale vectors [num_u][ld] (null: block scales)
    int64_t p_ld, q_ld;
    const float *blk;                           // 128 x 128 block scales [row block][num_u ..]
    int64_t blk_ld;
    int blk_rows;
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

__device__ __forceinline__ void mul2(float &d0, float &d1, float a0, float a1, float b0, float b1)
{
    asm("{\n\t.reg .b64 pa, pb, pd;\n\t"
        "mov.b64 pa, {%2, %3};\n\tmov.b64 pb, {%4, %5};\n\t"
        "mul.rn.f32x2 pd, pa, pb;\n\tmov.b64 {%0, %1}, pd;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
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

__device__ __forceinline__ float4 peer_ld4(uint32_t local, uint32_t rank)
{
    uint32_t a;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(local), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}

template <int N>
__device__ __forceinline__ void reg_dec()
{
    if constexpr (N > 0) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <int N>
__device__ __forceinline__ void reg_inc()
{
    if constexpr (N > 0) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
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

// Stores the N totals of each of a warp's 32 rows (r0 + lane), W columns (64 bytes) at a time.
template <int N, int W, bool F32, bool FRAG>
__device__ __forceinline__ void store_rows(const Args &g, uint8_t *st, const float (&acc)[N], int lane, int64_t r0,
                                           int q0)
{
    constexpr int E = F32 ? 4 : 2;
    const int row = lane >> 2, piece = lane & 3;
#pragma unroll
    for (int j = 0; j < N; j += W) {
        if (q0 + j >= g.Q) break;
        __syncwarp();
        if constexpr (FRAG) {
#pragma unroll
            for (int i = 0; i < W / 2; ++i) {   // 8 columns n of row r, two of them in this thread
                const int n = i % (W / 8), r = i / (W / 8) * 8 + row;
                const float *v = acc + (j / 32 * 2 + i / (W / 4)) * 16 + (j % 32 / 8 + n) * 4 + (i / (W / 8) & 1) * 2;
                const int at = F32 ? n * 2 + piece / 2 : n;     // the 16-byte piece they belong to
                uint8_t *d = st + r * 64 + ((at ^ (r >> 1)) & 3) * 16;
                if (F32)
                    *reinterpret_cast<float2 *>(d + (piece & 1) * 8) = make_float2(v[0], v[1]);
                else
                    *reinterpret_cast<uint32_t *>(d + piece * 4) = f8::pack_bf16_rn(v[0], v[1]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4 && !FRAG; ++i) {
            uint4 w;
            const float *v = acc + j + i * (W / 4);
            if (F32)
                w = make_uint4(f_bits(v[0]), f_bits(v[1]), f_bits(v[2]), f_bits(v[3]));
            else
                w = make_uint4(f8::pack_bf16_rn(v[0], v[1]), f8::pack_bf16_rn(v[2], v[3]),
                               f8::pack_bf16_rn(v[F32 ? 0 : 4], v[F32 ? 0 : 5]),
                               f8::pack_bf16_rn(v[F32 ? 0 : 6], v[F32 ? 0 : 7]));
            *reinterpret_cast<uint4 *>(st + lane * 64 + ((i ^ (lane >> 1)) & 3) * 16) = w;
        }
        __syncwarp();
        const int col = q0 + j + piece * (W / 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = row + i * 8;
            const uint4 w = *reinterpret_cast<const uint4 *>(st + r * 64 + ((piece ^ (r >> 1)) & 3) * 16);
            if (r0 + r < g.P) {
                uint8_t *dst = static_cast<uint8_t *>(g.y) + ((r0 + r) * g.ldy + col) * E;
                if (col + W / 4 <= g.Q) {
                    *reinterpret_cast<uint4 *>(dst) = w;
                } else {
                    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int k = 0; k < W / 4; ++k)
                        if (col + k < g.Q) {
                            if (F32)
                                reinterpret_cast<uint32_t *>(dst)[k] = a[k & 3];
                            else
                                reinterpret_cast<uint16_t *>(dst)[k] = (uint16_t)(a[(k >> 1) & 3] >> (16 * (k & 1)));
                        }
                }
            }
        }
    }
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

// The factors of the 16 values that a read of 16 rows and 32 columns leaves in a thread: rows l / 4 (scale r[0])
// and l / 4 + 8 (r[1]) of four pairs of columns (scales w).
__device__ __forceinline__ void frag_factors(float (&f)[16], const float *r, const float2 (&w)[4])
{
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        mul2(f[4 * k], f[4 * k + 1], w[k].x, w[k].y, r[0], r[0]);
        mul2(f[4 * k + 2], f[4 * k + 3], w[k].x, w[k].y, r[1], r[1]);
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

// The first `valid` of 4 values at columns n .. n + 3 (n a multiple of 4).
__device__ __forceinline__ void store4(const Args &g, int64_t m, int n, const float (&v)[4], int valid)
{
    if (valid >= 4) {
        if (g.out_f32)
            *reinterpret_cast<float4 *>(static_cast<float *>(g.y) + m * g.ldy + n) =
                make_float4(v[0], v[1], v[2], v[3]);
        else
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(g.y) + m * g.ldy + n) =
                make_uint2(f8::pack_bf16_rn(v[0], v[1]), f8::pack_bf16_rn(v[2], v[3]));
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < valid) store_one(g, m, n + k, v[k]);
    }
}

__device__ __forceinline__ float bias_of(const Args &g, int n)
{
    return g.bias ? bits_f((uint32_t)__ldg(g.bias + n) << 16) : 0.0f;
}

// ---- Products of scales that overflow.  The tiles form sa sb first, one factor for an element's block sum (or for a
// row's).  Where that is infinite although both scales are finite, the term can still be an ordinary number, or 0.  A CTA
// that met such a product goes over its tiles once they are stored, and sums the elements concerned again, one by one.
// It is seen on a row's factor, or, where each column has a factor of its own, on a total that is not finite.  Nothing of
// it is in the loop over the units: a second form of that loop for large scales took 682 us instead of 597 (8192 x 13824
// x 5120); with the warp that copies the scales looking at them it was 629 instead of 617, and 600 instead of 570 (5120 x
// 5120 x 14391).  As it is: 618 instead of 617, and 586 instead of 576.

// Values of two codes (the low byte first).
__device__ __forceinline__ float2 code_values(uint32_t c, bool e5m2)
{
    uint32_t h;
    if (e5m2)
        asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
    else
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// sum a[k] b[k] over n codes (both 16-byte aligned)
__device__ __forceinline__ float code_sum(const uint8_t *a, const uint8_t *b, int n, bool a_e5m2, bool b_e5m2)
{
    float sum = 0.0f;
    int k = 0;
    for (; k + 16 <= n; k += 16) {
        const uint4 v = *reinterpret_cast<const uint4 *>(a + k), w = *reinterpret_cast<const uint4 *>(b + k);
        const uint32_t x[4] = {v.x, v.y, v.z, v.w}, y[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 c = code_values(x[i >> 1] >> (16 * (i & 1)), a_e5m2);
            const float2 d = code_values(y[i >> 1] >> (16 * (i & 1)), b_e5m2);
            sum = fmaf(c.x, d.x, fmaf(c.y, d.y, sum));
        }
    }
    for (; k < n; ++k) sum = fmaf(code_values(a[k], a_e5m2).x, code_values(b[k], b_e5m2).x, sum);
    return sum;
}

// The scales of element (p, q) in unit u.
__device__ __forceinline__ float2 scales_of(const Args &g, int64_t p, int64_t q, int u)
{
    return make_float2(g.p_vec ? g.p_vec[u * g.p_ld + p] : g.blk[p / 128 * g.blk_ld + u],
                       g.q_vec ? g.q_vec[u * g.q_ld + q] : g.blk[q / 128 * g.blk_ld + u]);
}

__device__ __forceinline__ bool overflows(float2 s)
{
    return fabsf(s.x * s.y) > FLT_TOP && fabsf(s.x) <= FLT_TOP && fabsf(s.y) <= FLT_TOP;
}

// Whether row p has a scale that can be part of an overflow (the other one is finite).
__device__ __forceinline__ bool may_overflow(const Args &g, int64_t p)
{
    bool may = false;
    for (int u = 0; u < g.num_u; ++u) may |= fabsf(scales_of(g, p, 0, u).x) > 1.0f;
    return may;
}

// The total of an element over all units, as if no product of scales could overflow; false if none does.
__device__ __forceinline__ bool sum_again(const Args &g, int64_t p, int64_t q, float &total)
{
    int u = 0;
    while (u < g.num_u && !overflows(scales_of(g, p, q, u))) ++u;
    if (u == g.num_u) return false;
    total = 0.0f;
#pragma unroll 1
    for (u = 0; u < g.num_u; ++u) {
        float sum = code_sum(g.p_codes + p * g.p_codes_ld + u * KU, g.q_codes + q * g.q_codes_ld + u * KU,
                             min(KU, g.K - u * KU), g.p_e5m2, g.q_e5m2);
        const float2 s = scales_of(g, p, q, u);
        float f = s.x * s.y;
        if (overflows(s)) {
            // Both are above 1.  2^40 goes from the one to the sum (below 2^40, and at least 2^-32 if not 0); what is
            // too large even so meets a sum that takes it past the largest number anyway, or 0.
            sum *= 1099511627776.0f;
            f = fminf(fmaxf(s.x * (1.0f / 1099511627776.0f) * s.y, -FLT_TOP), FLT_TOP);
        }
        total = fmaf(sum, f, total);
    }
    return true;
}

template <bool SWAP>
__device__ __forceinline__ void store_again(const Args &g, int64_t p, int64_t q)
{
    float v;
    if (p < g.P && q < g.Q && sum_again(g, p, q, v)) {
        const int n = (int)(SWAP ? p : q);
        store_one(g, SWAP ? q : p, n, v + bias_of(g, n));
    }
}

// All elements of a CTA's tiles.
template <int BN, bool SWAP, bool PAIR>
__device__ __forceinline__ void tiles_again(const Args &g, int t0, int tstep, int rank)
{
    for (int t = t0; t < g.num_tiles; t += tstep) {
        int pb, qb;
        tile_coords(t, g, pb, qb);
        for (int i = threadIdx.x; i < BP * (BN / 16); i += blockDim.x) {            // 16 elements of a row
            const int p = (PAIR ? pb * 2 + rank : pb) * BP + i % BP, q = qb * BN + i / BP * 16;
            if (p < g.P && may_overflow(g, p))
#pragma unroll 1
                for (int j = 0; j < 16; ++j) store_again<SWAP>(g, p, q + j);
        }
    }
}

template <int BN, bool SWAP, bool VECB, bool PAIR>
__global__ void __launch_bounds__(Cfg<BN, VECB, PAIR, SWAP>::THREADS, Cfg<BN, VECB, PAIR, SWAP>::CTAS)
k_gemm_f8_block(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                const __grid_constant__ Args g)
{
    using namespace sm100;
    using C = Cfg<BN, VECB, PAIR, SWAP>;
    constexpr bool PVEC = C::PVEC, QVEC = C::QVEC;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sP = smem;
    uint8_t *sQ = sP + C::STAGES * C::P_BYTES;
    uint8_t *sSt = smem + C::RING;
    float *sPv = reinterpret_cast<float *>(sSt + C::STORE);               // [SLOTS][SG][BP]
    float *sQv = sPv + C::PV;                                             // [SLOTS][SG][BN]
    uint64_t *full = reinterpret_cast<uint64_t *>(sQv + C::QV);
    uint64_t *done = full + C::STAGES;                                    // the MMAs that read a stage have completed
    uint64_t *tempty = done + C::STAGES;
    uint64_t *drain = tempty + 2;
    uint64_t *sfull = drain + 2;
    uint64_t *sempty = sfull + SLOTS;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(sempty + SLOTS);
    volatile uint32_t *abort_flag = tmem_holder + 1;
    volatile uint32_t *again = tmem_holder + 2;                           // a product of scales may have overflowed

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&done[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&tempty[a], C::EPI_WARPS * (PAIR ? 2 : 1));
            mbar_init(&drain[a], 1);
        }
        for (int s = 0; s < SLOTS; ++s) {
            mbar_init(&sfull[s], 1);
            mbar_init(&sempty[s], C::EPI_WARPS);
        }
        *abort_flag = 0u;
        *again = 0u;
        fence_barrier_init();
        prefetch_tensormap(&tmP);
        prefetch_tensormap(&tmQ);
    }
    // Scales of rows past the last one are never copied: 0, so that nothing looks like an overflow there.
    for (int i = threadIdx.x; i < (C::PV + C::QV) / 4; i += C::THREADS)
        reinterpret_cast<float4 *>(sPv)[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    fence_proxy_async();
    if (warp == 1) {
        if (PAIR) {
            tmem_alloc_pair(tmem_holder, C::TMEM_COLS);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(tmem_holder, C::TMEM_COLS);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    if (PAIR) cluster_sync();                   // the barriers of both CTAs are ready
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    pdl_enter();

    const int split = C::SPLITS ? g.split : 1;
    const int rank = PAIR || split > 1 ? (int)cluster_rank() : 0;
    const int share = PAIR ? 2 : split;         // CTAs per tile
    const int t0 = blockIdx.x / share, tstep = gridDim.x / share;
    const int u0 = PAIR ? 0 : (int)((int64_t)g.num_u * rank / split);
    const int u1 = PAIR ? g.num_u : (int)((int64_t)g.num_u * (rank + 1) / split);
    const int p_of = PAIR ? 2 : 1, p_at = PAIR ? rank : 0;                // this CTA's 128 rows of a tile

    if (warp < 4) {
        reg_dec<C::REG_LOW>();
        if (warp == 0) {
            // ---------------------------------------------------- operands
            uint32_t stage = 0, phase = 0;
            int issued = 0;
            bool ok = true;
            for (int t = t0; ok && t < g.num_tiles; t += tstep) {
                int pb, qb;
                tile_coords(t, g, pb, qb);
                const int prow = (pb * p_of + p_at) * BP, qrow = qb * BN + (PAIR ? rank * (BN / 2) : 0);
                for (int u = u0; u < u1; ++u) {
                    if (!mbar_wait_spin(&done[stage], phase ^ 1u, abort_flag, g.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    if (elect_one()) {
                        // a withheld copy's wait can only run out
                        const bool skip = g.withhold && blockIdx.x == 0 && issued == 0;
                        if (PAIR) {
                            // both CTAs' copies complete on the issuing CTA's barrier
                            if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * (C::P_BYTES + C::Q_BYTES));
                            const uint32_t bar = peer_addr(smem_addr(&full[stage]), 0);
                            if (!skip) tma_load_2d_pair(sP + stage * C::P_BYTES, &tmP, u * KU, prow, bar);
                            tma_load_2d_pair(sQ + stage * C::Q_BYTES, &tmQ, u * KU, qrow, bar);
                        } else {
                            mbar_arrive_expect_tx(&full[stage], C::P_BYTES + C::Q_BYTES);
                            if (!skip) tma_load_2d(sP + stage * C::P_BYTES, &tmP, u * KU, prow, &full[stage]);
                            tma_load_2d(sQ + stage * C::Q_BYTES, &tmQ, u * KU, qrow, &full[stage]);
                        }
                    }
                    __syncwarp();
                    ++issued;
                    if (++stage == C::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // Whether the tiles are done or a wait gave up: the copies land before the block leaves (a pair's all
            // complete on the issuing CTA's barriers), and so do the completions of the MMAs.
            // Each lane waits for a stage.
            const uint32_t mine = (stage + C::STAGES - 1 - lane % C::STAGES) % C::STAGES;
            const uint32_t ph = (mine < stage) ? phase : (phase ^ 1u);
            const auto landed = [&](volatile uint32_t *flag, uint64_t limit) {
                bool all = true;
                if (lane < C::STAGES && lane < issued) {
                    if (!PAIR || rank == 0) all = mbar_wait_bounded(&full[mine], ph, flag, limit);
                    if (all || !flag) all &= mbar_wait_bounded(&done[mine], ph, flag, limit);
                }
                return __all_sync(0xFFFFFFFFu, all) != 0;
            };
            const bool all = landed(abort_flag, g.timeout_ns);
            // Once a wait has given up, the MMA warps may still issue a unit that the promotion warps' last
            // hand-off lets through.  Their drain says that they have left, not that every completion that they
            // asked for has arrived, so those are waited for again then, whatever the abort flag says.
            if (lane < 2) mbar_wait_bounded(&drain[lane], 0, nullptr, 2 * g.timeout_ns + DRAIN_NS);
            __syncwarp();
            if (!all) landed(nullptr, DRAIN_NS);
        } else if (warp == 3) {
            // ---------------------------------------------------- scales
            // A slot holds those of SG consecutive units of a tile (the last one of a tile maybe fewer).
            uint32_t slot = 0, phase = 0;
            bool ok = true;
            for (int t = t0; ok && t < g.num_tiles; t += tstep) {
                int pb, qb;
                tile_coords(t, g, pb, qb);
                const int prow = (pb * p_of + p_at) * BP, qrow = qb * BN;
                // scales of the tile's rows (a pair's second CTA may lie past the last row: none): whole 16-byte
                // pieces by bulk copy, the last 1 to 3 one by one, so that nothing past the last row is read
                const int pn = PVEC ? max(0, min(BP, g.P - prow)) : 0, qn = QVEC ? min(BN, g.Q - qrow) : 0;
                const int pw = pn & ~3, qw = qn & ~3;
                for (int u = u0; u < u1; u += SG) {
                    if (!mbar_wait_spin(&sempty[slot], phase ^ 1u, abort_flag, g.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    const int n = min(SG, u1 - u);
                    if ((pn | qn) & 3) {                // lane = 8 x unit + 4 x operand + scale
                        const int i = lane >> 3, k = lane & 3;
                        const bool q = lane & 4;
                        if (i < n && k < ((q ? qn : pn) & 3)) {
                            if (q)
                                async_load4(sQv + (slot * SG + i) * BN + qw + k, g.q_vec + (u + i) * g.q_ld + qrow + qw + k,
                                            &sfull[slot]);
                            else
                                async_load4(sPv + (slot * SG + i) * BP + pw + k, g.p_vec + (u + i) * g.p_ld + prow + pw + k,
                                            &sfull[slot]);
                        }
                        __syncwarp();
                    }
                    if (elect_one()) {
                        mbar_arrive_expect_tx(&sfull[slot], (uint32_t)(n * (pw + qw) * 4));
                        for (int i = 0; i < n; ++i) {
                            if (PVEC && pw > 0)
                                bulk_load(sPv + (slot * SG + i) * BP, g.p_vec + (u + i) * g.p_ld + prow, pw * 4,
                                          &sfull[slot]);
                            if (QVEC && qw > 0)
                                bulk_load(sQv + (slot * SG + i) * BN, g.q_vec + (u + i) * g.q_ld + qrow, qw * 4,
                                          &sfull[slot]);
                        }
                    }
                    __syncwarp();
                    if (++slot == SLOTS) {
                        slot = 0;
                        phase ^= 1u;
                    }
                }
            }
            // (a slot that was never filled counts as landed: its barrier's phase before the first)
            for (uint32_t s = 0; s < (uint32_t)SLOTS; ++s)
                mbar_wait_bounded(&sfull[s], s < slot ? phase : (phase ^ 1u), nullptr, DRAIN_NS);
        } else if (!PAIR || rank == 0) {
            // ---------------------------------------------------- MMA issuers
            // One warp for each accumulator: issuing a unit's MMAs and commits takes one thread as long
            // as the tensor core takes to run them, so the two take turns.  The loop is warp-uniform and
            // one elected lane issues.
            const uint32_t b = warp - 1;
            uint32_t stage = 0, phase = 0, tph = 1;
            const uint64_t pd0 = smem_desc_sw128(smem_addr(sP)), qd0 = smem_desc_sw128(smem_addr(sQ));
            const uint32_t d = tmem_base + b * BN;
            bool ok = true;
            for (int t = t0; ok && t < g.num_tiles; t += tstep) {
                for (int u = u0; u < u1; ++u) {
                    if (((uint32_t)(u - u0) & 1u) == b) {
                        if (!mbar_wait_spin(&tempty[b], tph, abort_flag, g.timeout_ns) ||
                            !mbar_wait_spin(&full[stage], phase, abort_flag, g.timeout_ns)) {
                            ok = false;
                            break;
                        }
                        tph ^= 1u;
                        tc_fence_after();
                        const uint64_t pd = pd0 + stage * (C::P_BYTES / 16), qd = qd0 + stage * (C::Q_BYTES / 16);
                        if (elect_one()) {
                            if (PAIR) {
#pragma unroll
                                for (int k = 0; k < KU / 32; ++k)
                                    mma_f8f6f4_pair(d, pd + 2 * k, qd + 2 * k, g.idesc, k > 0);
                                mma_commit_pair(&done[stage]);
                            } else {
#pragma unroll
                                for (int k = 0; k < KU / 32; ++k)
                                    mma_f8f6f4(d, pd + 2 * k, qd + 2 * k, g.idesc, k > 0);
                                mma_commit(&done[stage]);
                            }
                        }
                        __syncwarp();
                    }
                    if (++stage == C::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // no MMA may still be running when TMEM is released
            if (elect_one()) {
                if (PAIR)
                    mma_commit_pair(&drain[b]);
                else
                    mma_commit(&drain[b]);
            }
            __syncwarp();
            mbar_wait_bounded(&drain[b], 0, nullptr, DRAIN_NS);
        }
        __syncwarp();
        if (C::SPLITS && split > 1) {
            cluster_sync();
            cluster_sync();
        }
    } else {
        // ------------------------------------------------------- promotion
        reg_inc<C::REG_HIGH>();
        const int q4 = warp & 3;                         // TMEM lane quarter
        const int prow = q4 * 32 + lane;                 // this thread's row of the CTA's tile
        const int c0 = (warp / 4 - 1) * C::ACC;          // and its first column
        const uint32_t ta = tmem_base + ((uint32_t)(q4 * 32) << 16) + c0;
        const uint32_t rel = PAIR ? peer_addr(smem_addr(tempty), 0) : smem_addr(tempty);   // of the issuing CTA
        // Unit by unit through the stages' completions.  None is missed: a stage is read again only by a unit
        // STAGES later, and that one waits for an accumulator that a unit after this one has left.
        uint32_t slot = 0, sphase = 0, stage = 0, phase = 0;
        bool ok = true;
        for (int t = t0; ok && t < g.num_tiles; t += tstep) {
            int pb, qb;
            tile_coords(t, g, pb, qb);
            pb = pb * p_of + p_at;
            float acc[C::ACC];
#pragma unroll
            for (int j = 0; j < C::ACC; ++j) acc[j] = 0.0f;
            // block scales: of the tile's 128 rows of b (SWAP), of this thread's columns, which lie in one
            // block (ACC 64, 128) or have their second block begin `turn` columns on
            const int first = SWAP ? pb : (qb * BN + c0) / 128;
            const float *blk = VECB ? nullptr : g.blk + min(first, g.blk_rows - 1) * g.blk_ld;
            const float *blk2 = VECB ? nullptr : g.blk + min(first + 1, g.blk_rows - 1) * g.blk_ld;
            const int turn = 128 - (qb * BN + c0) % 128;
            // Lane l holds those of units u0 + 32 i + l: a global load for each unit would cost its whole
            // latency, since the wait for the accumulator's reads waits for it too.
            float bs = 1.0f, bs2 = 1.0f;
            for (int u = u0; u < u1; u += SG) {
                if (!VECB && ((u - u0) & 31) == 0) {
                    bs = u + lane < u1 ? __ldg(blk + u + lane) : 0.0f;
                    if (C::TWO_BLOCKS) bs2 = u + lane < u1 ? __ldg(blk2 + u + lane) : 0.0f;
                }
                ok = mbar_wait_spin(&sfull[slot], sphase, abort_flag, g.timeout_ns);
                float rc[SG], rc2[SG];
#pragma unroll
                for (int i = 0; i < SG && !C::FRAG; ++i) {
                    rc[i] = PVEC ? sPv[(slot * SG + i) * BP + prow] : 1.0f;
                    if (C::TWO_BLOCKS && !VECB) rc2[i] = rc[i] * __shfl_sync(0xFFFFFFFFu, bs2, ((u - u0) & 31) + i);
                    if (!VECB) rc[i] *= __shfl_sync(0xFFFFFFFFu, bs, ((u - u0) & 31) + i);
                }
                const float *cv = sQv + slot * SG * BN + c0;
                // Unrolled over the group, so that the accumulator of each unit is known at compile time.
#pragma unroll
                for (int i = 0; i < SG; ++i) {
                    if (u + i < u1) {
                        constexpr int odd[4] = {0, 1, 0, 1};
                        const uint32_t b = odd[i & 3];
                        // (after a time-out the group is finished on whatever lies there, and then left)
                        ok &= mbar_wait_spin(&done[stage], phase, abort_flag, g.timeout_ns);
                        if (++stage == C::STAGES) {
                            stage = 0;
                            phase ^= 1u;
                        }
                        tc_fence_after();
                        // the accumulator is free once its last read has landed
                        const auto release = [&] {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) {
                                if (PAIR)
                                    mbar_arrive_remote(rel + b * 8);
                                else
                                    mbar_arrive(&tempty[b]);
                            }
                        };
                        if constexpr (C::FRAG) {
                            // Chunk c: rows 0 - 15 (c even) or 16 - 31 of the warp, 32 columns from 32 (c / 2).
                            // The next chunk's read and factors go out before this one's additions.
                            const float *cols = cv + i * BN + (lane & 3) * 2;
                            const float *rows = sPv + (slot * SG + i) * BP + q4 * 32 + lane / 4;
                            const float r[4] = {rows[0], rows[8], rows[16], rows[24]};
                            float2 w[4];
                            float f[2][16];
                            uint32_t d[2][16];
#pragma unroll
                            for (int k = 0; k < 4; ++k) w[k] = *reinterpret_cast<const float2 *>(cols + 8 * k);
                            tmem_ld_16x256b_x4(ta + b * BN, d[0]);
                            frag_factors(f[0], r, w);
#pragma unroll
                            for (int c = 0; c < C::NCH; ++c) {
                                const int n = c + 1;
                                tmem_landed<16>(d[c & 1]);
                                if (n < C::NCH) {
                                    if (n % 2 == 0) {
#pragma unroll
                                        for (int k = 0; k < 4; ++k)
                                            w[k] = *reinterpret_cast<const float2 *>(cols + n / 2 * 32 + 8 * k);
                                    }
                                    tmem_ld_16x256b_x4(ta + ((uint32_t)(n & 1) << 20) + b * BN + n / 2 * 32, d[n & 1]);
                                    frag_factors(f[n & 1], r + (n & 1) * 2, w);
                                } else {
                                    release();
                                }
#pragma unroll
                                for (int k = 0; k < 16; k += 2)
                                    fma2(acc[c * 16 + k], acc[c * 16 + k + 1], bits_f(d[c & 1][k]),
                                         bits_f(d[c & 1][k + 1]), f[c & 1][k], f[c & 1][k + 1]);
                            }
                        } else {
                            // One chunk in flight for each warp: the two warps of a scheduler take turns at
                            // reading and adding.
#pragma unroll
                            for (int c = 0; c < C::NCH; ++c) {
                                uint32_t d[C::CH];
                                tmem_ld_32x32b_x16(ta + b * BN + c * C::CH, d);
                                tmem_landed<C::CH>(d);
                                if (c + 1 == C::NCH) release();
                                const float f = C::TWO_BLOCKS && !VECB && c * C::CH >= turn ? rc2[i] : rc[i];
                                promote<C::CH, QVEC>(acc + c * C::CH, d, f, cv + i * BN + c * C::CH);
                            }
                        }
                    }
                }
                if (!ok) break;
                if (!QVEC) {                            // (down here the factors have long arrived)
                    float top = 0.0f;
#pragma unroll
                    for (int i = 0; i < SG; ++i) {
                        top = fmaxf(top, fabsf(rc[i]));
                        if (C::TWO_BLOCKS) top = fmaxf(top, fabsf(rc2[i]));
                    }
                    if (top > FLT_TOP) *again = 1u;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sempty[slot]);
                if (++slot == SLOTS) {
                    slot = 0;
                    sphase ^= 1u;
                }
            }
            if (!ok) break;
            const int p = pb * BP + prow;
            const int q0 = qb * BN + c0;
            if (QVEC) {
                float z[4] = {};                        // 0 times a finite total is 0
#pragma unroll
                for (int j = 0; j < C::ACC; j += 2) fma2(z[j % 4], z[j % 4 + 1], acc[j], acc[j + 1], 0.0f, 0.0f);
                if (!((z[0] + z[1]) + (z[2] + z[3]) == 0.0f)) *again = 1u;
            }
            if (C::SPLITS && split > 1) {
                // the last unit's MMAs have completed: nothing reads or writes the ring any more.
                // Staged along y's contiguous axis, with a pitch that keeps 16-byte accesses free of
                // bank conflicts
                float *st = reinterpret_cast<float *>(smem);
                if (SWAP) {
#pragma unroll
                    for (int j = 0; j < C::ACC; ++j) st[(c0 + j) * (BP + 4) + prow] = acc[j];
                } else if (C::FRAG) {
#pragma unroll
                    for (int j = 0; j < C::ACC; j += 2)
                        *reinterpret_cast<float2 *>(st + (q4 * 32 + (j >> 1 & 1) * 8 + (j >> 4 & 1) * 16 + lane / 4) * (BN + 4) +
                                                    c0 + j / 32 * 32 + j % 16 / 4 * 8 + (lane & 3) * 2) =
                            make_float2(acc[j], acc[j + 1]);
                } else {
#pragma unroll
                    for (int j = 0; j < C::ACC; j += 4)
                        *reinterpret_cast<float4 *>(st + prow * (BN + 4) + c0 + j) =
                            make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
                }
            } else if (SWAP) {
                const float bv = p < g.P ? bias_of(g, p) : 0.0f;
#pragma unroll
                for (int j = 0; j < C::ACC; ++j)
                    if (p < g.P && q0 + j < g.Q) store_one(g, q0 + j, p, acc[j] + bv);
            }
            if (!SWAP && !(C::SPLITS && split > 1)) {
                // Rows leave through shared memory, 64 bytes of each of the warp's 32 rows at a time, so
                // that a store writes 8 rows x 64 bytes (whole sectors) and not 32 x 16.  16-byte piece i
                // of row r sits at piece i ^ (r / 2 % 4): no bank conflicts either way.
                uint8_t *st = sSt + (warp - 4) * ST_BYTES;
                const int64_t r0 = (int64_t)pb * BP + q4 * 32;
                if (g.bias) {
                    // The columns' biases pass through the same place: one load per lane and 32 columns,
                    // not one per column (3641 x 8576 x 491, FP32 output: 98 -> 55 us).
                    float *sb = reinterpret_cast<float *>(st);
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < C::ACC; j += 32)
                        sb[j + lane] = q0 + j + lane < g.Q ? bias_of(g, q0 + j + lane) : 0.0f;
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < C::ACC && C::FRAG; j += 2) {
                        const float2 v = *reinterpret_cast<const float2 *>(sb + j / 32 * 32 + j % 16 / 4 * 8 + (lane & 3) * 2);
                        acc[j] += v.x;
                        acc[j + 1] += v.y;
                    }
#pragma unroll
                    for (int j = 0; j < C::ACC && !C::FRAG; j += 4) {
                        const float4 v = *reinterpret_cast<const float4 *>(sb + j);
                        acc[j] += v.x;
                        acc[j + 1] += v.y;
                        acc[j + 2] += v.z;
                        acc[j + 3] += v.w;
                    }
                }
                if (g.out_f32)
                    store_rows<C::ACC, 16, true, C::FRAG>(g, st, acc, lane, r0, q0);
                else
                    store_rows<C::ACC, 32, false, C::FRAG>(g, st, acc, lane, r0, q0);
            }
        }
        __syncwarp();
        if (C::SPLITS && split > 1) {
            cluster_sync();
            if (ok && t0 < g.num_tiles) {
                int pb, qb;
                tile_coords(t0, g, pb, qb);
                const uint32_t st = smem_addr(smem);
                // pieces of 4 along y's contiguous axis; rank r adds up the r-th part of them
                constexpr int INNER = SWAP ? BP : BN;
                const int pieces = BP * BN / 4;
                const int p1 = pieces * (rank + 1) / split;
                for (int i = pieces * rank / split + (int)threadIdx.x - 128; i < p1; i += 32 * C::EPI_WARPS) {
                    const int e = i * 4;
                    const int o = e / INNER, in = e % INNER;
                    const uint32_t addr = st + (o * (INNER + 4) + in) * 4;
                    float4 part[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (k < split) part[k] = peer_ld4(addr, (uint32_t)k);
                    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (k < split) {
                            v[0] += part[k].x;
                            v[1] += part[k].y;
                            v[2] += part[k].z;
                            v[3] += part[k].w;
                        }
                    const int m = (SWAP ? qb * BN : pb * BP) + o, n = (SWAP ? pb * BP : qb * BN) + in;
                    if (m < (SWAP ? g.Q : g.P)) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (n + k < (SWAP ? g.P : g.Q)) v[k] += bias_of(g, n + k);
                        store4(g, m, n, v, (SWAP ? g.P : g.Q) - n);
                    }
                }
            }
            cluster_sync();
        }
    }

    tc_fence_before();
    if (PAIR) cluster_sync();                   // neither CTA's memory is used by the other any more
    __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        if (PAIR)
            tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
        else
            tmem_dealloc(tmem_base, C::TMEM_COLS);
    }
    if (*again && !*abort_flag) tiles_again<BN, SWAP, PAIR>(g, t0, tstep, rank);
    if (threadIdx.x == 0 && *abort_flag) status_or(g.status, HIF4_FLAG_TIMEOUT);
}

// Clusters of `size` CTAs that fit on the device at once (cached per kernel, size and device).
int resident_clusters(const void *kernel, cudaLaunchConfig_t cfg, int size)
{
    struct Entry {
        const void *kernel;
        int size, dev, n;
    };
    static std::mutex mu;
    static Entry table[256];
    static int used = 0;
    int dev = 0;
    cudaGetDevice(&dev);
    std::lock_guard<std::mutex> lk(mu);
    for (int i = 0; i < used; ++i)
        if (table[i].kernel == kernel && table[i].size == size && table[i].dev == dev) return table[i].n;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)size;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)size);
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        n = 0;
    }
    if (used < 256) table[used++] = Entry{kernel, size, dev, n};
    return n;
}

struct Call {
    const uint8_t *a, *b;
    int64_t M, N, K, lda, ldb;
    const float *sa, *sb;
    int64_t lds_a, lds_b;
    bool a_e5m2, b_e5m2;
};

// tiles: not null to have the choice only (rows and columns of a tile, CTAs that share its K, CTAs).
template <int BN, bool SWAP, bool VECB, bool PAIR>
hif4_status launch(const Call &c, Args g, cudaStream_t stream, int32_t *tiles)
{
    using CF = Cfg<BN, VECB, PAIR, SWAP>;
    const uint8_t *p = SWAP ? c.b : c.a, *q = SWAP ? c.a : c.b;
    g.P = (int)(SWAP ? c.N : c.M);
    g.Q = (int)(SWAP ? c.M : c.N);
    constexpr int TP = PAIR ? 2 * BP : BP;       // rows of a tile
    g.num_p = (g.P + TP - 1) / TP;
    g.num_q = (g.Q + BN - 1) / BN;
    g.num_u = (int)f8::blocks_of(c.K);
    g.K = (int)c.K;
    g.p_codes = p;
    g.q_codes = q;
    g.p_codes_ld = SWAP ? c.ldb : c.lda;
    g.q_codes_ld = SWAP ? c.lda : c.ldb;
    g.p_e5m2 = SWAP ? c.b_e5m2 : c.a_e5m2;
    g.q_e5m2 = SWAP ? c.a_e5m2 : c.b_e5m2;
    if ((int64_t)g.num_p * g.num_q > INT32_MAX / 8) return HIF4_ERR_UNSUPPORTED;
    g.num_tiles = g.num_p * g.num_q;
    g.p_vec = SWAP ? (VECB ? c.sb : nullptr) : c.sa;
    g.p_ld = SWAP ? c.lds_b : c.lds_a;
    g.q_vec = SWAP ? c.sa : (VECB ? c.sb : nullptr);
    g.q_ld = SWAP ? c.lds_a : c.lds_b;
    g.blk = VECB ? nullptr : c.sb;
    g.blk_ld = c.lds_b;
    g.blk_rows = (int)f8::blocks_of(c.N);
    g.idesc = sm100::idesc_f8_f32(TP, BN, SWAP ? c.b_e5m2 : c.a_e5m2, SWAP ? c.a_e5m2 : c.b_e5m2);

    auto k = k_gemm_f8_block<BN, SWAP, VECB, PAIR>;
    if (CF::REG_HIGH > 0) {
        // the promotion warps wait for registers that the launch must have brought along
        static const bool enough = [&] {
            cudaFuncAttributes at;
            return cudaFuncGetAttributes(&at, k) == cudaSuccess &&
                   at.numRegs * CF::THREADS >= 128 * CF::REG_LOW + 32 * CF::EPI_WARPS * CF::REG_HIGH;
        }();
        if (!enough) return HIF4_ERR_UNSUPPORTED;
    }
    const hif4_status st = allow_smem(reinterpret_cast<const void *>(k), CF::SMEM);
    if (st != HIF4_OK) return st;

    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(CF::THREADS);
    cfg.dynamicSmemBytes = CF::SMEM;
    cfg.stream = stream;
    int split = 1;
    if (CF::SPLITS) {
        // K is shared by as many CTAs as can all be resident at once, while each keeps at least 8 units:
        // with fewer, filling the ring and joining the parts costs more than it saves (1 x 5120 x 5120,
        // 40 units: 12.7 us on 1 CTA a tile, 9.4 on 2, 8.6 on 3 or 4, 8.8 on 5 or 6, 13.3 on 8, whose
        // clusters no longer fit beside one another).  The occupancy query counts one CTA to an SM for a kernel
        // that allocates tensor memory, though two run where they fit: clusters stay within one.
        for (int s = 2; s <= 8 && g.num_u >= 8 * s && (int64_t)g.num_tiles * s <= (int64_t)sm_count() * CF::CTAS; ++s)
            if (resident_clusters(reinterpret_cast<const void *>(k), cfg, s) >= g.num_tiles) split = s;
    }
    g.split = split;
    const int cluster = PAIR ? 2 : split;
    int64_t grid = (int64_t)g.num_tiles * cluster;
    const int64_t slots = (int64_t)sm_count() * CF::CTAS / cluster * cluster;
    if (split == 1 && grid > slots) grid = slots;       // persistent
    if (tiles) {
        tiles[0] = TP;
        tiles[1] = BN;
        tiles[2] = split;
        tiles[3] = (int32_t)grid;
        return HIF4_OK;
    }
    CUtensorMap tmP, tmQ;
    if (!make_tensor_map_u8_2d_sw128(&tmP, p, (uint64_t)c.K, (uint64_t)g.P, (uint64_t)(SWAP ? c.ldb : c.lda), KU,
                                     BP) ||
        !make_tensor_map_u8_2d_sw128(&tmQ, q, (uint64_t)c.K, (uint64_t)g.Q, (uint64_t)(SWAP ? c.lda : c.ldb), KU,
                                     PAIR ? BN / 2 : BN))
        return HIF4_ERR_UNSUPPORTED;            // the driver's encoder refused the layout
    cfg.gridDim = dim3((unsigned)grid);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t le = cudaLaunchKernelEx(&cfg, k, tmP, tmQ, g);
    if (le != cudaSuccess) {
        (void)cudaGetLastError();
        return cuda_failed(le);
    }
    return launch_status();
}

template <bool VECB>
hif4_status dispatch(const Call &c, const Args &g, cudaStream_t s, int32_t *tiles = nullptr)
{
    if (c.M <= 16) return launch<16, true, VECB, false>(c, g, s, tiles);
    if (c.M <= 32) return launch<32, true, VECB, false>(c, g, s, tiles);
    // 128 x 128 tiles of one CTA, or 256 x 192 or 256 x 256 tiles of a pair, by estimated time in ns: each
    // wave of tiles takes its units and its stores.  The larger a tile, the less a product costs in operand
    // bytes and hand-offs; the smaller, the better the waves fill the SMs.  One wave of the smallest tiles is always
    // chosen, since no larger tile takes less per unit; where it leaves half the SMs idle, they share K (launch).
    // Measured when the rule was set (us, device time; 128 x 128 / 256 x 192 / 256 x 256; the chosen ones have
    // moved by -7 to +2 % since): 128 x 5120 x 5120 12.9 / 19.5 / 23.4,
    // 512 x 5120 x 13824 68.3 / 50.6 / 57.8, 768 x 5120 x 13824 70.5 / 88.2 / 58.7, 1024 x 5120 x 5120
    // 40.4 / 38.3 / 44.6, 2048 x 13824 x 5120 165 / 147 / 142, 8192 x 5120 x 13824 628 / 575 / 544.
    // A unit takes longer where b has a scale per row: two operations per element instead of one.
    const int64_t units = f8::blocks_of(c.K), sms = sm_count(), pairs = sms / 2;
    const int64_t small = f8::blocks_of(c.M) * f8::blocks_of(c.N), rows2 = (c.M + 255) / 256;
    const int64_t mid = rows2 * ((c.N + 191) / 192), wide = rows2 * ((c.N + 255) / 256);
    const int64_t t_small = (small + sms - 1) / sms * (units * (VECB ? 420 : 290) + 1500);
    const int64_t t_mid = (mid + pairs - 1) / pairs * (units * (VECB ? 580 : 415) + 1900);
    const int64_t t_wide = (wide + pairs - 1) / pairs * (units * (VECB ? 715 : 475) + 2200);
    if (t_small <= t_mid && t_small <= t_wide) return launch<128, false, VECB, false>(c, g, s, tiles);
    if (t_mid < t_wide) return launch<192, false, VECB, true>(c, g, s, tiles);
    return launch<256, false, VECB, true>(c, g, s, tiles);
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

extern "C" hif4_status hif4_debug_gemm_f8_block_tiles(int64_t M, int64_t N, int64_t K, int32_t b_block_rows,
                                                      int32_t *tiles)
{
    if (M < 1 || N < 1 || K < 1 || (b_block_rows != 1 && b_block_rows != 128) || !tiles) return HIF4_ERR_INVALID_ARG;
    if (M > INT32_MAX / 2 || N > INT32_MAX / 2 || K > INT32_MAX / 2) return HIF4_ERR_UNSUPPORTED;
    gemm8b::Call c{};
    c.M = M;
    c.N = N;
    c.K = K;
    return b_block_rows == 1 ? gemm8b::dispatch<true>(c, gemm8b::Args{}, nullptr, tiles)
                             : gemm8b::dispatch<false>(c, gemm8b::Args{}, nullptr, tiles);
}
