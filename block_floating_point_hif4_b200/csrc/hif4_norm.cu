// hif4_norm.cu — layer norm: forward (BF16, FP32 or block-scaled FP8 output)
// and backward (input gradient, and the reduction of the weight's and bias's
// gradients).
//
// A row of C elements belongs to a group of T threads (8 to 32 lanes, or a
// whole block); thread t owns the 8-element granules t, t + T, ... (at most V
// of them), so x (and dy) are read once.  The granules' columns are the same
// for every row a thread meets: gamma and beta, and in the backward pass the
// column sums, stay in registers for the life of a block, and a block takes
// rows b, b + grid, ...
//
// Measured (device time in a loop; a call on cold operands takes 204 us for the
// first): forward 57600 x 5120 BF16, FP32 parameters, with statistics: 195 to
// 212 us by the card's state, 0.92 to 0.85 of the copy bandwidth.  Four granules
// a thread (160 threads a row, three CTAs per SM): with two (320 threads) 232 us,
// since a row's shuffles and reciprocal are paid once per warp; two rows side
// by side on two granules each 262 us; next row prefetched in registers 263 us.
// FP8 output 250 us, 0.55, still less than the norm and the quantizer one after
// the other (345 us): a row is one chain of dependent steps (statistics, maxima,
// quotient, encoding; 560 instructions per warp and row against 425), which the
// 15 warps of an SM do not hide.  Issue slots are not the bound: 56 % busy, the
// plain norm's 54 %.  Backward 336 us, 0.80 (two granules a thread; with four
// its 200 registers leave one CTA per SM: 495 us).
//
// Other widths, 16384 rows BF16, share of the copy bandwidth: forward 0.86 at
// 5120 columns, 0.69 at 5128 (the class of up to 512 threads a row), 0.85 at
// 8192, 0.77 at 12288, 0.81 at 16384; backward 0.72, 0.66, 0.82, 0.37, 0.36.
// Past 8192 columns the backward kernel's rows have 1024 threads of 64 registers,
// 48 of which gamma and the column sums want: it spills 528 bytes (568 for FP32).
//
// A thread fetches its own granules up to three rows ahead with cp.async into
// its own places of shared memory: no barrier, no registers for data in flight,
// and a granule that the row ends in is filled up with zeros by the copy.
//
// Forward statistics, in FP32: each warp takes its sum, then its sum of
// squares about the warp's own mean, and the warps' (n, mean, M2) are merged
// as  mean = sum n_w mean_w / C,  M2 = sum M2_w + n_w (mean_w - mean)^2 :
// nowhere is a square taken about a point far from the row's values, and a
// row of several warps costs one block barrier.
//
// Backward, with xh = (x - mean) rstd and w = dy gamma:
//   dx = rstd (w - mean(w) - xh mean(w xh)),
//   dgamma = sum over rows of dy xh,  dbeta = sum over rows of dy.
// Every block writes its partial column sums to the workspace, and a second
// kernel adds them in a fixed order: the result does not depend on timing.
#include "hif4_f8.cuh"
#include "hif4_pdl.cuh"

namespace hif4 {
namespace {

using namespace f8;

constexpr int kMaxCols = 16384;
constexpr int kMaxRows = 1 << 30;        // row numbers plus a grid's rows stay below 2^31
constexpr int kSmallThreads = 256;       // block size of the sub-warp and one-warp rows
constexpr int kMaxPartials = 592;        // most blocks of the backward kernel (4 per SM of 148)

enum NormOut { OUT_BF16 = 0, OUT_F32 = 1, OUT_E4M3 = 2, OUT_E5M2 = 3 };

struct NormArgs {
    const void *x;
    int64_t ldx;
    const void *gamma, *beta;    // nullable
    uint32_t param_bf16;
    int rows, cols;
    float inv_cols, eps;
    void *y;                     // BF16 / FP32 / FP8 codes
    int64_t ldy;
    float *scale;                // FP8 outputs
    int64_t lds;
    float *mean, *rstd;          // nullable
    uint32_t *status;
};

struct NormBwdArgs {
    const void *dy;
    int64_t lddy;
    const void *x;
    int64_t ldx;
    const float *mean, *rstd;
    const void *gamma;           // nullable
    uint32_t param_bf16;
    int rows, cols;
    float inv_cols;
    void *dx;                    // nullable
    int64_t lddx;
    float *part;                 // [blocks][2][cols rounded up to 8]; null when neither sum is wanted
};

// ---- packed FP32 pairs (one instruction for two elements)
typedef unsigned long long f2;

__device__ __forceinline__ f2 pack2(float lo, float hi)
{
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unpack2(f2 v)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b)
{
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b)
{
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c)
{
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float sum2(f2 v)
{
    const float2 p = unpack2(v);
    return p.x + p.y;
}

template <bool BF16>
__device__ __forceinline__ void widen8(const Raw8<BF16> &r, f2 (&v)[4])
{
    float e[8];
    f8::widen8<BF16>(r, e);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pack2(e[2 * i], e[2 * i + 1]);
}

// The 8 parameters of a granule (naturally aligned; loaded once per block).
__device__ __forceinline__ void load_params(const void *p, uint32_t bf16, int col, int valid, float dflt, f2 (&v)[4])
{
    float e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = dflt;
    if (p && valid >= 8 && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
        if (bf16)
            f8::widen8<true>(load_raw8<true>(p, col, 8), e);
        else
            f8::widen8<false>(load_raw8<false>(p, col, 8), e);
    } else if (p) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < valid)
                e[i] = bf16 ? bits_f((uint32_t)static_cast<const uint16_t *>(p)[col + i] << 16)
                            : static_cast<const float *>(p)[col + i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pack2(e[2 * i], e[2 * i + 1]);
}

// Sum over the first N lanes (the others hold 0), given to all.
template <int N>
__device__ __forceinline__ float warps_sum(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        if (o < N) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return __shfl_sync(0xFFFFFFFFu, v, 0);
}

// N maxima (NaN above all) over groups of W lanes, side by side.
template <int W, int N>
__device__ __forceinline__ void group_maxs(float (&v)[N])
{
#pragma unroll
    for (int o = W / 2; o; o >>= 1)
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = max_nan(v[k], __shfl_xor_sync(0xFFFFFFFFu, v[k], o));
}

// ---- the rows in flight: `depth` stages of [piece][thread] 16-byte pieces, each
// written and read by its thread alone.  Four stages (three rows of 10 KB ahead in
// each of three CTAs per SM for 5120 BF16), fewer where wide rows leave no room.
template <bool BF16>
constexpr int pieces() { return BF16 ? 1 : 2; }

template <bool BF16>
constexpr int depth(int wide, int v, int arrays)
{
    const int stage = arrays * v * pieces<BF16>() * (wide ? wide : kSmallThreads) * 16;
    // shared memory of a CTA: one, two or three of them to an SM
    const int room = (wide > 320 || (!wide && v > 2) ? 200 : wide == 160 ? 68 : 104) * 1024;
    return stage * 4 <= room ? 4 : stage * 2 <= room ? 2 : 1;
}

// L1: through the first-level cache, for the FP32 pieces, two of which share a
// 32-byte sector that each would otherwise fetch from L2.
template <bool L1>
__device__ __forceinline__ void async16(uint4 *dst, const void *src, int bytes)
{
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    if (L1)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(bytes) : "memory");
    else
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(bytes) : "memory");
}

// Starts the copy of a granule; elements from `valid` on become 0 (nothing is read for valid = 0).
template <bool BF16>
__device__ __forceinline__ void fetch8(uint4 *dst, int threads, const uint8_t *src, int valid)
{
    if (BF16) {
        async16<false>(dst, src, valid * 2);
    } else {
        async16<true>(dst, src, min(valid, 4) * 4);
        async16<true>(dst + threads, valid > 4 ? src + 16 : src, max(valid - 4, 0) * 4);
    }
}

template <bool BF16>
__device__ __forceinline__ Raw8<BF16> fetched8(const uint4 *src, int threads)
{
    Raw8<BF16> r;
    r.w[0] = src[0];
    if (!BF16) r.w[BF16 ? 0 : 1] = src[threads];
    return r;
}

__device__ __forceinline__ void fetch_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void fetch_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int W>
__device__ __forceinline__ float group_sum(float v)
{
#pragma unroll
    for (int o = W / 2; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// XB: x is BF16.  V: granules per thread.  LANES: lanes of a row's group in a
// warp (8, 16 or 32); WIDE: 0, or the largest block the row may belong to.
template <bool XB, int OUT, int V, int LANES, int WIDE>
__global__ void __launch_bounds__(WIDE ? WIDE : kSmallThreads, WIDE == 160 ? 3 : 1) k_norm_fwd(NormArgs a)
{
    constexpr int kDepth = depth<XB>(WIDE, V, 1), P = pieces<XB>(), ESZ = XB ? 2 : 4;
    constexpr int OSZ = OUT == OUT_BF16 ? 2 : OUT == OUT_F32 ? 4 : 1;
    constexpr int NW = WIDE ? WIDE / 32 : 1;
    extern __shared__ uint4 smem_rows[];
    __shared__ float4 sStat[WIDE ? 2 : 1][NW];                  // (n, mean, M2, sum) of each warp's part
    if (WIDE && threadIdx.x < 2 * NW) (&sStat[0][0])[threadIdx.x] = make_float4(0, 0, 0, 0);
    pdl_enter();
    const int T = WIDE ? blockDim.x : LANES;
    const int t = WIDE ? threadIdx.x : threadIdx.x % LANES;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rpb = WIDE ? 1 : kSmallThreads / LANES;           // rows in flight per block
    const int nt = blockDim.x;
    const bool tail = a.cols & 7;

    const int step = gridDim.x * rpb;
    // the groups of a warp leave the loop together (shuffles): wrow is the warp's first row
    int row = blockIdx.x * rpb + (WIDE ? 0 : threadIdx.x / LANES);
    int wrow = WIDE ? row : blockIdx.x * rpb + warp * (32 / LANES);
    int valid[V];
#pragma unroll
    for (int v = 0; v < V; ++v) valid[v] = max(0, min(8, a.cols - (t + v * T) * 8));

    uint4 *ring = smem_rows + threadIdx.x;                       // [kDepth][V][P][nt]
    const uint8_t *src = static_cast<const uint8_t *>(a.x) + ((int64_t)row * a.ldx + t * 8) * ESZ;
    const int64_t src_step = (int64_t)step * a.ldx * ESZ;
    uint8_t *dst = static_cast<uint8_t *>(a.y) + ((int64_t)row * a.ldy + t * 8) * OSZ;
    const int64_t dst_step = (int64_t)step * a.ldy * OSZ;
    int frow = row;                                              // the next row to fetch
    // granules past the row read as 0 for good; those of rows past the last one are never used
#pragma unroll
    for (int i = 0; i < kDepth * V; ++i)
        if (valid[i % V] == 0)
#pragma unroll
            for (int p = 0; p < P; ++p) ring[(i * P + p) * nt] = make_uint4(0, 0, 0, 0);
    auto fetch = [&](int stage) {
        if (frow < a.rows) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (valid[v] > 0)
                    fetch8<XB>(ring + (stage * V + v) * P * nt, nt, src + v * T * 8 * ESZ, valid[v]);
        }
        fetch_commit();
        frow += step;
        src += src_step;
    };
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) fetch(i);

    f2 gm[V][4], bt[V][4];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        load_params(a.gamma, a.param_bf16, (t + v * T) * 8, valid[v], 1.0f, gm[v]);
        load_params(a.beta, a.param_bf16, (t + v * T) * 8, valid[v], 0.0f, bt[v]);
    }
    float n_w = 0.0f;                                            // elements of a row in this warp's (group's) part
#pragma unroll
    for (int v = 0; v < V; ++v) n_w += (float)valid[v];
    n_w = group_sum<LANES>(n_w);
    const float inv_n_w = n_w > 0.0f ? 1.0f / n_w : 0.0f;

    uint32_t bad = 0;
    int buf = 0, stage = 0;
    if (WIDE) __syncthreads();                                   // sStat is cleared
    for (; wrow < a.rows;) {
        const bool live = row < a.rows;
        fetch((stage + kDepth - 1) % kDepth);
        fetch_wait<kDepth - 1>();
        f2 x[V][4];
#pragma unroll
        for (int v = 0; v < V; ++v) widen8<XB>(fetched8<XB>(ring + (stage * V + v) * P * nt, nt), x[v]);
        stage = (stage + 1) % kDepth;

        f2 s = 0;                                                // elements past the row read as 0
#pragma unroll
        for (int v = 0; v < V; ++v) s = add2(s, add2(add2(x[v][0], x[v][1]), add2(x[v][2], x[v][3])));
        const float sum_w = group_sum<LANES>(sum2(s));
        float mean = sum_w * inv_n_w, m2 = 0.0f;
        {
            const f2 neg = pack2(-mean, -mean);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                f2 d[4], q = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) d[i] = add2(x[v][i], neg);
                if (tail) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 e = unpack2(d[i]);
                        d[i] = pack2(2 * i < valid[v] ? e.x : 0.0f, 2 * i + 1 < valid[v] ? e.y : 0.0f);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) q = fma2(d[i], d[i], q);
                m2 += valid[v] > 0 ? sum2(q) : 0.0f;
            }
        }
        m2 = group_sum<LANES>(m2);
        if (WIDE) {
            if (lane == 0) sStat[buf][warp] = make_float4(n_w, mean, m2, sum_w);
            __syncthreads();
            // lane w holds warp w's part; warps that do not exist count 0 elements
            const float4 p = lane < NW ? sStat[buf][lane] : make_float4(0, 0, 0, 0);
            mean = warps_sum<NW>(p.w) * a.inv_cols;
            const float d = p.y - mean;
            m2 = warps_sum<NW>(fmaf(p.x * d, d, p.z));
            buf ^= 1;
        }
        const float rstd = __frsqrt_rn(fmaf(m2, a.inv_cols, a.eps));
        if (t == 0 && live) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
        const f2 neg = pack2(-mean, -mean), r2 = pack2(rstd, rstd);
        float y[V][8];
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 e = unpack2(fma2(mul2(add2(x[v][i], neg), r2), gm[v][i], bt[v][i]));
                y[v][2 * i] = e.x;
                y[v][2 * i + 1] = e.y;
            }
        if (OUT == OUT_BF16 || OUT == OUT_F32) {
            if (live) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (valid[v] > 0) store8<OUT == OUT_BF16>(dst, v * T * 8, y[v], valid[v]);
            }
        } else {
            constexpr int W = LANES < 16 ? LANES : 16;           // lanes of a 128-block
            float m[V];
            bool ok = true;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int n = live ? valid[v] : 0;
                if (n < 8) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (i >= n) y[v][i] = 0.0f;
                }
                m[v] = amax8_nan(y[v]);
            }
            group_maxs<W, V>(m);
#pragma unroll
            for (int v = 0; v < V; ++v) ok = ok && m[v] <= 3.402823466e38f;      // false for NaN too
            if (!__all_sync(0xFFFFFFFFu, ok)) {                  // rare: map what is not finite, and again
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    sanitize_all(y[v], bad);
                    m[v] = amax8_nan(y[v]);
                }
                group_maxs<W, V>(m);
            }
            // lane 2 v of a block's lanes forms the factor of granule v's block, lane 2 v + 1 its scale
            const int l = t % W;
            float mine = m[0];
#pragma unroll
            for (int v = 1; v < V; ++v) mine = (l >> 1) == v ? m[v] : mine;
            const float s8 = scale_or_factor(f_bits(mine), fmt_max(OUT == OUT_E5M2 ? HIF4_E5M2 : HIF4_E4M3), l & 1);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float f = __shfl_sync(0xFFFFFFFFu, s8, 2 * v, W);
                const uint32_t lo = encode4<OUT == OUT_E5M2>(y[v][0], y[v][1], y[v][2], y[v][3], f);
                const uint32_t hi = encode4<OUT == OUT_E5M2>(y[v][4], y[v][5], y[v][6], y[v][7], f);
                if (live && valid[v] > 0) store_codes8(dst + v * T * 8, lo, hi, valid[v]);
            }
            const int c = (t - l + (l >> 1) * T) * 8;            // first column of the lane's block
            if ((l & 1) && (l >> 1) < V && c < a.cols && live) a.scale[(int64_t)(c / BLK) * a.lds + row] = s8;
        }
        row += step;
        wrow += step;
        dst += dst_step;
    }
    if (bad) status_or(a.status, HIF4_FLAG_NONFINITE);
}

// TAIL: the row may end inside a granule.
template <bool XB, int V, int LANES, int WIDE, bool TAIL = true>
__global__ void __launch_bounds__(WIDE ? WIDE : kSmallThreads, WIDE == 320 && XB ? 2 : 1) k_norm_bwd(NormBwdArgs a)
{
    constexpr int kDepth = depth<XB>(WIDE, V, 2), P = pieces<XB>(), ESZ = XB ? 2 : 4;
    extern __shared__ uint4 smem_rows[];
    constexpr int NW = WIDE ? WIDE / 32 : 1;
    __shared__ float2 sSum[WIDE ? 2 : 1][NW];
    pdl_enter();
    const int T = WIDE ? blockDim.x : LANES;
    const int t = WIDE ? threadIdx.x : threadIdx.x % LANES;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rpb = WIDE ? 1 : kSmallThreads / LANES;
    const int nw = blockDim.x >> 5;
    const int nt = blockDim.x;

    const int step = gridDim.x * rpb;
    int row = blockIdx.x * rpb + (WIDE ? 0 : threadIdx.x / LANES);
    int wrow = WIDE ? row : blockIdx.x * rpb + warp * (32 / LANES);
    int valid[V];
#pragma unroll
    for (int v = 0; v < V; ++v) valid[v] = max(0, min(8, a.cols - (t + v * T) * 8));

    uint4 *ring = smem_rows + threadIdx.x;                       // [kDepth][x, dy][V][P][nt]
    const uint8_t *xs = static_cast<const uint8_t *>(a.x) + ((int64_t)row * a.ldx + t * 8) * ESZ;
    const uint8_t *ds = static_cast<const uint8_t *>(a.dy) + ((int64_t)row * a.lddy + t * 8) * ESZ;
    const int64_t x_step = (int64_t)step * a.ldx * ESZ, d_step = (int64_t)step * a.lddy * ESZ;
    uint8_t *dst = static_cast<uint8_t *>(a.dx) + ((int64_t)row * a.lddx + t * 8) * ESZ;
    const int64_t dst_step = (int64_t)step * a.lddx * ESZ;
    int frow = row;
    auto fetch = [&](int stage) {
        const bool in = frow < a.rows;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int n = in ? valid[v] : 0;
            const uint8_t *from = xs + v * T * 8 * ESZ;
            int nx = n;
            if (!TAIL && valid[v] == 0) {
                // x past the row is the row's first granule: w is 0 there, and xh must be finite if the row's is
                from = xs - t * 8 * ESZ;
                nx = in ? 8 : 0;
            }
            fetch8<XB>(ring + (stage * 2 * V + v) * P * nt, nt, nx > 0 ? from : static_cast<const uint8_t *>(a.x), nx);
            fetch8<XB>(ring + (stage * 2 * V + V + v) * P * nt, nt,
                       n > 0 ? ds + v * T * 8 * ESZ : static_cast<const uint8_t *>(a.dy), n);
        }
        fetch_commit();
        if (in) {
            xs += x_step;
            ds += d_step;
        }
        frow += step;
    };
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) fetch(i);

    f2 gm[V][4], dg[V][4], db[V][4];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        load_params(a.gamma, a.param_bf16, (t + v * T) * 8, valid[v], 1.0f, gm[v]);
#pragma unroll
        for (int i = 0; i < 4; ++i) dg[v][i] = db[v][i] = 0;
    }
    int buf = 0, stage = 0;
    // Statistics a row ahead.  0 past the last row, where dy reads as 0 too: nothing is added there.
    float cmean = row < a.rows ? a.mean[row] : 0.0f, crstd = row < a.rows ? a.rstd[row] : 0.0f;
    for (; wrow < a.rows;) {
        const bool live = row < a.rows;
        const float mean = cmean, rstd = crstd;
        const int nrow = row + step;
        cmean = nrow < a.rows ? a.mean[nrow] : 0.0f;
        crstd = nrow < a.rows ? a.rstd[nrow] : 0.0f;
        fetch((stage + kDepth - 1) % kDepth);
        fetch_wait<kDepth - 1>();
        f2 xh[V][4], w[V][4], s1 = 0, s2 = 0;
        const f2 neg = pack2(-mean, -mean), r2 = pack2(rstd, rstd);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            f2 d[4];
            widen8<XB>(fetched8<XB>(ring + (stage * 2 * V + v) * P * nt, nt), xh[v]);
            widen8<XB>(fetched8<XB>(ring + (stage * 2 * V + V + v) * P * nt, nt), d);
#pragma unroll
            for (int i = 0; i < 4; ++i) xh[v][i] = mul2(add2(xh[v][i], neg), r2);
            if (TAIL && valid[v] < 8) {
                // past the row x is 0 here, and xh may be infinite: 0 times it would be NaN
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 e = unpack2(xh[v][i]);
                    xh[v][i] = pack2(2 * i < valid[v] ? e.x : 0.0f, 2 * i + 1 < valid[v] ? e.y : 0.0f);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                dg[v][i] = fma2(d[i], xh[v][i], dg[v][i]);
                db[v][i] = add2(db[v][i], d[i]);
                w[v][i] = mul2(d[i], gm[v][i]);
                s1 = add2(s1, w[v][i]);
                s2 = fma2(w[v][i], xh[v][i], s2);
            }
        }
        stage = (stage + 1) % kDepth;
        float t1 = group_sum<LANES>(sum2(s1)), t2 = group_sum<LANES>(sum2(s2));
        if (WIDE) {
            if (lane == 0) sSum[buf][warp] = make_float2(t1, t2);
            __syncthreads();
            const float2 p = lane < nw ? sSum[buf][lane] : make_float2(0.0f, 0.0f);
            t1 = warps_sum<NW>(p.x);
            t2 = warps_sum<NW>(p.y);
            buf ^= 1;
        }
        if (a.dx) {
            const float c1 = t1 * a.inv_cols, c2 = t2 * a.inv_cols;
            const f2 n1 = pack2(-c1, -c1), n2 = pack2(-c2, -c2);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float o[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 e = unpack2(mul2(fma2(xh[v][i], n2, add2(w[v][i], n1)), r2));
                    o[2 * i] = e.x;
                    o[2 * i + 1] = e.y;
                }
                if (live && valid[v] > 0) store8<XB>(dst, v * T * 8, o, valid[v]);
            }
        }
        row += step;
        wrow += step;
        dst += dst_step;
    }
    if (!a.part) return;
    const int pitch = (a.cols + 7) & ~7;
    float *pg = a.part + (int64_t)blockIdx.x * 2 * pitch, *pb = pg + pitch;
    if (WIDE) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (valid[v] > 0) {                                  // whole granules: the pitch has room
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 g0 = unpack2(dg[v][2 * i]), g1 = unpack2(dg[v][2 * i + 1]);
                    const float2 b0 = unpack2(db[v][2 * i]), b1 = unpack2(db[v][2 * i + 1]);
                    reinterpret_cast<float4 *>(pg + (t + v * T) * 8)[i] = make_float4(g0.x, g0.y, g1.x, g1.y);
                    reinterpret_cast<float4 *>(pb + (t + v * T) * 8)[i] = make_float4(b0.x, b0.y, b1.x, b1.y);
                }
            }
    } else {
        // The block's row groups, added in order: group g's sums lie at g * W in the memory of the rows,
        // of which no copy is in flight any more.
        constexpr int W = LANES * V * 8;
        float *sCol = reinterpret_cast<float *>(smem_rows);
        const int g = threadIdx.x / LANES;
        asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
            __syncthreads();
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<float2 *>(sCol + g * W + (t + v * LANES) * 8 + 2 * i) =
                        unpack2(pass ? db[v][i] : dg[v][i]);
            __syncthreads();
            for (int c = threadIdx.x; c < a.cols; c += kSmallThreads) {
                float s = 0.0f;
                for (int k = 0; k < kSmallThreads / LANES; ++k) s += sCol[k * W + c];
                (pass ? pb : pg)[c] = s;
            }
        }
    }
}

// Column sums over the blocks' partials: 32 columns per block, the partials
// split over 32 rows of threads and joined in a fixed order.
__global__ void __launch_bounds__(1024) k_norm_bwd_join(const float *part, int parts, int cols, float *dgamma,
                                                        float *dbeta)
{
    __shared__ float s[32][33];
    pdl_enter();
    const int pitch = (cols + 7) & ~7;
    const int c = blockIdx.x * 32 + threadIdx.x;                 // over 2 x pitch: dgamma, then dbeta
    float v = 0.0f;
    if (c < 2 * pitch) {
#pragma unroll 4
        for (int p = threadIdx.y; p < parts; p += 32) v += part[(int64_t)p * 2 * pitch + c];
    }
    s[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    v = s[threadIdx.x][threadIdx.y];                             // lane = part, warp = column
    v = group_sum<32>(v);
    const int co = blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0) {
        if (co < cols) {
            if (dgamma) dgamma[co] = v;
        } else if (dbeta && co >= pitch && co - pitch < cols) {
            dbeta[co - pitch] = v;
        }
    }
}

// Threads of a row's group and granules per thread: 8, 16 or 32 lanes of a warp
// up to 1024 columns, a block beyond.
struct Shape {
    int lanes, v, threads, wide;
};

Shape shape_of(int64_t cols, int wide_v)
{
    const int g = (int)((cols + 7) / 8);
    if (g <= 8) return Shape{8, 1, kSmallThreads, 0};
    if (g <= 16) return Shape{16, 1, kSmallThreads, 0};
    if (g <= 32) return Shape{32, 1, kSmallThreads, 0};
    if (g <= 64) return Shape{32, 2, kSmallThreads, 0};
    if (g <= 128) return Shape{32, 4, kSmallThreads, 0};
    const int threads = (g + 32 * wide_v - 1) / (32 * wide_v) * 32;
    return Shape{32, wide_v, threads, threads <= 640 / wide_v ? 640 / wide_v : threads <= 512 ? 512 : 1024};
}

// Blocks of a persistent launch over `rows`, and its dynamic shared memory.
template <typename A>
hif4_status grid_of(void (*k)(A), const Shape &sh, int rows, size_t smem, int64_t &grid)
{
    const hif4_status st = allow_smem(reinterpret_cast<const void *>(k), smem);
    if (st != HIF4_OK) return st;
    const int rpb = sh.wide ? 1 : kSmallThreads / sh.lanes;
    grid = ((int64_t)rows + rpb - 1) / rpb;
    const int64_t most = (int64_t)sm_count() * blocks_per_sm(reinterpret_cast<const void *>(k), sh.threads, smem);
    if (grid > most) grid = most;
    return HIF4_OK;
}

template <bool XB, int OUT>
hif4_status launch_fwd(const NormArgs &a, cudaStream_t s)
{
    const Shape sh = shape_of(a.cols, 4);
    void (*k)(NormArgs) = sh.wide == 160 ? k_norm_fwd<XB, OUT, 4, 32, 160>
                          : sh.wide ? k_norm_fwd<XB, OUT, 4, 32, 512>
                          : sh.lanes == 8 ? k_norm_fwd<XB, OUT, 1, 8, 0>
                          : sh.lanes == 16 ? k_norm_fwd<XB, OUT, 1, 16, 0>
                          : sh.v == 1 ? k_norm_fwd<XB, OUT, 1, 32, 0>
                          : sh.v == 2 ? k_norm_fwd<XB, OUT, 2, 32, 0> : k_norm_fwd<XB, OUT, 4, 32, 0>;
    const size_t smem = (size_t)depth<XB>(sh.wide, sh.v, 1) * sh.v * pieces<XB>() * sh.threads * 16;
    int64_t grid;
    const hif4_status st = grid_of(k, sh, a.rows, smem, grid);
    if (st != HIF4_OK) return st;
    return launch_pdl(k, dim3((unsigned)grid), dim3((unsigned)sh.threads), smem, s, a);
}

template <bool XB>
hif4_status launch_bwd(const NormBwdArgs &a, float *dgamma, float *dbeta, cudaStream_t s)
{
    const Shape sh = shape_of(a.cols, 2);
    // Rows of whole granules have a variant without the test for what lies past them where registers are
    // short: 57600 x 5120 BF16 336 us without, 382 with it; no difference in the other shapes.
    const bool whole = a.cols % 8 == 0;
    void (*k)(NormBwdArgs) = sh.wide == 320 && whole ? k_norm_bwd<XB, 2, 32, 320, false>
                             : sh.wide == 320 ? k_norm_bwd<XB, 2, 32, 320>
                             : sh.wide == 512 ? k_norm_bwd<XB, 2, 32, 512>
                             : sh.wide ? k_norm_bwd<XB, 2, 32, 1024>
                             : sh.lanes == 8 ? k_norm_bwd<XB, 1, 8, 0>
                             : sh.lanes == 16 ? k_norm_bwd<XB, 1, 16, 0>
                             : sh.v == 1 ? k_norm_bwd<XB, 1, 32, 0>
                             : sh.v == 2 ? k_norm_bwd<XB, 2, 32, 0> : k_norm_bwd<XB, 4, 32, 0>;
    const size_t smem = (size_t)depth<XB>(sh.wide, sh.v, 2) * 2 * sh.v * pieces<XB>() * sh.threads * 16;
    int64_t grid;
    hif4_status st = grid_of(k, sh, a.rows, smem, grid);
    if (st != HIF4_OK) return st;
    if (grid > kMaxPartials) grid = kMaxPartials;
    st = launch_pdl(k, dim3((unsigned)grid), dim3((unsigned)sh.threads), smem, s, a);
    if (st != HIF4_OK || !a.part) return st;
    return launch_pdl(k_norm_bwd_join, dim3((unsigned)((2 * ((a.cols + 7) & ~7) + 31) / 32)), dim3(32, 32), 0, s, a.part,
                      (int)grid, a.cols, dgamma, dbeta);
}

bool valid_dtype(hif4_dtype d) { return d == HIF4_F32 || d == HIF4_BF16; }
int64_t elem(hif4_dtype d) { return d == HIF4_BF16 ? 2 : 4; }

// Checks shared by the two forward calls; fills a.
hif4_status fwd_args(NormArgs &a, const void *x, hif4_dtype dtype, int64_t rows, int64_t cols, int64_t ldx,
                     const void *gamma, const void *beta, hif4_dtype param, float eps, float *mean, float *rstd)
{
    if (!x || !(eps >= 0.0f) || eps > 3.402823466e38f) return HIF4_ERR_INVALID_ARG;
    if (ldx < cols) return HIF4_ERR_SHAPE;
    if (!aligned16(x) || (ldx * elem(dtype)) % 16) return HIF4_ERR_ALIGNMENT;
    if ((gamma && !aligned_to(gamma, elem(param))) || (beta && !aligned_to(beta, elem(param))) ||
        !aligned_to(mean, 4) || !aligned_to(rstd, 4))
        return HIF4_ERR_ALIGNMENT;
    if (cols > kMaxCols || rows > kMaxRows) return HIF4_ERR_UNSUPPORTED;
    a.x = x;
    a.ldx = ldx;
    a.gamma = gamma;
    a.beta = beta;
    a.param_bf16 = param == HIF4_BF16;
    a.rows = (int)rows;
    a.cols = (int)cols;
    a.inv_cols = (float)(1.0 / (double)cols);
    a.eps = eps;
    a.mean = mean;
    a.rstd = rstd;
    return HIF4_OK;
}

} // namespace
} // namespace hif4

using namespace hif4;

extern "C" hif4_status hif4_layer_norm(const void *x, hif4_dtype dtype, int64_t rows, int64_t cols, int64_t ldx,
                                       const void *gamma, const void *beta, hif4_dtype param_dtype, float eps,
                                       void *y, hif4_dtype out_dtype, int64_t ldy, float *mean, float *rstd,
                                       hif4_stream_t stream)
{
    if (rows < 0 || cols < 0 || !valid_dtype(dtype) || !valid_dtype(param_dtype) || !valid_dtype(out_dtype))
        return HIF4_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return HIF4_OK;
    if (!y) return HIF4_ERR_INVALID_ARG;
    NormArgs a{};
    const hif4_status st = fwd_args(a, x, dtype, rows, cols, ldx, gamma, beta, param_dtype, eps, mean, rstd);
    if (st != HIF4_OK) return st;
    if (ldy < cols) return HIF4_ERR_SHAPE;
    if (!aligned16(y) || (ldy * elem(out_dtype)) % 16) return HIF4_ERR_ALIGNMENT;
    a.y = y;
    a.ldy = ldy;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == HIF4_BF16)
        return out_dtype == HIF4_BF16 ? launch_fwd<true, OUT_BF16>(a, s) : launch_fwd<true, OUT_F32>(a, s);
    return out_dtype == HIF4_BF16 ? launch_fwd<false, OUT_BF16>(a, s) : launch_fwd<false, OUT_F32>(a, s);
}

extern "C" hif4_status hif4_layer_norm_f8(const void *x, hif4_dtype dtype, int64_t rows, int64_t cols, int64_t ldx,
                                          const void *gamma, const void *beta, hif4_dtype param_dtype, float eps,
                                          hif4_f8_format fmt, uint8_t *q, int64_t ldq, float *scale, int64_t lds,
                                          float *mean, float *rstd, uint32_t *status, hif4_stream_t stream)
{
    if (rows < 0 || cols < 0 || !valid_dtype(dtype) || !valid_dtype(param_dtype) || !f8::valid_fmt(fmt))
        return HIF4_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return HIF4_OK;
    if (!q || !scale) return HIF4_ERR_INVALID_ARG;
    NormArgs a{};
    const hif4_status st = fwd_args(a, x, dtype, rows, cols, ldx, gamma, beta, param_dtype, eps, mean, rstd);
    if (st != HIF4_OK) return st;
    if (ldq < cols || lds < rows) return HIF4_ERR_SHAPE;
    if (!aligned16(q) || ldq % 16 || !aligned_to(scale, 4)) return HIF4_ERR_ALIGNMENT;
    a.y = q;
    a.ldy = ldq;
    a.scale = scale;
    a.lds = lds;
    a.status = status;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (fmt == HIF4_E5M2)
        return dtype == HIF4_BF16 ? launch_fwd<true, OUT_E5M2>(a, s) : launch_fwd<false, OUT_E5M2>(a, s);
    return dtype == HIF4_BF16 ? launch_fwd<true, OUT_E4M3>(a, s) : launch_fwd<false, OUT_E4M3>(a, s);
}

extern "C" size_t hif4_layer_norm_backward_workspace(int64_t rows, int64_t cols)
{
    if (rows <= 0 || cols <= 0 || cols > kMaxCols) return 0;
    const int64_t n = rows < kMaxPartials ? rows : kMaxPartials;
    return (size_t)n * 2 * (size_t)((cols + 7) & ~(int64_t)7) * sizeof(float);
}

extern "C" hif4_status hif4_layer_norm_backward(const void *dy, int64_t lddy, const void *x, hif4_dtype dtype,
                                                int64_t rows, int64_t cols, int64_t ldx, const float *mean,
                                                const float *rstd, const void *gamma, hif4_dtype param_dtype,
                                                void *dx, int64_t lddx, float *dgamma, float *dbeta,
                                                void *workspace, size_t ws_bytes, hif4_stream_t stream)
{
    if (rows < 0 || cols < 0 || !valid_dtype(dtype) || !valid_dtype(param_dtype)) return HIF4_ERR_INVALID_ARG;
    if (cols == 0) return HIF4_OK;
    if (cols > kMaxCols || rows > kMaxRows) return HIF4_ERR_UNSUPPORTED;
    if (!aligned_to(dgamma, 4) || !aligned_to(dbeta, 4)) return HIF4_ERR_ALIGNMENT;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (rows == 0) {                                             // sums over no rows
        for (float *p : {dgamma, dbeta})
            if (p) {
                const cudaError_t e = cudaMemsetAsync(p, 0, (size_t)cols * sizeof(float), s);
                if (e != cudaSuccess) return cuda_failed(e);
            }
        return HIF4_OK;
    }
    if (!dy || !x || !mean || !rstd || (!dx && !dgamma && !dbeta)) return HIF4_ERR_INVALID_ARG;
    if (ldx < cols || lddy < cols || (dx && lddx < cols)) return HIF4_ERR_SHAPE;
    const int64_t e = elem(dtype);
    if (!aligned16(x) || !aligned16(dy) || !aligned16(dx) || (ldx * e) % 16 || (lddy * e) % 16 ||
        (dx && (lddx * e) % 16) || !aligned_to(mean, 4) || !aligned_to(rstd, 4) ||
        (gamma && !aligned_to(gamma, elem(param_dtype))))
        return HIF4_ERR_ALIGNMENT;
    const bool sums = dgamma || dbeta;
    if (sums) {
        if (!workspace || ws_bytes < hif4_layer_norm_backward_workspace(rows, cols)) return HIF4_ERR_WORKSPACE;
        if (!aligned_to(workspace, 256)) return HIF4_ERR_ALIGNMENT;
    }
    NormBwdArgs a{};
    a.dy = dy;
    a.lddy = lddy;
    a.x = x;
    a.ldx = ldx;
    a.mean = mean;
    a.rstd = rstd;
    a.gamma = gamma;
    a.param_bf16 = param_dtype == HIF4_BF16;
    a.rows = (int)rows;
    a.cols = (int)cols;
    a.inv_cols = (float)(1.0 / (double)cols);
    a.dx = dx;
    a.lddx = lddx;
    a.part = sums ? static_cast<float *>(workspace) : nullptr;
    return dtype == HIF4_BF16 ? launch_bwd<true>(a, dgamma, dbeta, s) : launch_bwd<false>(a, dgamma, dbeta, s);
}
