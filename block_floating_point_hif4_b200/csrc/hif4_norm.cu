// hif4_norm.cu — layer norm: forward (BF16, FP32 or block-scaled FP8 output)
// and backward (input gradient, and the reduction of the weight's and bias's
// gradients).
//
// A row of C elements belongs to a group of T threads (8 or 32 lanes, or a
// whole block); thread t owns the 8-element granules t, t + T, ... (at most V
// of them) and keeps them in registers, so x (and dy) are read once.  The
// granules' columns are the same for every row a thread meets: gamma and beta,
// and in the backward pass the column sums, stay in registers for the life of
// a block, and a block takes rows b, b + grid, ...
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
constexpr int kSmallThreads = 256;       // block size of the sub-warp and one-warp rows
constexpr int kMaxPartials = 592;        // most blocks of the backward kernel (4 per SM of 148)

enum NormOut { OUT_BF16 = 0, OUT_F32 = 1, OUT_F8 = 2 };

struct NormArgs {
    const void *x;
    int64_t ldx;
    const void *gamma, *beta;    // nullable
    uint32_t param_bf16;
    int rows, cols;
    float inv_cols, eps;
    void *y;                     // BF16 / FP32 / FP8 codes
    int64_t ldy;
    float *scale;                // OUT_F8
    int64_t lds;
    float fmax;
    uint32_t e5m2;
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
    float *part;                 // [blocks][2][cols]; null when neither sum is wanted
};

// The 8 parameters of a granule (naturally aligned; loaded once per block).
__device__ __forceinline__ void load_params(const void *p, uint32_t bf16, int col, int valid, float dflt,
                                            float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = dflt;
        if (p && i < valid)
            v[i] = bf16 ? bits_f((uint32_t)static_cast<const uint16_t *>(p)[col + i] << 16)
                        : static_cast<const float *>(p)[col + i];
    }
}

template <int W>
__device__ __forceinline__ float group_sum(float v)
{
#pragma unroll
    for (int o = W / 2; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// XB: x is BF16.  V: granules per thread.  LANES: lanes of a row's group in a
// warp (8 or 32); WIDE: 0, or the largest block the row may belong to.
template <bool XB, int OUT, int V, int LANES, int WIDE>
__global__ void __launch_bounds__(WIDE ? WIDE : kSmallThreads) k_norm_fwd(NormArgs a)
{
    __shared__ float2 sStat[WIDE ? 2 : 1][32];
    pdl_enter();
    const int T = WIDE ? blockDim.x : LANES;
    const int t = WIDE ? threadIdx.x : threadIdx.x % LANES;
    const int warp = threadIdx.x >> 5;
    const int rpb = WIDE ? 1 : kSmallThreads / LANES;           // rows in flight per block
    const int nw = blockDim.x >> 5;

    int valid[V];
    float gm[V][8], bt[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int col = (t + v * T) * 8;
        valid[v] = max(0, min(8, a.cols - col));
        load_params(a.gamma, a.param_bf16, col, valid[v], 1.0f, gm[v]);
        load_params(a.beta, a.param_bf16, col, valid[v], 0.0f, bt[v]);
    }
    // elements of this warp's (or group's) part of a row
    float n_w = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) n_w += (float)valid[v];
    n_w = group_sum<LANES>(n_w);
    const float inv_n_w = n_w > 0.0f ? 1.0f / n_w : 0.0f;

    uint32_t bad = 0;
    int buf = 0;
    const int64_t step = (int64_t)gridDim.x * rpb;
    // the groups of a warp leave the loop together (shuffles): wrow is the warp's first row
    int64_t row = (int64_t)blockIdx.x * rpb + (WIDE ? 0 : threadIdx.x / LANES);
    int64_t wrow = WIDE ? row : (int64_t)blockIdx.x * rpb + warp * (32 / LANES);
    Raw8<XB> cur[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
        cur[v] = load_raw8<XB>(a.x, row * a.ldx + (t + v * T) * 8, row < a.rows ? valid[v] : 0);
    for (; wrow < a.rows; wrow += step, row += step) {
        const bool live = row < a.rows;
        float x[V][8];
#pragma unroll
        for (int v = 0; v < V; ++v) widen8<XB>(cur[v], x[v]);
        const int64_t nrow = row + step;
#pragma unroll
        for (int v = 0; v < V; ++v)                              // the next row is in flight meanwhile
            cur[v] = load_raw8<XB>(a.x, nrow * a.ldx + (t + v * T) * 8, nrow < a.rows ? valid[v] : 0);

        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) s += x[v][i];            // elements past the row read as 0
        float mean = group_sum<LANES>(s) * inv_n_w;
        float m2 = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = x[v][i] - mean;
                m2 += i < valid[v] ? d * d : 0.0f;
            }
        m2 = group_sum<LANES>(m2);
        if (WIDE) {
            if ((threadIdx.x & 31) == 0) sStat[buf][warp] = make_float2(mean * n_w, m2);
            __syncthreads();
            // lane w holds warp w's part; n_w of another warp follows from its columns
            const int lane = threadIdx.x & 31;
            const float2 p = lane < nw ? sStat[buf][lane] : make_float2(0.0f, 0.0f);
            float n = 0.0f;
            if (lane < nw) {
#pragma unroll
                for (int v = 0; v < V; ++v) n += (float)max(0, min(256, a.cols - (lane * 32 + v * T) * 8));
            }
            mean = group_sum<32>(p.x) * a.inv_cols;
            const float d = n > 0.0f ? p.x / n - mean : 0.0f;
            m2 = group_sum<32>(p.y + n * d * d);
            buf ^= 1;
        }
        const float var = m2 * a.inv_cols;
        const float rstd = __frsqrt_rn(var + a.eps);
        if (t == 0 && live) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int col = (t + v * T) * 8;
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = fmaf((x[v][i] - mean) * rstd, gm[v][i], bt[v][i]);
            const int n = live ? valid[v] : 0;
            if (OUT != OUT_F8) {
                if (n > 0) store8<OUT == OUT_BF16>(a.y, row * a.ldy + col, y, n);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i >= n) y[i] = 0.0f;
                constexpr int W = LANES < 16 ? LANES : 16;       // lanes of a 128-block
                uint32_t m = amax_bits(y);
#pragma unroll
                for (int o = W / 2; o; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
                if (__any_sync(0xFFFFFFFFu, m >= kInfBits)) {    // rare: map what is not finite, and again
                    sanitize_all(y, bad);
                    m = amax_bits(y);
#pragma unroll
                    for (int o = W / 2; o; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
                }
                const float s = scale_or_factor(m, a.fmax, t & 1);
                const float f = __shfl_sync(0xFFFFFFFFu, s, 0, W);
                uint32_t lo, hi;
                if (a.e5m2) {
                    lo = encode4<true>(y[0], y[1], y[2], y[3], f);
                    hi = encode4<true>(y[4], y[5], y[6], y[7], f);
                } else {
                    lo = encode4<false>(y[0], y[1], y[2], y[3], f);
                    hi = encode4<false>(y[4], y[5], y[6], y[7], f);
                }
                if (n > 0) {
                    store_codes8(static_cast<uint8_t *>(a.y) + row * a.ldy + col, lo, hi, n);
                }
                // the block's second lane holds the scale
                if (live && t % W == 1 && col - 8 < a.cols) a.scale[(int64_t)(col / BLK) * a.lds + row] = s;
            }
        }
    }
    if (bad) status_or(a.status, HIF4_FLAG_NONFINITE);
}

template <bool XB, int V, int LANES, int WIDE>
__global__ void __launch_bounds__(WIDE ? WIDE : kSmallThreads) k_norm_bwd(NormBwdArgs a)
{
    __shared__ float2 sSum[WIDE ? 2 : 1][32];
    __shared__ float sCol[WIDE ? 1 : kSmallThreads * V * 8];     // column sums of the block's row groups
    pdl_enter();
    const int T = WIDE ? blockDim.x : LANES;
    const int t = WIDE ? threadIdx.x : threadIdx.x % LANES;
    const int warp = threadIdx.x >> 5;
    const int rpb = WIDE ? 1 : kSmallThreads / LANES;
    const int nw = blockDim.x >> 5;

    int valid[V];
    float gm[V][8], dg[V][8], db[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int col = (t + v * T) * 8;
        valid[v] = max(0, min(8, a.cols - col));
        load_params(a.gamma, a.param_bf16, col, valid[v], 1.0f, gm[v]);
#pragma unroll
        for (int i = 0; i < 8; ++i) dg[v][i] = db[v][i] = 0.0f;
    }
    int buf = 0;
    const int64_t step = (int64_t)gridDim.x * rpb;
    int64_t row = (int64_t)blockIdx.x * rpb + (WIDE ? 0 : threadIdx.x / LANES);
    int64_t wrow = WIDE ? row : (int64_t)blockIdx.x * rpb + warp * (32 / LANES);
    Raw8<XB> cx[V], cd[V];
    float cmean = 0.0f, crstd = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int n = row < a.rows ? valid[v] : 0;
        cx[v] = load_raw8<XB>(a.x, row * a.ldx + (t + v * T) * 8, n);
        cd[v] = load_raw8<XB>(a.dy, row * a.lddy + (t + v * T) * 8, n);
    }
    if (row < a.rows) {
        cmean = a.mean[row];
        crstd = a.rstd[row];
    }
    for (; wrow < a.rows; wrow += step, row += step) {
        const bool live = row < a.rows;
        const float mean = cmean, rstd = crstd;
        float s1 = 0.0f, s2 = 0.0f;
        float xh[V][8], d[V][8];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            widen8<XB>(cx[v], xh[v]);
            widen8<XB>(cd[v], d[v]);                             // 0 past the row and for rows past the end
        }
        const int64_t nrow = row + step;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int n = nrow < a.rows ? valid[v] : 0;
            cx[v] = load_raw8<XB>(a.x, nrow * a.ldx + (t + v * T) * 8, n);
            cd[v] = load_raw8<XB>(a.dy, nrow * a.lddy + (t + v * T) * 8, n);
        }
        if (nrow < a.rows) {
            cmean = a.mean[nrow];
            crstd = a.rstd[nrow];
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int n = live ? valid[v] : 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                xh[v][i] = i < n ? (xh[v][i] - mean) * rstd : 0.0f;
                dg[v][i] = fmaf(d[v][i], xh[v][i], dg[v][i]);
                db[v][i] += d[v][i];
                d[v][i] *= gm[v][i];
                s1 += d[v][i];
                s2 = fmaf(d[v][i], xh[v][i], s2);
            }
        }
        s1 = group_sum<LANES>(s1);
        s2 = group_sum<LANES>(s2);
        if (WIDE) {
            if ((threadIdx.x & 31) == 0) sSum[buf][warp] = make_float2(s1, s2);
            __syncthreads();
            const int lane = threadIdx.x & 31;
            const float2 p = lane < nw ? sSum[buf][lane] : make_float2(0.0f, 0.0f);
            s1 = group_sum<32>(p.x);
            s2 = group_sum<32>(p.y);
            buf ^= 1;
        }
        const float c1 = s1 * a.inv_cols, c2 = s2 * a.inv_cols;
        if (a.dx) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = rstd * (d[v][i] - c1 - xh[v][i] * c2);
                if (live && valid[v] > 0) store8<XB>(a.dx, row * a.lddx + (t + v * T) * 8, o, valid[v]);
            }
        }
    }
    if (!a.part) return;
    float *pg = a.part + (int64_t)blockIdx.x * 2 * a.cols, *pb = pg + a.cols;
    if (WIDE) {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < valid[v]) {
                    pg[(t + v * T) * 8 + i] = dg[v][i];
                    pb[(t + v * T) * 8 + i] = db[v][i];
                }
    } else {
        // the block's row groups, added in order: group g's sums lie at g * (LANES V 8)
        constexpr int W = LANES * V * 8;
        const int g = threadIdx.x / LANES;
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
            if (pass) __syncthreads();
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int i = 0; i < 8; ++i) sCol[g * W + (t + v * LANES) * 8 + i] = pass ? db[v][i] : dg[v][i];
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
    const int c = blockIdx.x * 32 + threadIdx.x;                 // over 2 x cols: dgamma, then dbeta
    float v = 0.0f;
    if (c < 2 * cols)
        for (int p = threadIdx.y; p < parts; p += 32) v += part[(int64_t)p * 2 * cols + c];
    s[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    v = s[threadIdx.x][threadIdx.y];                             // lane = part, warp = column
    v = group_sum<32>(v);
    const int co = blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && co < 2 * cols) {
        if (co < cols) {
            if (dgamma) dgamma[co] = v;
        } else if (dbeta) {
            dbeta[co - cols] = v;
        }
    }
}

// Threads of a row's group and granules per thread.  8 lanes up to 64 columns,
// a warp up to 1024, then a block.
struct Shape {
    int lanes, v, threads, wide;
};

Shape shape_of(int64_t cols)
{
    const int g = (int)((cols + 7) / 8);
    if (g <= 8) return Shape{8, 1, kSmallThreads, 0};
    if (g <= 32) return Shape{32, 1, kSmallThreads, 0};
    if (g <= 64) return Shape{32, 2, kSmallThreads, 0};
    if (g <= 128) return Shape{32, 4, kSmallThreads, 0};
    return Shape{32, 2, (g + 63) / 64 * 32, g <= 1024 ? 512 : 1024};
}

template <bool XB, int OUT>
hif4_status launch_fwd(const NormArgs &a, cudaStream_t s)
{
    const Shape sh = shape_of(a.cols);
    void (*k)(NormArgs);
    if (sh.wide)
        k = sh.wide == 512 ? k_norm_fwd<XB, OUT, 2, 32, 512> : k_norm_fwd<XB, OUT, 2, 32, 1024>;
    else if (sh.lanes == 8)
        k = k_norm_fwd<XB, OUT, 1, 8, 0>;
    else
        k = sh.v == 1 ? k_norm_fwd<XB, OUT, 1, 32, 0>
                      : sh.v == 2 ? k_norm_fwd<XB, OUT, 2, 32, 0> : k_norm_fwd<XB, OUT, 4, 32, 0>;
    const int rpb = sh.wide ? 1 : kSmallThreads / sh.lanes;
    int64_t grid = ((int64_t)a.rows + rpb - 1) / rpb;
    const int64_t most = (int64_t)sm_count() * blocks_per_sm(reinterpret_cast<const void *>(k), sh.threads, 0);
    if (grid > most) grid = most;
    return launch_pdl(k, dim3((unsigned)grid), dim3((unsigned)sh.threads), 0, s, a);
}

template <bool XB>
hif4_status launch_bwd(const NormBwdArgs &a, float *dgamma, float *dbeta, cudaStream_t s)
{
    const Shape sh = shape_of(a.cols);
    void (*k)(NormBwdArgs);
    if (sh.wide)
        k = sh.wide == 512 ? k_norm_bwd<XB, 2, 32, 512> : k_norm_bwd<XB, 2, 32, 1024>;
    else if (sh.lanes == 8)
        k = k_norm_bwd<XB, 1, 8, 0>;
    else
        k = sh.v == 1 ? k_norm_bwd<XB, 1, 32, 0>
                      : sh.v == 2 ? k_norm_bwd<XB, 2, 32, 0> : k_norm_bwd<XB, 4, 32, 0>;
    const int rpb = sh.wide ? 1 : kSmallThreads / sh.lanes;
    int64_t grid = ((int64_t)a.rows + rpb - 1) / rpb;
    const int64_t most = (int64_t)sm_count() * blocks_per_sm(reinterpret_cast<const void *>(k), sh.threads, 0);
    if (grid > most) grid = most;
    if (grid > kMaxPartials) grid = kMaxPartials;
    hif4_status st = launch_pdl(k, dim3((unsigned)grid), dim3((unsigned)sh.threads), 0, s, a);
    if (st != HIF4_OK || !a.part) return st;
    return launch_pdl(k_norm_bwd_join, dim3((unsigned)((2 * a.cols + 31) / 32)), dim3(32, 32), 0, s, a.part,
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
    if (cols > kMaxCols || rows > INT32_MAX) return HIF4_ERR_UNSUPPORTED;
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
    a.fmax = f8::fmt_max(fmt);
    a.e5m2 = fmt == HIF4_E5M2;
    a.status = status;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return dtype == HIF4_BF16 ? launch_fwd<true, OUT_F8>(a, s) : launch_fwd<false, OUT_F8>(a, s);
}

extern "C" size_t hif4_layer_norm_backward_workspace(int64_t rows, int64_t cols)
{
    if (rows <= 0 || cols <= 0 || cols > kMaxCols) return 0;
    const int64_t n = rows < kMaxPartials ? rows : kMaxPartials;
    return (size_t)n * 2 * (size_t)cols * sizeof(float);
}

extern "C" hif4_status hif4_layer_norm_backward(const void *dy, int64_t lddy, const void *x, hif4_dtype dtype,
                                                int64_t rows, int64_t cols, int64_t ldx, const float *mean,
                                                const float *rstd, const void *gamma, hif4_dtype param_dtype,
                                                void *dx, int64_t lddx, float *dgamma, float *dbeta,
                                                void *workspace, size_t ws_bytes, hif4_stream_t stream)
{
    if (rows < 0 || cols < 0 || !valid_dtype(dtype) || !valid_dtype(param_dtype)) return HIF4_ERR_INVALID_ARG;
    if (cols == 0) return HIF4_OK;
    if (cols > kMaxCols || rows > INT32_MAX) return HIF4_ERR_UNSUPPORTED;
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
