// hif4_f8_quant.cu — FP8 quantization with one FP32 scale per block of 128.
//
// HBM-bound streaming kernels: every input element is read once, whatever
// layouts are asked for, and every code byte and scale written once.
//
//   k_f8_rows   1 x 128 blocks, row-major codes only: 16 lanes own a block,
//               8 elements each; four xor-shuffles give its maximum.
//   k_f8_tile   everything else: one 128 x 128 tile per CTA, an 8 x 8 piece
//               per thread in registers, so that row maxima, column maxima
//               and the tile's maximum all come from one read.  The
//               transposed codes go through shared memory, so that they too
//               leave in 16-byte pieces of consecutive rows.
#include "hif4_f8.cuh"

namespace hif4 {
namespace {

using namespace f8;

struct F8QuantArgs {
    const void *x;
    int64_t rows, cols, ldx;
    uint8_t *q;
    int64_t ldq;
    float *scale;
    int64_t lds;
    uint8_t *qt;
    int64_t ldqt;
    float *scale_t;
    int64_t ldst;
    uint32_t nblk;             // column blocks
    FastDiv nblk_div;
    uint32_t items;            // k_f8_rows: rows x nblk
    uint32_t *status;
    float fmax;
    bool e5m2;
};

constexpr int kThreads = 256;

template <bool BF16>
__global__ void __launch_bounds__(kThreads) k_f8_rows(F8QuantArgs a)
{
    const int l16 = threadIdx.x & 15;
    uint32_t bad = 0;
    const uint32_t stride = gridDim.x * (kThreads / 16);
    // all lanes of a warp take the same number of trips (shuffles below)
    const uint32_t first = blockIdx.x * (kThreads / 16) + (threadIdx.x >> 5) * 2;
    for (uint32_t w = first; w < a.items; w += stride) {
        const uint32_t it = w + ((threadIdx.x >> 4) & 1);
        const bool live = it < a.items;
        const uint32_t row = live ? a.nblk_div.div(it) : 0;
        const uint32_t blk = live ? it - row * a.nblk : 0;
        const int64_t col = (int64_t)blk * BLK + l16 * 8;
        const int valid = live ? (int)max((int64_t)0, min((int64_t)8, a.cols - col)) : 0;
        float v[8];
        widen8<BF16>(load_raw8<BF16>(a.x, (int64_t)row * a.ldx + col, valid), v);
        sanitize_all(v, bad);
        float m = amax8(v);
#pragma unroll
        for (int o = 8; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const ScalePair sp = scale_pair(m, a.fmax);
        const uint32_t lo = cvt4(v[0] * sp.factor, v[1] * sp.factor, v[2] * sp.factor, v[3] * sp.factor, a.e5m2);
        const uint32_t hi = cvt4(v[4] * sp.factor, v[5] * sp.factor, v[6] * sp.factor, v[7] * sp.factor, a.e5m2);
        if (valid > 0) store_codes8(a.q + (int64_t)row * a.ldq + col, lo, hi, valid);
        if (live && l16 == 0) a.scale[(int64_t)blk * a.lds + row] = sp.scale;
    }
    if (bad) status_or(a.status, HIF4_FLAG_NONFINITE);
}

// 16 codes of one column (rows c16 * 16 ..) from the staged tile: column c's
// 8-byte unit g (rows 8 g ..) sits at unit g ^ (c / 8) of its 128-byte line,
// so that the writes of a half-warp (16 columns 8 apart, one g) and the reads
// below are free of bank conflicts.
__device__ __forceinline__ uint4 staged16(const uint8_t *sT, int c, int c16)
{
    const int s = c >> 3;
    const uint4 w = *reinterpret_cast<const uint4 *>(sT + c * BLK + (((2 * c16) ^ (s & ~1)) * 8));
    return (s & 1) ? make_uint4(w.z, w.w, w.x, w.y) : w;
}

// SQUARE: 128 x 128 blocks (both layouts share the tile's scale); otherwise
// 1 x 128 blocks row-wise and 128 x 1 blocks for the transposed codes.
template <bool BF16, bool SQUARE>
__global__ void __launch_bounds__(kThreads) k_f8_tile(F8QuantArgs a)
{
    __shared__ __align__(16) uint8_t sT[BLK * BLK];
    __shared__ float sMax[kThreads / 32][BLK];
    const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4, warp = threadIdx.x >> 5;
    const uint32_t rb = a.nblk_div.div(blockIdx.x);
    const uint32_t cb = blockIdx.x - rb * a.nblk;
    const int64_t r0 = (int64_t)rb * BLK + rg * 8;
    const int64_t c0 = (int64_t)cb * BLK + cg * 8;
    const int cvalid = (int)max((int64_t)0, min((int64_t)8, a.cols - c0));
    const int rvalid = (int)max((int64_t)0, min((int64_t)8, a.rows - r0));

    float v[8][8];
    {
        Raw8<BF16> raw[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) raw[i] = load_raw8<BF16>(a.x, (r0 + i) * a.ldx + c0, i < rvalid ? cvalid : 0);
#pragma unroll
        for (int i = 0; i < 8; ++i) widen8<BF16>(raw[i], v[i]);
    }
    uint32_t bad = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) sanitize_all(v[i], bad);
    if (bad) status_or(a.status, HIF4_FLAG_NONFINITE);

    float tile_factor = 0.0f;
    if (SQUARE) {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, amax8(v[i]));
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        if ((threadIdx.x & 31) == 0) sMax[warp][0] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) m = fmaxf(m, sMax[w][0]);
        const ScalePair sp = scale_pair(m, a.fmax);
        tile_factor = sp.factor;
        if (threadIdx.x == 0) {
            if (a.q) a.scale[(int64_t)rb * a.lds + cb] = sp.scale;
            if (a.qt) a.scale_t[(int64_t)cb * a.ldst + rb] = sp.scale;
        }
    }
    if (a.q) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float f = tile_factor;
            if (!SQUARE) {
                float m = amax8(v[i]);
#pragma unroll
                for (int o = 8; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
                const ScalePair sp = scale_pair(m, a.fmax);
                f = sp.factor;
                if (cg == 0 && i < rvalid) a.scale[(int64_t)cb * a.lds + r0 + i] = sp.scale;
            }
            const uint32_t lo = cvt4(v[i][0] * f, v[i][1] * f, v[i][2] * f, v[i][3] * f, a.e5m2);
            const uint32_t hi = cvt4(v[i][4] * f, v[i][5] * f, v[i][6] * f, v[i][7] * f, a.e5m2);
            if (i < rvalid && cvalid > 0) store_codes8(a.q + (r0 + i) * a.ldq + c0, lo, hi, cvalid);
        }
    }
    if (a.qt) {
        if (!SQUARE) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float m = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i][j]));
                m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));
                if ((threadIdx.x & 31) < 16) sMax[warp][cg * 8 + j] = m;
            }
            __syncthreads();
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float f = tile_factor;
            if (!SQUARE) {
                float m = 0.0f;
#pragma unroll
                for (int w = 0; w < kThreads / 32; ++w) m = fmaxf(m, sMax[w][cg * 8 + j]);
                const ScalePair sp = scale_pair(m, a.fmax);
                f = sp.factor;
                if (rg == 0 && j < cvalid) a.scale_t[(int64_t)rb * a.ldst + c0 + j] = sp.scale;
            }
            const uint32_t lo = cvt4(v[0][j] * f, v[1][j] * f, v[2][j] * f, v[3][j] * f, a.e5m2);
            const uint32_t hi = cvt4(v[4][j] * f, v[5][j] * f, v[6][j] * f, v[7][j] * f, a.e5m2);
            *reinterpret_cast<uint2 *>(sT + (cg * 8 + j) * BLK + ((rg ^ cg) * 8)) = make_uint2(lo, hi);
        }
        __syncthreads();
        const int64_t rbase = (int64_t)rb * BLK;
#pragma unroll
        for (int k = 0; k < BLK * BLK / 16 / kThreads; ++k) {
            const int p = threadIdx.x + k * kThreads;
            const int c = p >> 3, c16 = p & 7;
            const int64_t col = (int64_t)cb * BLK + c;
            const int64_t row = rbase + c16 * 16;
            if (col < a.cols && row < a.rows) {
                const uint4 w = staged16(sT, c, c16);
                uint8_t *dst = a.qt + col * a.ldqt + row;
                if (row + 16 <= a.rows) {
                    *reinterpret_cast<uint4 *>(dst) = w;
                } else {
                    store_codes8(dst, w.x, w.y, (int)min((int64_t)8, a.rows - row));
                    if (a.rows - row > 8) store_codes8(dst + 8, w.z, w.w, (int)(a.rows - row - 8));
                }
            }
        }
    }
}

} // namespace
} // namespace hif4

using namespace hif4;

extern "C" hif4_status hif4_quantize_f8(const void *x, hif4_dtype dtype, int64_t rows, int64_t cols, int64_t ldx,
                                        hif4_f8_format fmt, int32_t block_rows, uint8_t *q, int64_t ldq,
                                        float *scale, int64_t lds, uint8_t *qt, int64_t ldqt, float *scale_t,
                                        int64_t ldst, uint32_t *status, hif4_stream_t stream)
{
    if (rows < 0 || cols < 0 || (dtype != HIF4_F32 && dtype != HIF4_BF16) || !f8::valid_fmt(fmt))
        return HIF4_ERR_INVALID_ARG;
    if (block_rows != 1 && block_rows != 128) return HIF4_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return HIF4_OK;
    if (!x || (!q && !qt) || (q && !scale) || (qt && !scale_t)) return HIF4_ERR_INVALID_ARG;
    const int64_t rblk = f8::blocks_of(rows), cblk = f8::blocks_of(cols);
    const bool square = block_rows == 128;
    if (ldx < cols) return HIF4_ERR_SHAPE;
    if (q && (ldq < cols || lds < (square ? cblk : rows))) return HIF4_ERR_SHAPE;
    if (qt && (ldqt < rows || ldst < (square ? rblk : cols))) return HIF4_ERR_SHAPE;
    const int64_t esz = dtype == HIF4_BF16 ? 2 : 4;
    if (!aligned16(x) || ldx % (16 / esz)) return HIF4_ERR_ALIGNMENT;
    if (q && (!aligned16(q) || ldq % 16 || !aligned_to(scale, 4))) return HIF4_ERR_ALIGNMENT;
    if (qt && (!aligned16(qt) || ldqt % 16 || !aligned_to(scale_t, 4))) return HIF4_ERR_ALIGNMENT;
    if (rows > INT32_MAX || cols > INT32_MAX || rows > (int64_t)INT32_MAX / cblk) return HIF4_ERR_UNSUPPORTED;

    F8QuantArgs a{};
    a.x = x;
    a.rows = rows;
    a.cols = cols;
    a.ldx = ldx;
    a.q = q;
    a.ldq = ldq;
    a.scale = scale;
    a.lds = lds;
    a.qt = qt;
    a.ldqt = ldqt;
    a.scale_t = scale_t;
    a.ldst = ldst;
    a.nblk = (uint32_t)cblk;
    a.nblk_div = FastDiv((uint32_t)cblk);
    a.items = (uint32_t)(rows * cblk);
    a.status = status;
    a.fmax = f8::fmt_max(fmt);
    a.e5m2 = fmt == HIF4_E5M2;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (!square && !qt) {
        int64_t grid = ((int64_t)a.items + kThreads / 16 - 1) / (kThreads / 16);
        const int64_t most = 32 * (int64_t)sm_count();
        if (grid > most) grid = most;
        if (dtype == HIF4_BF16)
            k_f8_rows<true><<<(unsigned)grid, kThreads, 0, s>>>(a);
        else
            k_f8_rows<false><<<(unsigned)grid, kThreads, 0, s>>>(a);
        return launch_status();
    }
    const unsigned grid = (unsigned)(rblk * cblk);
    if (dtype == HIF4_BF16) {
        if (square)
            k_f8_tile<true, true><<<grid, kThreads, 0, s>>>(a);
        else
            k_f8_tile<true, false><<<grid, kThreads, 0, s>>>(a);
    } else {
        if (square)
            k_f8_tile<false, true><<<grid, kThreads, 0, s>>>(a);
        else
            k_f8_tile<false, false><<<grid, kThreads, 0, s>>>(a);
    }
    return launch_status();
}
