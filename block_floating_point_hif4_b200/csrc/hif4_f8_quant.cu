// hif4_f8_quant.cu — FP8 quantization with one FP32 scale per block of 128.
//
// HBM-bound streaming kernels: every input element is read once, whatever
// layouts are asked for, and every code byte and scale written once.
//
//   k_f8_rows   1 x 128 blocks, row-major codes only: 8 lanes own a block,
//               16 elements each.
//   k_f8_tile   everything else: one 128 x 128 tile per CTA, an 8 x 8 piece
//               per thread in registers, so that row maxima, column maxima
//               and the tile's maximum all come from one read.  The
//               transposed codes go through shared memory, so that they too
//               leave in 16-byte pieces of consecutive rows.
//
// What the arithmetic costs is kept below the memory's time: maxima on pairs
// of 16-bit keys (BF16), one of the two quotients of a block in each lane
// instead of both in all, packed FP32 products, and a test for what is not
// finite once per block's maximum.  Measured (device time): 57600 x 5120 BF16
// rows 150.5 us, 5.94 TB/s of algorithmic bytes, 0.91 of the copy bandwidth
// (229 us with scalar maxima and both quotients in every lane, 172 us before
// the register limit of 32, i.e. 8 blocks per SM); prefetching the next strip in
// registers measured slower (187 us).  16384 x 5120, both layouts, 62.6 us,
// 0.83 (84 us while the piece was held as FP32 values, 116 registers); a
// 13824 x 5120 weight in 128 x 128 blocks, both layouts, 50.1 us, 0.86; 8192 x
// 5120 FP32 rows 34.0 us, 0.94.  A call on cold operands takes about 5 % longer.
// The tile kernel's issue slots are 69 % busy with 4 CTAs per SM, each of which
// loads, encodes and stores one tile after the other's end.
#include "hif4_f8.cuh"
#include "hif4_pdl.cuh"

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
    uint32_t items;            // k_f8_rows: strips of 32 rows x nblk
    uint32_t *status;
    float fmax;
};

constexpr int kThreads = 256;
constexpr int kRowsPerCta = kThreads / 8;      // k_f8_rows: rows of a 128-column strip that a block takes at once

// 1 x 128 blocks, row-major codes.  Eight lanes own a block: two granules each,
// 64 elements apart, so that a load of the eight covers 128 consecutive bytes
// of BF16.  The 32 groups of a CTA take one 128-column strip of 32 consecutive
// rows, whose scales are 32 consecutive floats.
template <bool BF16, bool E5M2>
__global__ void __launch_bounds__(kThreads, BF16 ? 8 : 6) k_f8_rows(F8QuantArgs a)
{
    pdl_enter();
    const int l8 = threadIdx.x & 7, group = threadIdx.x >> 3;
    bool bad = false;
    for (uint32_t it = blockIdx.x; it < a.items; it += gridDim.x) {
        const uint32_t strip = a.nblk_div.div(it);
        const uint32_t blk = it - strip * a.nblk;
        const int64_t row = (int64_t)strip * kRowsPerCta + group;
        const int64_t col = (int64_t)blk * BLK + l8 * 8;
        const bool live = row < a.rows;
        const int v0 = live ? (int)max((int64_t)0, min((int64_t)8, a.cols - col)) : 0;
        const int v1 = live ? (int)max((int64_t)0, min((int64_t)8, a.cols - col - 64)) : 0;
        const int64_t off = row * a.ldx + col;
        Raw8<BF16> r0 = load_raw8<BF16>(a.x, off, v0), r1 = load_raw8<BF16>(a.x, off + 64, v1);
        uint32_t m = max(amax_bits<BF16>(r0), amax_bits<BF16>(r1));
#pragma unroll
        for (int o = 4; o; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        float x[2][8];
        widen8<BF16>(r0, x[0]);
        widen8<BF16>(r1, x[1]);
        if (__any_sync(0xFFFFFFFFu, m >= kInfBits)) {            // rare: map what is not finite, and again
            uint32_t mapped = 0;
            sanitize_all(x[0], mapped);
            sanitize_all(x[1], mapped);
            bad |= mapped != 0;
            m = max(amax_bits(x[0]), amax_bits(x[1]));
#pragma unroll
            for (int o = 4; o; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        }
        const float s = scale_or_factor(m, a.fmax, l8 & 1);
        const float f = __shfl_sync(0xFFFFFFFFu, s, 0, 8);
        uint8_t *q = a.q + row * a.ldq + col;
        if (v0 > 0)
            store_codes8(q, encode4<E5M2>(x[0][0], x[0][1], x[0][2], x[0][3], f),
                         encode4<E5M2>(x[0][4], x[0][5], x[0][6], x[0][7], f), v0);
        if (v1 > 0)
            store_codes8(q + 64, encode4<E5M2>(x[1][0], x[1][1], x[1][2], x[1][3], f),
                         encode4<E5M2>(x[1][4], x[1][5], x[1][6], x[1][7], f), v1);
        if (live && l8 == 1) a.scale[(int64_t)blk * a.lds + row] = s;
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

// 4 x 4 bytes: word i holds row i; -> word j holds column j.
__device__ __forceinline__ void transpose4(uint32_t &a, uint32_t &b, uint32_t &c, uint32_t &d)
{
    const uint32_t ab0 = __byte_perm(a, b, 0x5140), ab1 = __byte_perm(a, b, 0x7362);   // a0 b0 a1 b1, a2 b2 a3 b3
    const uint32_t cd0 = __byte_perm(c, d, 0x5140), cd1 = __byte_perm(c, d, 0x7362);
    a = __byte_perm(ab0, cd0, 0x5410);
    b = __byte_perm(ab0, cd0, 0x7632);
    c = __byte_perm(ab1, cd1, 0x5410);
    d = __byte_perm(ab1, cd1, 0x7632);
}

// Element j of a raw granule.
template <bool BF16>
__device__ __forceinline__ float element(const Raw8<BF16> &r, int j)
{
    if (BF16) {
        const uint32_t w = j < 2 ? r.w[0].x : j < 4 ? r.w[0].y : j < 6 ? r.w[0].z : r.w[0].w;
        return j & 1 ? bf16_hi(w) : bf16_lo(w);
    }
    const uint4 h = r.w[!BF16 && j >= 4 ? 1 : 0];
    return bits_f((j & 3) == 0 ? h.x : (j & 3) == 1 ? h.y : (j & 3) == 2 ? h.z : h.w);
}

__device__ __forceinline__ uint32_t finite_max(uint32_t bits) { return min(bits, kInfBits - 1); }

// NaN -> 0 in a raw granule.
template <bool BF16>
__device__ __forceinline__ void clear_nan(Raw8<BF16> &r)
{
#pragma unroll
    for (int k = 0; k < (BF16 ? 1 : 2); ++k) {
        uint32_t w[4] = {r.w[k].x, r.w[k].y, r.w[k].z, r.w[k].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (BF16) {
                if ((w[i] & 0x7FFFu) > 0x7F80u) w[i] &= 0xFFFF0000u;
                if ((w[i] & 0x7FFF0000u) > kInfBits) w[i] &= 0x0000FFFFu;
            } else if ((w[i] & 0x7FFFFFFFu) > kInfBits) {
                w[i] = 0;
            }
        }
        r.w[k] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Bits of the largest magnitude of each of the 8 columns of 8 granules.
template <bool BF16>
__device__ __forceinline__ void column_max(const Raw8<BF16> (&r)[8], uint32_t (&m)[8])
{
    if (BF16) {
        uint32_t p[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            p[0] = max_u16x2(p[0], r[i].w[0].x & 0x7FFF7FFFu);
            p[1] = max_u16x2(p[1], r[i].w[0].y & 0x7FFF7FFFu);
            p[2] = max_u16x2(p[2], r[i].w[0].z & 0x7FFF7FFFu);
            p[3] = max_u16x2(p[3], r[i].w[0].w & 0x7FFF7FFFu);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) m[j] = j & 1 ? p[j >> 1] & 0xFFFF0000u : p[j >> 1] << 16;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            m[j] = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m[j] = max(m[j], f_bits(element<BF16>(r[i], j)) & 0x7FFFFFFFu);
        }
    }
}

// SQUARE: 128 x 128 blocks (both layouts hold the same codes); otherwise
// 1 x 128 blocks row-wise and 128 x 1 blocks for the transposed codes.
// Thread (rg, cg) = (t / 16, t % 16) owns rows 8 rg .. and columns 8 cg .. of
// the tile.
template <bool BF16, bool SQUARE, bool E5M2>
__global__ void __launch_bounds__(kThreads, BF16 ? 4 : 2) k_f8_tile(F8QuantArgs a)
{
    __shared__ __align__(16) uint8_t sT[BLK * BLK];
    __shared__ __align__(16) uint32_t sMax[kThreads / 32][BLK];
    __shared__ __align__(16) float sF[BLK];
    pdl_enter();
    const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4, warp = threadIdx.x >> 5;
    const uint32_t rb = a.nblk_div.div(blockIdx.x);
    const uint32_t cb = blockIdx.x - rb * a.nblk;
    const int64_t r0 = (int64_t)rb * BLK + rg * 8;
    const int64_t c0 = (int64_t)cb * BLK + cg * 8;
    const int cvalid = (int)max((int64_t)0, min((int64_t)8, a.cols - c0));
    const int rvalid = (int)max((int64_t)0, min((int64_t)8, a.rows - r0));

    // The piece stays as it was read (BF16: half the registers of its FP32 values).
    Raw8<BF16> raw[8];
    uint32_t rmax[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) raw[i] = load_raw8<BF16>(a.x, (r0 + i) * a.ldx + c0, i < rvalid ? cvalid : 0);
    {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            rmax[i] = amax_bits<BF16>(raw[i]);
            m = max(m, rmax[i]);
        }
        if (m >= kInfBits) {                                     // rare
            // NaN -> 0 here; an infinity counts as FLT_MAX in the maxima (finite_max) and meets its code,
            // the largest one, by the saturating conversion
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                clear_nan<BF16>(raw[i]);
                rmax[i] = amax_bits<BF16>(raw[i]);
            }
            status_or(a.status, HIF4_FLAG_NONFINITE);
        }
    }

    float f[8];                                                  // factors: of the rows, then of the columns
    if (SQUARE) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, rmax[i]);
        m = __reduce_max_sync(0xFFFFFFFFu, m);
        if ((threadIdx.x & 31) == 0) sMax[warp][0] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) m = max(m, sMax[w][0]);
        const float s = scale_or_factor(finite_max(m), a.fmax, cg & 1);
        const float t = __shfl_sync(0xFFFFFFFFu, s, 0);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = t;
        if (threadIdx.x == 1) {
            if (a.q) a.scale[(int64_t)rb * a.lds + cb] = s;
            if (a.qt) a.scale_t[(int64_t)cb * a.ldst + rb] = s;
        }
    } else if (a.q) {
        // The 16 lanes of a row group hold parts of the same 8 rows: halving exchanges leave lane bits
        // 3..1 with the maximum of row (bits 3..1), and bit 0 chooses the quotient that the lane forms.
        uint32_t k4[4], k2[2], k1;
        const bool b3 = cg & 8, b2 = cg & 4, b1 = cg & 2;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, b3 ? rmax[i] : rmax[i + 4], 8);
            k4[i] = max(b3 ? rmax[i + 4] : rmax[i], other);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, b2 ? k4[i] : k4[i + 2], 4);
            k2[i] = max(b2 ? k4[i + 2] : k4[i], other);
        }
        {
            const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, b1 ? k2[0] : k2[1], 2);
            k1 = max(b1 ? k2[1] : k2[0], other);
        }
        k1 = max(k1, __shfl_xor_sync(0xFFFFFFFFu, k1, 1));
        const float s = scale_or_factor(finite_max(k1), a.fmax, cg & 1);
        const int row = cg >> 1;
        if ((cg & 1) && row < rvalid) a.scale[(int64_t)cb * a.lds + r0 + row] = s;
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __shfl_sync(0xFFFFFFFFu, s, 2 * i, 16);
    }
    if (!SQUARE && a.qt) {
        // column maxima: over the thread's rows, the warp's two row groups, then the warps
        uint32_t cm[8];
        column_max<BF16>(raw, cm);
#pragma unroll
        for (int j = 0; j < 8; ++j) cm[j] = max(cm[j], __shfl_xor_sync(0xFFFFFFFFu, cm[j], 16));
        if ((threadIdx.x & 31) < 16) {
            *reinterpret_cast<uint4 *>(&sMax[warp][cg * 8]) = make_uint4(cm[0], cm[1], cm[2], cm[3]);
            *reinterpret_cast<uint4 *>(&sMax[warp][cg * 8 + 4]) = make_uint4(cm[4], cm[5], cm[6], cm[7]);
        }
        __syncthreads();
        const int c = threadIdx.x & (BLK - 1);
        uint32_t m = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) m = max(m, sMax[w][c]);
        const bool want_scale = threadIdx.x >= BLK;              // the two halves form one quotient each
        const float s = scale_or_factor(finite_max(m), a.fmax, want_scale);
        const int64_t col = (int64_t)cb * BLK + c;
        if (!want_scale)
            sF[c] = s;
        else if (col < a.cols)
            a.scale_t[(int64_t)rb * a.ldst + col] = s;
    }

    uint32_t w0[8], w1[8];                                       // SQUARE: codes of the thread's rows
    if (SQUARE || a.q) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float v[8];
            widen8<BF16>(raw[i], v);
            const uint32_t lo = encode4<E5M2>(v[0], v[1], v[2], v[3], f[i]);
            const uint32_t hi = encode4<E5M2>(v[4], v[5], v[6], v[7], f[i]);
            if (a.q && i < rvalid && cvalid > 0) store_codes8(a.q + (r0 + i) * a.ldq + c0, lo, hi, cvalid);
            if (SQUARE) {
                w0[i] = lo;
                w1[i] = hi;
            }
        }
    }
    if (!a.qt) return;
    if (SQUARE) {
        transpose4(w0[0], w0[1], w0[2], w0[3]);
        transpose4(w0[4], w0[5], w0[6], w0[7]);
        transpose4(w1[0], w1[1], w1[2], w1[3]);
        transpose4(w1[4], w1[5], w1[6], w1[7]);
    } else {
        __syncthreads();                                         // sF is complete
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = sF[cg * 8 + j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        uint32_t lo, hi;                                         // column j: rows 0..3, 4..7
        if (SQUARE) {
            lo = j < 4 ? w0[j & 3] : w1[j & 3];
            hi = j < 4 ? w0[4 + (j & 3)] : w1[4 + (j & 3)];
        } else {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = element<BF16>(raw[i], j);
            lo = encode4<E5M2>(v[0], v[1], v[2], v[3], f[j]);
            hi = encode4<E5M2>(v[4], v[5], v[6], v[7], f[j]);
        }
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

template <bool BF16, bool E5M2>
hif4_status launch_quant(F8QuantArgs &a, bool square, cudaStream_t s)
{
    const int64_t cblk = a.nblk;
    if (!square && !a.qt) {
        const int64_t items = (a.rows + kRowsPerCta - 1) / kRowsPerCta * cblk;
        a.items = (uint32_t)items;
        const void *k = reinterpret_cast<const void *>(k_f8_rows<BF16, E5M2>);
        const int64_t most = 8 * (int64_t)sm_count() * blocks_per_sm(k, kThreads, 0);
        return launch_pdl(k_f8_rows<BF16, E5M2>, dim3((unsigned)(items < most ? items : most)), dim3(kThreads), 0, s,
                          a);
    }
    const dim3 grid((unsigned)(f8::blocks_of(a.rows) * cblk));
    return square ? launch_pdl(k_f8_tile<BF16, true, E5M2>, grid, dim3(kThreads), 0, s, a)
                  : launch_pdl(k_f8_tile<BF16, false, E5M2>, grid, dim3(kThreads), 0, s, a);
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
    a.status = status;
    a.fmax = f8::fmt_max(fmt);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == HIF4_BF16)
        return fmt == HIF4_E5M2 ? launch_quant<true, true>(a, square, s) : launch_quant<true, false>(a, square, s);
    return fmt == HIF4_E5M2 ? launch_quant<false, true>(a, square, s) : launch_quant<false, false>(a, square, s);
}
