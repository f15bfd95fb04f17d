// hif4_f8.cuh — device helpers of the block-scaled FP8 operators: granule
// loads and stores of BF16 / FP32 rows, the scale pair of a 128-block and the
// conversion to FP8 codes.
//
// A block's scale and its encoding factor, from its largest magnitude a
// (raised to 2^-100, so that neither quotient overflows or is subnormal):
//   s = fl32(a / F),  r = fl32(F / a),  q = RNE_f8(fl32(x r)),
// F the largest finite value of the format (448 for E4M3, 57344 for E5M2).
// Both quotients are correctly rounded, and |x r| <= F (1 + 2^-23), which the
// saturating conversion takes to F.  x r is rounded to FP32 before the
// conversion; that product, not a quotient per element, is the definition,
// since a division per element would cost more than the whole kernel.
#pragma once

#include <cuda_bf16.h>

#include "hif4_internal.cuh"

namespace hif4 {
namespace f8 {

constexpr int BLK = 128;                       // elements per scale block
constexpr float kTiny = 7.888609052210118e-31f; // 2^-100

__host__ __device__ constexpr float fmt_max(int fmt) { return fmt == HIF4_E5M2 ? 57344.0f : 448.0f; }

// One of the two, from the bits of the maximum: a warp forms both in one go, the
// scale in some lanes and the factor in others.  Either quotient
// takes about as long as encoding eight elements.
__device__ __forceinline__ float scale_or_factor(uint32_t amax_bits, float fmax, bool scale)
{
    const float a = fmaxf(bits_f(amax_bits), kTiny);
    return __fdiv_rn(scale ? a : fmax, scale ? fmax : a);
}

// Two codes, lo in the low byte (round to nearest even, saturating).
template <bool E5M2>
__device__ __forceinline__ uint32_t cvt2(float lo, float hi)
{
    uint16_t r;
    if (E5M2)
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Codes of a f and b f (one packed FP32 product).
template <bool E5M2>
__device__ __forceinline__ uint32_t encode2(float a, float b, float f)
{
    float x, y;
    asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %4};\n\t"
        "mul.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
        : "=f"(x), "=f"(y)
        : "f"(a), "f"(b), "f"(f));
    return cvt2<E5M2>(x, y);
}

template <bool E5M2>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, float f)
{
    return encode2<E5M2>(a, b, f) | encode2<E5M2>(c, d, f) << 16;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// NaN -> 0, +-Inf -> +-FLT_MAX over a granule; *bad set when it did.  One test
// of the largest magnitude word covers the ordinary case.
template <int N>
__device__ __forceinline__ void sanitize_all(float (&v)[N], uint32_t &bad)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) m = max(m, f_bits(v[i]) & 0x7FFFFFFFu);
    if (m >= 0x7F800000u) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = sanitize(v[i], bad);
    }
}

// One granule = 8 consecutive elements of a row, raw: one 16-byte vector of
// BF16, two of FP32.
template <bool BF16>
struct Raw8 {
    uint4 w[BF16 ? 1 : 2];
};

// Granule at element `off` of a 16-byte aligned row; the elements from
// `valid` on (0..8) read as 0 and are not touched in memory.
template <bool BF16>
__device__ __forceinline__ Raw8<BF16> load_raw8(const void *base, int64_t off, int valid)
{
    Raw8<BF16> r;
    if (valid >= 8) {
        if (BF16) {
            r.w[0] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + off));
        } else {
            const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const float *>(base) + off);
            r.w[0] = __ldcs(p);
            r.w[BF16 ? 0 : 1] = __ldcs(p + 1);
        }
    } else {
        uint32_t e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            e[i] = 0;
            if (i < valid)
                e[i] = BF16 ? (uint32_t)(static_cast<const uint16_t *>(base)[off + i])
                            : (static_cast<const uint32_t *>(base)[off + i]);
        }
        if (BF16) {
            r.w[0] = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
        } else {
            r.w[0] = make_uint4(e[0], e[1], e[2], e[3]);
            r.w[BF16 ? 0 : 1] = make_uint4(e[4], e[5], e[6], e[7]);
        }
    }
    return r;
}

template <bool BF16>
__device__ __forceinline__ void widen8(const Raw8<BF16> &r, float (&v)[8])
{
    if (BF16) {
        const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_lo(w[i]);
            v[2 * i + 1] = bf16_hi(w[i]);
        }
    } else {
        const uint4 a = r.w[0], b = r.w[BF16 ? 0 : 1];
        v[0] = bits_f(a.x); v[1] = bits_f(a.y); v[2] = bits_f(a.z); v[3] = bits_f(a.w);
        v[4] = bits_f(b.x); v[5] = bits_f(b.y); v[6] = bits_f(b.z); v[7] = bits_f(b.w);
    }
}

__device__ __forceinline__ uint32_t pack_bf16_rn(float lo, float hi)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Stores the first `valid` of 8 values at element `off` (BF16 by round to
// nearest even, or FP32).
template <bool BF16>
__device__ __forceinline__ void store8(void *base, int64_t off, const float (&v)[8], int valid)
{
    if (BF16) {
        uint16_t *p = static_cast<uint16_t *>(base) + off;
        const uint4 w = make_uint4(pack_bf16_rn(v[0], v[1]), pack_bf16_rn(v[2], v[3]), pack_bf16_rn(v[4], v[5]),
                                   pack_bf16_rn(v[6], v[7]));
        if (valid >= 8) {
            *reinterpret_cast<uint4 *>(p) = w;
        } else {
            const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < valid) p[i] = (uint16_t)(a[i >> 1] >> (16 * (i & 1)));
        }
    } else {
        float *p = static_cast<float *>(base) + off;
        if (valid >= 8) {
            reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < valid) p[i] = v[i];
        }
    }
}

// The first `valid` of 8 code bytes at p (8-byte aligned).
__device__ __forceinline__ void store_codes8(uint8_t *p, uint32_t lo, uint32_t hi, int valid)
{
    if (valid >= 8) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(lo, hi);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < valid) p[i] = (uint8_t)((i < 4 ? lo : hi) >> (8 * (i & 3)));
    }
}

// Bits of the largest magnitude of a granule (as FP32; NaN above Inf above
// every finite value).  BF16: on pairs of 15-bit keys.
template <bool BF16>
__device__ __forceinline__ uint32_t amax_bits(const Raw8<BF16> &r)
{
    if (BF16) {
        const uint32_t m = max_u16x2(max_u16x2(r.w[0].x & 0x7FFF7FFFu, r.w[0].y & 0x7FFF7FFFu),
                                     max_u16x2(r.w[0].z & 0x7FFF7FFFu, r.w[0].w & 0x7FFF7FFFu));
        return max(m << 16, m & 0xFFFF0000u);
    }
    const uint4 a = r.w[0], b = r.w[BF16 ? 0 : 1];
    return max(max(max(a.x & 0x7FFFFFFFu, a.y & 0x7FFFFFFFu), max(a.z & 0x7FFFFFFFu, a.w & 0x7FFFFFFFu)),
               max(max(b.x & 0x7FFFFFFFu, b.y & 0x7FFFFFFFu), max(b.z & 0x7FFFFFFFu, b.w & 0x7FFFFFFFu)));
}

__device__ __forceinline__ uint32_t amax_bits(const float (&v)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, f_bits(v[i]) & 0x7FFFFFFFu);
    return m;
}

// Largest magnitude, NaN if there is one.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float amax8_nan(const float (&v)[8])
{
    return max_nan(max_nan(max_nan(fabsf(v[0]), fabsf(v[1])), max_nan(fabsf(v[2]), fabsf(v[3]))),
                   max_nan(max_nan(fabsf(v[4]), fabsf(v[5])), max_nan(fabsf(v[6]), fabsf(v[7]))));
}

constexpr uint32_t kInfBits = 0x7F800000u;

inline bool valid_fmt(int fmt) { return fmt == HIF4_E4M3 || fmt == HIF4_E5M2; }
inline int64_t blocks_of(int64_t n) { return (n + BLK - 1) / BLK; }

} // namespace f8
} // namespace hif4
