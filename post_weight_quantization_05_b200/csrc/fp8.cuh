// e4m3 values with one fp32 scale per block of 128: the scale of a block, the
// code of a value, and loads and stores of the element types around them.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace gptq {
namespace fp8 {

constexpr int BLOCK = 128;               // values per scale along a row
constexpr float E4M3_MAX = 448.0f;       // the largest finite e4m3 value, 1.75 * 2^8
constexpr float AMAX_FLOOR = 0x1p-90f;   // keeps the scale of a block of zeros positive and normal
constexpr uint32_t INF_BITS = 0x7F800000u;

// The scale of a block whose largest magnitude has the fp32 bits `amax_bits`
// (NaN if the block holds a NaN or an infinity).
__device__ __forceinline__ float block_scale(uint32_t amax_bits) {
    if (amax_bits >= INF_BITS) return __uint_as_float(0x7FC00000u);
    return div_by_recip(fmaxf(__uint_as_float(amax_bits), AMAX_FLOOR), E4M3_MAX, 1.0f / E4M3_MAX);
}

__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two e4m3 codes, `lo` in the low byte: round to nearest even, at most 448.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two fp32 values in one 64-bit register, and arithmetic on both at once.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// Codes of the real quotients x / s, rounded once, without a division or a
// branch.
//
// Rounding x y, y = rcp_approx(s), or even RN(x / s), can go wrong where the
// quotient lies beside the middle of two codes, and for 16-bit x that is
// common: s is the rounded 1 / 448 of one of them, so x / s is just beside a
// middle whenever 448 x / amax is one, about one value in 250.  Codes have four
// significant bits and middles five, so:
//   h = x y rounded to five bits (Veltkamp's splitting: c = (2^19 + 1) q,
//       h = c - (c - q)), the five-bit number nearest x / s up to an error far
//       below half their spacing;
//   r = x - h s in one fused multiply-add, whose sign is exact.
// If h is a code, it is the answer, and if it is a middle, the sign of r
// decides, or the even code where r = 0.  Either way the answer is h moved by
// 2^-15 towards r's sign and rounded to four bits: 2^-15 is one unit in the
// last place of 448, and smaller than the spacing of five-bit numbers from
// 2^-10, the smallest middle, up.  (Just below 2^-10 the move may end on that
// middle, which rounds to the even 0 as it should.)  r y 2^40 saturated to
// [-1/2, 1/2] is the sign: a remainder that is not zero is at least 2^-29 of h s
// (29 bits of h s against 24 of x).  The sign of a zero code is x's.
// Needs x and s far enough above 2^-126 (SMALL_SCALE).
struct Coder {
    uint64_t y, minus_s;
    float sign_scale;
    __device__ __forceinline__ Coder(float s, float r) : y(pack2(r, r)), minus_s(pack2(-s, -s)), sign_scale(0x1p40f * r) {}
    // codes of the two values of x, the first in the low byte, sign bits to be set by the caller
    __device__ __forceinline__ uint32_t two(uint64_t x) const {
        const uint64_t minus1 = pack2(-1.0f, -1.0f);
        const uint64_t q = mul2(x, y), c = mul2(q, pack2(0x1p19f + 1.0f, 0x1p19f + 1.0f));
        const uint64_t h = fma2(fma2(q, minus1, c), minus1, c);
        float ra, rb, a, b;
        unpack2(fma2(h, minus_s, x), ra, rb);
        asm("fma.rn.sat.f32 %0, %1, %2, 0f3F000000;" : "=f"(a) : "f"(ra), "f"(sign_scale));   // 0, 1/2 or 1
        asm("fma.rn.sat.f32 %0, %1, %2, 0f3F000000;" : "=f"(b) : "f"(rb), "f"(sign_scale));
        const uint64_t low = add2(h, pack2(-0x1p-15f, -0x1p-15f));
        unpack2(fma2(pack2(a, b), pack2(0x1p-14f, 0x1p-14f), low), a, b);
        return e4m3x2(a, b);
    }
    __device__ __forceinline__ uint32_t four(const float* v) const {
        const uint32_t signs = __byte_perm(__byte_perm(__float_as_uint(v[0]), __float_as_uint(v[1]), 0x0073),
                                           __byte_perm(__float_as_uint(v[2]), __float_as_uint(v[3]), 0x0073), 0x5410);
        const uint32_t codes = two(pack2(v[0], v[1])) | (two(pack2(v[2], v[3])) << 16);
        return (codes & 0x7F7F7F7Fu) | (signs & 0x80808080u);
    }
    __device__ __forceinline__ uint32_t one(float v) const {
        return (two(pack2(v, v)) & 0x7Fu) | (__float_as_uint(v) >> 31 << 7);
    }
};

// Blocks whose scale is below this take their values and scale times
// SMALL_LIFT first, exactly, so that the remainders above are exact.
constexpr float SMALL_SCALE = 0x1p-40f;
constexpr float SMALL_LIFT = 0x1p64f;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// Eight consecutive values as they lie in memory.
template <typename T>
struct Raw8 {
    uint32_t w[2 * sizeof(T)];
};
template <typename T>
__device__ __forceinline__ Raw8<T> load_raw8(const T* p) {   // 16-byte aligned
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < int(sizeof(T)) / 2; ++i) {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(p) + i);
        r.w[4 * i] = a.x; r.w[4 * i + 1] = a.y; r.w[4 * i + 2] = a.z; r.w[4 * i + 3] = a.w;
    }
    return r;
}
__device__ __forceinline__ uint32_t raw_bits(float v) { return __float_as_uint(v); }
__device__ __forceinline__ uint32_t raw_bits(__nv_bfloat16 v) { return __bfloat16_as_ushort(v); }
__device__ __forceinline__ uint32_t raw_bits(__half v) { return __half_as_ushort(v); }
template <typename T>
__device__ __forceinline__ Raw8<T> load_some8(const T* p, int64_t n) {   // the first n, zeros behind them
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < int(2 * sizeof(T)); ++i) {
        if constexpr (sizeof(T) == 4)
            r.w[i] = i < n ? raw_bits(p[i]) : 0u;
        else
            r.w[i] = (2 * i < n ? raw_bits(p[2 * i]) : 0u) | (2 * i + 1 < n ? raw_bits(p[2 * i + 1]) << 16 : 0u);
    }
    return r;
}
__device__ __forceinline__ void widen8(const Raw8<float>& r, float* v) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r.w[i]);
}
__device__ __forceinline__ void widen8(const Raw8<__nv_bfloat16>& r, float* v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(r.w[i] << 16);
        v[2 * i + 1] = __uint_as_float(r.w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void widen8(const Raw8<__half>& r, float* v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r.w[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

// The largest magnitude of eight values in the type's own bits (16-bit types:
// one in each half of the word, to be joined by top_of), and as fp32 bits.
__device__ __forceinline__ uint32_t top8(const Raw8<float>& r) {
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = max(a, r.w[i] & 0x7FFFFFFFu);
    return a;
}
template <typename T>
__device__ __forceinline__ uint32_t top8(const Raw8<T>& r) {
    return __vmaxu2(__vmaxu2(r.w[0] & 0x7FFF7FFFu, r.w[1] & 0x7FFF7FFFu),
                    __vmaxu2(r.w[2] & 0x7FFF7FFFu, r.w[3] & 0x7FFF7FFFu));
}
template <typename T>
__device__ __forceinline__ uint32_t top_bits(uint32_t a);   // a 16-bit magnitude, or fp32 bits
template <>
__device__ __forceinline__ uint32_t top_bits<float>(uint32_t a) { return a; }
template <>
__device__ __forceinline__ uint32_t top_bits<__nv_bfloat16>(uint32_t a) { return a << 16; }
template <>
__device__ __forceinline__ uint32_t top_bits<__half>(uint32_t a) {
    return __float_as_uint(__half2float(__ushort_as_half(uint16_t(a))));
}

}  // namespace fp8
}  // namespace gptq
