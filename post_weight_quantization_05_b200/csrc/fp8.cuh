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

// Codes of the real quotients x / s, rounded once.
//
// q = x y with y = rcp_approx(s) is within three units in the last place of
// x / s (2^-23 of y's error, 2^-24 of the product's), so it rounds to the same
// code unless a middle of two codes lies that near.  Middles have at most five
// significant bits: q is near one when adding 4 leaves bits 3 .. 18 zero.
// For 16-bit x that is common -- s is the rounded 1 / 448 of one of them, so
// x / s sits just beside a middle whenever 448 x / amax is one, about one value in
// 250 -- and rounding x / s to fp32 first would be as wrong as q.  Such a q is
// replaced by its middle t moved by the remainder x - t s (exact in one fused
// multiply-add: 29 bits of t s against at most 24 of x).  256 times the
// remainder is at least 2^-21 of t if it is not zero, and at most 2^-13, far
// from the next middle (2^-5): the code is the nearer one, and an exact middle
// goes to the even one.  Needs x and s far enough above 2^-126 (SMALL_SCALE).
__device__ __forceinline__ bool near_middle(float q) { return ((__float_as_uint(q) + 4u) & 0x7FFF8u) == 0u; }
__device__ __forceinline__ float settle(float q, float x, float s, float y) {
    const float t = __uint_as_float((__float_as_uint(q) + 4u) & ~7u);
    const float r = __fmaf_rn(-t, s, x);
    return near_middle(q) ? copysignf(__fmaf_rn(r, 256.0f * y, t), x) : q;   // -0 stays -0
}
__device__ __forceinline__ uint32_t code1(float x, float s, float y) {
    return e4m3x2(settle(__fmul_rn(x, y), x, s, y), 0.0f);
}
__device__ __forceinline__ uint32_t codes4(const float* v, float s, float y) {
    float q[4];
    bool near = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        q[i] = __fmul_rn(v[i], y);
        near |= near_middle(q[i]);
    }
    if (near) {
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = settle(q[i], v[i], s, y);
    }
    return e4m3x2(q[0], q[1]) | (e4m3x2(q[2], q[3]) << 16);
}

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
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) { widen8(load_raw8(p), v); }
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) { widen8(load_raw8(p), v); }
__device__ __forceinline__ void load8(const __half* p, float (&v)[8]) { widen8(load_raw8(p), v); }

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
