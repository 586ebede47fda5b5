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
    return __fdiv_rn(fmaxf(__uint_as_float(amax_bits), AMAX_FLOOR), E4M3_MAX);
}

// A number that rounds to the same e4m3 value as the real quotient x / s,
// given y = RN(1 / s).  RN(x / s) itself would not do: a quotient just beside
// the middle of two e4m3 values can round onto it in fp32 and then go to the
// even neighbour instead of the nearer one, and for 16-bit x that is common (s
// is the rounded ratio of one of them to 448, so x / s sits beside a middle
// whenever 448 x / amax is one: about one value in 250).  So a quotient with
// at most five leading bits is moved by its remainder, scaled up to at least
// one unit in the last place: the remainder of a quotient that is not exactly a
// middle is at least 2^-29 of it (24-bit x against 24 + 5 bits), and 2^8 times
// the remainder is at least 2^-21 and at most 2^-15 of it, far from the next
// middle (2^-5).  Needs x and s far enough from 2^-126 for exact remainders.
__device__ __forceinline__ float quotient(float x, float s, float y) {
    float q = div_by_recip(x, s, y);
    if ((__float_as_uint(q) & 0x7FFFFu) == 0u)
        q = copysignf(__fmaf_rn(__fmul_rn(__fmaf_rn(-q, s, x), 256.0f), y, q), x);   // -0 stays -0
    return q;
}

// Two e4m3 codes, `lo` in the low byte: round to nearest even, at most 448.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Four codes of four values of a block with scale s, y = RN(1 / s).  x y is
// within two units in the last place of x / s, so unless one of the four lies
// within four of a number of at most five leading bits (the middles among
// them), rounding x y gives the codes.
__device__ __forceinline__ uint32_t codes4(const float* v, float s, float y) {
    float q[4];
    uint32_t near = ~0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        q[i] = __fmul_rn(v[i], y);
        near = min(near, (__float_as_uint(q[i]) + 4u) & 0x7FFF8u);
    }
    if (near == 0u) {
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = quotient(v[i], s, y);
    }
    return e4m3x2(q[0], q[1]) | (e4m3x2(q[2], q[3]) << 16);
}

// Blocks whose scale is below this take their values and scale times
// SMALL_LIFT first, exactly, so that the remainders in quotient() are exact.
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

// Eight consecutive values at a 16-byte aligned address.
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void load8(const __half* p, float (&v)[8]) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

}  // namespace fp8
}  // namespace gptq
