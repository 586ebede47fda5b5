// e4m3 codes and fp32 block scales of activations (1 x 128 blocks, a scale per
// token and 128 input channels) and of weights (128 x 128 blocks).
//
//   a = max |x| over the block;  s = RN(max(a, 2^-90) / 448);
//   c = x / s rounded once to e4m3 (half to even), at most 448.
//
// One pass: a block's values stay in registers between its maximum and its
// codes, so each value is read once and one byte is written for it.  The
// bound is HBM: 3 bytes a value (bf16) or 5 (fp32).
#include "fp8.cuh"
#include "kernels.h"

namespace gptq {
namespace fp8 {

constexpr int WARPS = 8;              // warps of a block, one token row each
constexpr int UNROLL = 4;             // 256-value steps of a warp in flight
constexpr int CHUNK = 256 * UNROLL;   // values of a row one warp takes

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Rows, aligned: 16 lanes hold one block, 8 values a lane, so a block's
// maximum is four shuffles and its codes leave as 8-byte stores.
template <typename T>
__global__ void __launch_bounds__(32 * WARPS)
    quant_rows_kernel(const T* __restrict__ x, int64_t m, int64_t d, int64_t ldx, uint8_t* __restrict__ codes,
                      int64_t ldc, float* __restrict__ scales, int64_t lds, int chunks, DevStatus* st) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t row = int64_t(blockIdx.x / chunks) * WARPS + (threadIdx.x >> 5);
    const int64_t k0 = int64_t(blockIdx.x % chunks) * CHUNK + lane * 8;
    if (row >= m) return;
    const T* xr = x + row * ldx;
    float v[UNROLL][8];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        const int64_t k = k0 + u * 256;
        if (k + 8 <= d) {
            load8(xr + k, v[u]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[u][i] = k + i < d ? to_f32(xr[k + i]) : 0.0f;
        }
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        const int64_t k = k0 + u * 256;
        uint32_t a = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) a = max(a, abs_bits(v[u][i]));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
        if (k - (lane & 15) * 8 >= d) continue;             // the block lies behind the row's end
        float s = block_scale(a);
        if ((lane & 15) == 0) {
            scales[(k / BLOCK) * lds + row] = s;
            if (a >= INF_BITS) record_error(st, GPTQ_ERR_NONFINITE, int(min(row, int64_t(0x7FFFFFFF))));
        }
        if (s < SMALL_SCALE) {
            s *= SMALL_LIFT;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[u][i] *= SMALL_LIFT;
        }
        const float y = __frcp_rn(s);
        const uint2 c = make_uint2(codes4(v[u], s, y), codes4(v[u] + 4, s, y));
        uint8_t* out = codes + row * ldc + k;
        if (k + 8 <= d) {
            *reinterpret_cast<uint2*>(out) = c;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (k + i < d) out[i] = uint8_t((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
        }
    }
}

// Rows at any alignment: a warp takes whole blocks, lane l the values l, l + 32,
// l + 64 and l + 96 of each, so loads and byte stores are still contiguous.
template <typename T>
__global__ void __launch_bounds__(32 * WARPS)
    quant_rows_any_kernel(const T* __restrict__ x, int64_t m, int64_t d, int64_t ldx, uint8_t* __restrict__ codes,
                          int64_t ldc, float* __restrict__ scales, int64_t lds, int chunks, DevStatus* st) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t row = int64_t(blockIdx.x / chunks) * WARPS + (threadIdx.x >> 5);
    const int64_t k0 = int64_t(blockIdx.x % chunks) * CHUNK + lane;
    if (row >= m) return;
    const T* xr = x + row * ldx;
    constexpr int BLOCKS = CHUNK / BLOCK;
    float v[BLOCKS][4];
#pragma unroll
    for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t k = k0 + b * BLOCK + 32 * i;
            v[b][i] = k < d ? to_f32(xr[k]) : 0.0f;
        }
#pragma unroll
    for (int b = 0; b < BLOCKS; ++b) {
        const int64_t kb = k0 - lane + b * BLOCK;
        if (kb >= d) break;
        uint32_t a = max(max(abs_bits(v[b][0]), abs_bits(v[b][1])), max(abs_bits(v[b][2]), abs_bits(v[b][3])));
        a = __reduce_max_sync(0xFFFFFFFFu, a);
        float s = block_scale(a);
        if (lane == 0) {
            scales[(kb / BLOCK) * lds + row] = s;
            if (a >= INF_BITS) record_error(st, GPTQ_ERR_NONFINITE, int(min(row, int64_t(0x7FFFFFFF))));
        }
        if (s < SMALL_SCALE) {
            s *= SMALL_LIFT;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[b][i] *= SMALL_LIFT;
        }
        const uint32_t c = codes4(v[b], s, __frcp_rn(s));
        uint8_t* out = codes + row * ldc + kb + lane;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (kb + lane + 32 * i < d) out[32 * i] = uint8_t(c >> (8 * i));
    }
}

// A 128 x 128 block of a weight per thread block, 64 values a thread in
// registers.  ALIGNED: thread t takes 8 consecutive columns (t % 16) of every
// sixteenth row; otherwise the columns lane, lane + 32, ... of every eighth.
template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(256)
    quant_weight_kernel(const T* __restrict__ w, int64_t n, int64_t d, int64_t ldw, uint8_t* __restrict__ codes,
                        int64_t ldc, float* __restrict__ scales, int nb, DevStatus* st) {
    __shared__ uint32_t part[8];
    pdl_wait();
    pdl_trigger();
    constexpr int ROWS = ALIGNED ? 8 : 16, COLS = 64 / ROWS;
    const int64_t bn = blockIdx.x / nb, bk = blockIdx.x % nb;
    const int t = threadIdx.x, lane = t & 31;
    const int64_t r0 = bn * BLOCK + (ALIGNED ? t / 16 : t / 32);
    const int64_t c0 = bk * BLOCK + (ALIGNED ? (t % 16) * 8 : lane);
    constexpr int RSTEP = ALIGNED ? 16 : 8, CSTEP = ALIGNED ? 1 : 32;
    float v[ROWS][COLS];
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int64_t r = r0 + i * RSTEP;
        if (ALIGNED && r < n && c0 + 8 <= d) {
            if constexpr (ALIGNED) load8(w + r * ldw + c0, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < COLS; ++j) {
                const int64_t c = c0 + j * CSTEP;
                v[i][j] = r < n && c < d ? to_f32(w[r * ldw + c]) : 0.0f;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
#pragma unroll
        for (int j = 0; j < COLS; ++j) a = max(a, abs_bits(v[i][j]));
    a = __reduce_max_sync(0xFFFFFFFFu, a);
    if (lane == 0) part[t / 32] = a;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) a = max(a, part[i]);
    float s = block_scale(a);
    if (t == 0) {
        scales[bn * nb + bk] = s;
        if (a >= INF_BITS) record_error(st, GPTQ_ERR_NONFINITE, int(bn * BLOCK));
    }
    const bool small = s < SMALL_SCALE;
    if (small) s *= SMALL_LIFT;
    const float y = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int64_t r = r0 + i * RSTEP;
        if (r >= n) break;
        if (small) {
#pragma unroll
            for (int j = 0; j < COLS; ++j) v[i][j] *= SMALL_LIFT;
        }
        uint8_t* out = codes + r * ldc + c0;
        if constexpr (ALIGNED) {
            const uint2 c = make_uint2(codes4(v[i], s, y), codes4(v[i] + 4, s, y));
            if (c0 + 8 <= d) {
                *reinterpret_cast<uint2*>(out) = c;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c0 + j < d) out[j] = uint8_t((j < 4 ? c.x : c.y) >> (8 * (j & 3)));
            }
        } else {
            const uint32_t c = codes4(v[i], s, y);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c0 + 32 * j < d) out[32 * j] = uint8_t(c >> (8 * j));
        }
    }
}

}  // namespace fp8

namespace {

template <typename T>
bool aligned_for(const void* x, int64_t ldx, const void* codes) {
    return (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && (ldx * int64_t(sizeof(T))) % 16 == 0 &&
           (reinterpret_cast<uintptr_t>(codes) & 15u) == 0;   // ldc is a multiple of 16 in every call
}

template <typename T>
int rows_of(const void* x, int64_t m, int64_t d, int64_t ldx, uint8_t* codes, int64_t ldc, float* scales,
            int64_t lds, cudaStream_t stream, DevStatus* st) {
    using namespace fp8;
    const int chunks = int((d + CHUNK - 1) / CHUNK);
    const dim3 grid(unsigned((m + WARPS - 1) / WARPS * chunks));
    const T* p = static_cast<const T*>(x);
    auto kernel = aligned_for<T>(x, ldx, codes) ? quant_rows_kernel<T> : quant_rows_any_kernel<T>;
    if (launch_pdl(kernel, grid, dim3(32 * WARPS), 0, stream, p, m, d, ldx, codes, ldc, scales, lds, chunks, st) !=
        cudaSuccess)
        return GPTQ_ERR_CUDA;
    count_launch();
    return GPTQ_OK;
}

template <typename T>
int weight_of(const void* w, int64_t n, int64_t d, int64_t ldw, uint8_t* codes, int64_t ldc, float* scales,
              cudaStream_t stream, DevStatus* st) {
    using namespace fp8;
    const int nb = int((d + BLOCK - 1) / BLOCK);
    const dim3 grid(unsigned((n + BLOCK - 1) / BLOCK * nb));
    auto kernel = aligned_for<T>(w, ldw, codes) ? quant_weight_kernel<T, true> : quant_weight_kernel<T, false>;
    if (launch_pdl(kernel, grid, dim3(256), 0, stream, static_cast<const T*>(w), n, d, ldw, codes, ldc, scales, nb,
                   st) != cudaSuccess)
        return GPTQ_ERR_CUDA;
    count_launch();
    return GPTQ_OK;
}

}  // namespace

int launch_fp8_quantize_rows(const void* x, int dtype, int64_t m, int64_t d, int64_t ldx, uint8_t* codes,
                             int64_t ldc, float* scales, int64_t lds, cudaStream_t stream, DevStatus* st) {
    if (dtype == GPTQ_F32) return rows_of<float>(x, m, d, ldx, codes, ldc, scales, lds, stream, st);
    if (dtype == GPTQ_BF16) return rows_of<__nv_bfloat16>(x, m, d, ldx, codes, ldc, scales, lds, stream, st);
    return rows_of<__half>(x, m, d, ldx, codes, ldc, scales, lds, stream, st);
}

int launch_fp8_quantize_weight(const void* w, int dtype, int64_t n, int64_t d, int64_t ldw, uint8_t* codes,
                               int64_t ldc, float* scales, cudaStream_t stream, DevStatus* st) {
    if (dtype == GPTQ_F32) return weight_of<float>(w, n, d, ldw, codes, ldc, scales, stream, st);
    if (dtype == GPTQ_BF16) return weight_of<__nv_bfloat16>(w, n, d, ldw, codes, ldc, scales, stream, st);
    return weight_of<__half>(w, n, d, ldw, codes, ldc, scales, stream, st);
}

}  // namespace gptq
