// e4m3 codes and fp32 block scales of activations (1 x 128 blocks, a scale per
// token and 128 input channels) and of weights (128 x 128 blocks).
//
//   a = max |x| over the block;  s = RN(max(a, 2^-90) / 448);
//   c = x / s rounded once to e4m3 (half to even), at most 448.
//
// One pass: a block's values stay in registers between its maximum and its
// codes, so each value is read once and one byte is written for it.  The
// bound is HBM: 3 bytes a value (bf16) or 5 (fp32).  Measured: rows 8192 x 11008
// bf16 53 us (5.1 TB/s; 103 with a division per value, 74 with a branch for the
// quotients next to a middle), fp32 69 us (6.6 TB/s); weight 8192 x 28672 bf16 131
// us (5.4 TB/s), fp32 195: reads and writes mixed, and in 16 bits the coder's issue
// slots behind them.
//
// That is for rows on 16-byte boundaries of at least a warp's 1024 channels.  The
// forms for any alignment are right but far from HBM: rows 8192 x 11008 at an odd
// pitch 127 us in bf16 and 105 in fp32, a weight of 3021 x 22881 bf16 327 us (22880
// columns, aligned: 43) and fp32 79.  Of rows of 128 channels seven eighths of
// a warp's loads are empty: 65536 of them in bf16 take 33 us, 8 times their bytes'.
#include "fp8.cuh"
#include "kernels.h"

namespace gptq {
namespace fp8 {

constexpr int WARPS = 8;              // warps of a block, one token row each
constexpr int UNROLL = 4;             // 256-value steps of a warp in flight
constexpr int CHUNK = 256 * UNROLL;   // values of a row one warp takes

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// The codes of a block: its values and scale are lifted together where the scale is small.
struct BlockCoder {
    bool small;
    Coder code;
    __device__ __forceinline__ explicit BlockCoder(float scale)
        : small(scale < SMALL_SCALE),
          code(small ? scale * SMALL_LIFT : scale, rcp_approx(small ? scale * SMALL_LIFT : scale)) {}
    template <int N>
    __device__ __forceinline__ void lift(float (&v)[N]) const {
        if (small) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] *= SMALL_LIFT;
        }
    }
    // four codes whose values' signs lie in bit 7 of each byte of `signs`
    __device__ __forceinline__ uint32_t four(const float* v, uint32_t signs) const {
        const uint32_t c = code.two(pack2(v[0], v[1])) | (code.two(pack2(v[2], v[3])) << 16);
        return (c & 0x7F7F7F7Fu) | (signs & 0x80808080u);
    }
    template <typename T>
    __device__ __forceinline__ uint2 eight(const Raw8<T>& raw) const {
        float v[8];
        widen8(raw, v);
        lift(v);
        if constexpr (sizeof(T) == 4)
            return make_uint2(code.four(v), code.four(v + 4));
        else   // the high bytes of the 16-bit values hold the signs
            return make_uint2(four(v, __byte_perm(raw.w[0], raw.w[1], 0x7531)),
                              four(v + 4, __byte_perm(raw.w[2], raw.w[3], 0x7531)));
    }
};
__device__ __forceinline__ void store8(uint8_t* out, uint2 c, int64_t n) {
    if (n >= 8) {
        *reinterpret_cast<uint2*>(out) = c;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) out[i] = uint8_t((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
    }
}

// The maxima over each half warp of UNROLL values of top8(), two 16-bit ones to a word.
template <typename T>
__device__ __forceinline__ void half_warp_tops(uint32_t (&a)[UNROLL]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int u = 0; u < UNROLL; ++u)
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) a[u] = max(a[u], __shfl_xor_sync(0xFFFFFFFFu, a[u], o));
    } else {
#pragma unroll
        for (int u = 0; u < UNROLL; u += 2) {
            uint32_t p = __vmaxu2(__byte_perm(a[u], a[u + 1], 0x5410), __byte_perm(a[u], a[u + 1], 0x7632));
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) p = __vmaxu2(p, __shfl_xor_sync(0xFFFFFFFFu, p, o));
            a[u] = p & 0xFFFFu;
            a[u + 1] = p >> 16;
        }
    }
}

// Rows, aligned: 16 lanes hold one block, 8 values a lane, so a block's
// maximum is four shuffles and its codes leave as 8-byte stores.  A warp has
// eight blocks in flight; one lane each computes their scales.
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
    Raw8<T> v[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        const int64_t k = k0 + u * 256;
        v[u] = k + 8 <= d ? load_raw8(xr + k) : load_some8(xr + k, d - k);
    }
    uint32_t a[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) a[u] = top8(v[u]);
    half_warp_tops<T>(a);
    const int mine = lane & (UNROLL - 1);
    uint32_t own = a[0];
#pragma unroll
    for (int u = 1; u < UNROLL; ++u) own = mine == u ? a[u] : own;
    own = top_bits<T>(own);
    const float scale = block_scale(own);
    const int64_t block = (k0 - (lane & 15) * 8 + mine * 256) / BLOCK;
    if ((lane & 15) < UNROLL && block * BLOCK < d) {
        scales[block * lds + row] = scale;
        if (own >= INF_BITS) record_error(st, GPTQ_ERR_NONFINITE, int(row));
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        const int64_t k = k0 + u * 256;
        const BlockCoder c(__shfl_sync(0xFFFFFFFFu, scale, (lane & 16) + u));
        if (k < d) store8(codes + row * ldc + k, c.eight(v[u]), d - k);
    }
}

// Rows at any alignment: a warp takes whole blocks, lane l the values l, l + 32,
// l + 64 and l + 96 of each: a warp's loads and stores are contiguous, but of one
// value a lane, and the codes leave a byte at a time.
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
        const float scale = block_scale(a);
        if (lane == 0) {
            scales[(kb / BLOCK) * lds + row] = scale;
            if (a >= INF_BITS) record_error(st, GPTQ_ERR_NONFINITE, int(row));
        }
        const BlockCoder coder(scale);
        coder.lift(v[b]);
        const uint32_t c = coder.code.four(v[b]);
        uint8_t* out = codes + row * ldc + kb + lane;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (kb + lane + 32 * i < d) out[32 * i] = uint8_t(c >> (8 * i));
    }
}

// A 128 x 128 block of a weight per thread block, aligned: thread t holds 8
// consecutive columns (t % 16) of every sixteenth row.
template <typename T>
__global__ void __launch_bounds__(256)
    quant_weight_kernel(const T* __restrict__ w, int64_t n, int64_t d, int64_t ldw, uint8_t* __restrict__ codes,
                        int64_t ldc, float* __restrict__ scales, int nb, DevStatus* st) {
    __shared__ uint32_t part[8];
    pdl_wait();
    pdl_trigger();
    const int64_t bn = blockIdx.x / nb, bk = blockIdx.x % nb;
    const int t = threadIdx.x;
    const int64_t r0 = bn * BLOCK + t / 16, k = bk * BLOCK + (t % 16) * 8;
    Raw8<T> v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = r0 + i * 16;
        v[i] = r < n && k + 8 <= d ? load_raw8(w + r * ldw + k) : load_some8(w + r * ldw + k, r < n ? d - k : 0);
    }
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t b = top8(v[i]);
        a = sizeof(T) == 4 ? max(a, b) : __vmaxu2(a, b);
    }
    if (sizeof(T) != 4) a = max(a & 0xFFFFu, a >> 16);
    a = __reduce_max_sync(0xFFFFFFFFu, a);
    if ((t & 31) == 0) part[t / 32] = a;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) a = max(a, part[i]);
    a = top_bits<T>(a);
    const float scale = block_scale(a);
    if (t == 0) {
        scales[bn * nb + bk] = scale;
        if (a >= INF_BITS) record_error(st, GPTQ_ERR_NONFINITE, int(bn * BLOCK));
    }
    const BlockCoder c(scale);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = r0 + i * 16;
        if (r >= n || k >= d) break;
        store8(codes + r * ldc + k, c.eight(v[i]), d - k);
    }
}

// The same at any alignment: columns lane, lane + 32, ... of every eighth row, one
// value a load and one byte a store.
template <typename T>
__global__ void __launch_bounds__(256)
    quant_weight_any_kernel(const T* __restrict__ w, int64_t n, int64_t d, int64_t ldw, uint8_t* __restrict__ codes,
                            int64_t ldc, float* __restrict__ scales, int nb, DevStatus* st) {
    __shared__ uint32_t part[8];
    pdl_wait();
    pdl_trigger();
    const int64_t bn = blockIdx.x / nb, bk = blockIdx.x % nb;
    const int t = threadIdx.x, lane = t & 31;
    const int64_t r0 = bn * BLOCK + t / 32, c0 = bk * BLOCK + lane;
    float v[16][4];
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t r = r0 + i * 8, c = c0 + j * 32;
            v[i][j] = r < n && c < d ? to_f32(w[r * ldw + c]) : 0.0f;
            a = max(a, abs_bits(v[i][j]));
        }
    a = __reduce_max_sync(0xFFFFFFFFu, a);
    if (lane == 0) part[t / 32] = a;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) a = max(a, part[i]);
    const float scale = block_scale(a);
    if (t == 0) {
        scales[bn * nb + bk] = scale;
        if (a >= INF_BITS) record_error(st, GPTQ_ERR_NONFINITE, int(bn * BLOCK));
    }
    const BlockCoder coder(scale);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int64_t r = r0 + i * 8;
        if (r >= n) break;
        coder.lift(v[i]);
        const uint32_t c = coder.code.four(v[i]);
        uint8_t* out = codes + r * ldc + c0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (c0 + 32 * j < d) out[32 * j] = uint8_t(c >> (8 * j));
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
    auto kernel = aligned_for<T>(w, ldw, codes) ? quant_weight_kernel<T> : quant_weight_any_kernel<T>;
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
