// Log probabilities of given tokens under rows of logits, the entropy of each
// row's distribution, and its k likeliest tokens.
//
//   M = max x;  S = sum e^(x - M);  T = sum e^(x - M) (x - M)
//   logp(v) = (x_v - M) - ln S;  entropy = ln S - T / S
//
// One pass over the logits: each thread keeps its own running (M, S, T), moved
// to a new maximum once per 32 values, and the block joins them at the end.
// The bound is HBM (each logit read once), so the k likeliest come out of the
// same pass: the threads' maxima are distinct elements of the row, so the k-th
// largest of a few of them (two per warp) is a threshold that at least k
// elements reach; only the threads whose maximum reaches it look at their
// elements again (L2 still holds the row), and the few that pass are ranked
// against each other by (value descending, index ascending).
//
// A row is one block's, or, when there are fewer rows than the GPU has room
// for, a cluster's: its blocks take turns in the row, and the first joins the
// sums and ranks the others' best through distributed shared memory.  The order
// of every sum is fixed: the same inputs give the same bits.
#include <atomic>

#include "fp8.cuh"
#include "kernels.h"

namespace gptq {
namespace lp {

constexpr int THREADS = 512, WARPS = THREADS / 32;
constexpr int MAX_TOP = 32;          // two maxima of each warp must be enough for the threshold
constexpr int MAX_SPLIT = 8;
constexpr int CAND = 1024;           // elements that reach the threshold, before the fallback
constexpr int BATCH = 32;            // values between two looks at the running maximum
constexpr float LOWEST = -3.402823466e38f;
constexpr float FAR = -1e30f;        // x - M from here on counts as this: e^FAR = 0, and 0 * FAR = 0
constexpr float LOG2E = 1.4426950408889634f;

struct Args {
    const void* logits;
    const int64_t* targets;
    int64_t n, vocab, ld;
    float *logp, *entropy, *top_logp;
    int32_t* top_ids;
    int top;
    DevStatus* st;
};

// fp32 values in an order-preserving map to unsigned (0: below every value).
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);   // -0 counts as +0
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
    return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ uint64_t key_of(float x, uint32_t index) {
    return (uint64_t(order_of(x)) << 32) | uint32_t(~index);
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

struct Sums {
    float m, s, t;
};
// The same sums about a larger maximum.
__device__ __forceinline__ void move_to(Sums& a, float m) {
    const float d = fmaxf(a.m - m, FAR), f = exp2_approx(d * LOG2E);
    a.t = f * fmaf(a.s, d, a.t);
    a.s *= f;
    a.m = m;
}
__device__ __forceinline__ void add_batch(Sums& a, const float (&x)[BATCH]) {
    float m = x[0];
#pragma unroll
    for (int i = 1; i < BATCH; ++i) m = fmaxf(m, x[i]);
    if (m > a.m) move_to(a, m);
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
        const float d = max_nan(x[i] - a.m, FAR), e = exp2_approx(d * LOG2E);
        a.s += e;
        a.t = fmaf(e, d, a.t);
    }
}

template <typename T, int E>
__device__ __forceinline__ void load_vec(const T* p, float* x) {
    if constexpr (E == 1) {
        x[0] = fp8::to_f32(__ldg(p));
    } else if constexpr (sizeof(T) == 4) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(p));
        x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else {
        float v[8];
        fp8::load8(p, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = v[i];
    }
}

// The elements of a row that one thread owns: every (THREADS * split)-th vector
// of E values from the first aligned one on, and at most one of the values
// before and behind those.
template <typename T, int E>
struct Mine {
    const T* row;
    int64_t head, nv, first, step;   // first aligned value, vectors, this thread's first and its step
    int64_t edge;                    // a value of its own outside the vectors, or -1
    __device__ __forceinline__ Mine(const T* r, int64_t vocab, uint32_t rank, uint32_t split) : row(r) {
        const uint32_t off = uint32_t(reinterpret_cast<uintptr_t>(r) & 15u);
        head = E == 1 ? 0 : min(vocab, int64_t(((16u - off) & 15u) / sizeof(T)));
        nv = (vocab - head) / E;
        first = int64_t(rank) * THREADS + threadIdx.x;
        step = int64_t(split) * THREADS;
        const int64_t tail = head + nv * E, t = threadIdx.x;
        edge = rank != 0 ? -1 : t < head ? t : tail + (t - head) < vocab ? tail + (t - head) : -1;
    }
    // f(value, index) for each of them
    template <typename F>
    __device__ __forceinline__ void each(F f) const {
        if (edge >= 0) f(fp8::to_f32(row[edge]), uint32_t(edge));
        for (int64_t v = first; v < nv; v += step) {
            float x[E];
            load_vec<T, E>(row + head + v * E, x);
#pragma unroll
            for (int i = 0; i < E; ++i) f(x[i], uint32_t(head + v * E + i));
        }
    }
};

__device__ __forceinline__ float ld_cluster_f32(const float* p, uint32_t rank) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapa_shared(p, rank)) : "memory");
    return v;
}
__device__ __forceinline__ uint64_t ld_cluster_u64(const uint64_t* p, uint32_t rank) {
    uint64_t v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(mapa_shared(p, rank)) : "memory");
    return v;
}

template <typename T, int E>
__global__ void __launch_bounds__(THREADS) logprobs_kernel(const Args g) {
    __shared__ uint64_t cand[CAND];
    __shared__ uint64_t best[MAX_TOP];
    __shared__ float red[3][WARPS];
    __shared__ float total[3];             // M, S, T of this block's share
    __shared__ uint32_t tops[2 * WARPS];   // the two largest thread maxima of each warp
    __shared__ uint64_t wkey[WARPS];
    __shared__ int count;
    constexpr uint32_t ALL = 0xFFFFFFFFu;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t split;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(split));
    const uint32_t rank = cluster_ctarank();
    const int64_t row = blockIdx.x / split;
    pdl_wait();
    pdl_trigger();
    const T* x0 = static_cast<const T*>(g.logits) + row * g.ld;
    const Mine<T, E> mine(x0, g.vocab, rank, split);

    // ---------------- the pass
    Sums a{LOWEST, 0.0f, 0.0f};
    constexpr int U = BATCH / E;
    constexpr float NONE = -INFINITY;
    for (int64_t v = mine.first; v < mine.nv; v += U * mine.step) {
        float x[BATCH];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (v + u * mine.step < mine.nv) {
                load_vec<T, E>(mine.row + mine.head + (v + u * mine.step) * E, x + u * E);
            } else {
#pragma unroll
                for (int i = 0; i < E; ++i) x[u * E + i] = NONE;
            }
        }
        add_batch(a, x);
    }
    if (mine.edge >= 0) {
        const float x = fp8::to_f32(mine.row[mine.edge]);
        if (x > a.m) move_to(a, x);
        const float d = max_nan(x - a.m, FAR), e = exp2_approx(d * LOG2E);
        a.s += e;
        a.t = fmaf(e, d, a.t);
    }
    const bool any = mine.first < mine.nv || mine.edge >= 0;
    const float own_max = a.s == 0.0f ? NONE : a.m;   // nothing but -inf leaves the starting maximum

    // ---------------- the block's sums, and two maxima of each warp
    float m = a.m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(ALL, m, o));
    if (lane == 0) red[0][warp] = m;
    if (g.top > 0) {
        const uint32_t o = any ? order_of(own_max) : 0u;
        const uint32_t t1 = __reduce_max_sync(ALL, o);
        const uint32_t who = __ballot_sync(ALL, o == t1);
        const uint32_t t2 = __reduce_max_sync(ALL, lane == __ffs(int(who)) - 1 ? 0u : o);
        if (lane == 0) {
            tops[2 * warp] = t1;
            tops[2 * warp + 1] = t2;
        }
    }
    if (tid == 0) count = 0;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WARPS; ++w) m = fmaxf(m, red[0][w]);
    move_to(a, m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a.s += __shfl_xor_sync(ALL, a.s, o);
        a.t += __shfl_xor_sync(ALL, a.t, o);
    }
    if (lane == 0) {
        red[1][warp] = a.s;
        red[2][warp] = a.t;
    }

    // ---------------- this block's candidates
    const int top = g.top;
    if (top > 0) {
        const uint32_t o = tops[lane];
        int above = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const uint32_t other = __shfl_sync(ALL, o, i);
            above += other > o || (other == o && i < lane);
        }
        const uint32_t pick = __ballot_sync(ALL, above == top - 1);
        const uint32_t thr = __shfl_sync(ALL, o, __ffs(int(pick)) - 1);
        if (any && order_of(own_max) >= thr) {
            mine.each([&](float x, uint32_t index) {
                if (order_of(x) >= thr && x == x) {
                    const int at = atomicAdd(&count, 1);
                    if (at < CAND) cand[at] = key_of(x, index);
                }
            });
        }
        if (tid < MAX_TOP) best[tid] = 0;
    }
    __syncthreads();
    if (tid == 0) {
        float s = 0.0f, t = 0.0f;
        for (int w = 0; w < WARPS; ++w) {
            s += red[1][w];
            t += red[2][w];
        }
        total[0] = m;
        total[1] = s;
        total[2] = t;
    }
    if (top > 0) {
        const int n = count;
        if (n <= CAND) {
            for (int c = tid; c < n; c += THREADS) {
                const uint64_t key = cand[c];
                int above = 0;
                for (int i = 0; i < n; ++i) above += cand[i] > key;
                if (above < top) best[above] = key;
            }
        } else {
            // Rows with very many equal or nearly sorted values: the largest key
            // below the last one found, `top` times over the thread's elements.
            uint64_t last = ~uint64_t(0);
            for (int k = 0; k < top; ++k) {
                uint64_t key = 0;
                mine.each([&](float x, uint32_t index) {
                    const uint64_t c = x == x ? key_of(x, index) : 0;
                    if (c < last && c > key) key = c;
                });
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const uint64_t other = __shfl_xor_sync(ALL, key, o);
                    key = other > key ? other : key;
                }
                if (lane == 0) wkey[warp] = key;
                __syncthreads();
#pragma unroll
                for (int w = 0; w < WARPS; ++w) key = wkey[w] > key ? wkey[w] : key;
                if (tid == 0) best[k] = key;
                last = key;
                __syncthreads();
            }
        }
    }
    __syncthreads();

    // ---------------- the row's sums and list, from its blocks
    if (split > 1) {
        cluster_sync();
        if (rank == 0) {
            float ms[MAX_SPLIT], mm = LOWEST;
            for (uint32_t q = 0; q < split; ++q) mm = fmaxf(mm, ms[q] = ld_cluster_f32(&total[0], q));
            float s = 0.0f, t = 0.0f;
            for (uint32_t q = 0; q < split; ++q) {
                Sums b{ms[q], ld_cluster_f32(&total[1], q), ld_cluster_f32(&total[2], q)};
                move_to(b, mm);
                s += b.s;
                t += b.t;
            }
            const int all = int(split) * top;
            if (tid < all) cand[tid] = ld_cluster_u64(&best[tid % top], uint32_t(tid / top));
            __syncthreads();
            if (tid == 0) {
                total[0] = mm;
                total[1] = s;
                total[2] = t;
            }
            if (tid < all) {
                const uint64_t key = cand[tid];
                int above = 0;
                for (int i = 0; i < all; ++i) above += cand[i] > key;
                if (key != 0 && above < top) best[above] = key;
            }
        }
        __syncthreads();
        cluster_sync();                       // the others' shared memory has been read
        if (rank != 0) return;
    }

    // ---------------- results
    const float M = total[0], S = total[1], Tsum = total[2];
    const float log_s = logf(S);
    const bool empty = S == 0.0f;             // every logit is -inf
    if (tid == 0) {
        if (!(S <= 3.4e38f)) record_error(g.st, GPTQ_ERR_NONFINITE, int(min(row, int64_t(0x7FFFFFFF))));
        const int64_t target = g.targets[row];
        float lp = 0.0f;                      // a negative target is not scored
        if (target >= g.vocab) {
            record_error(g.st, GPTQ_ERR_INVALID_ARG, int(min(row, int64_t(0x7FFFFFFF))));
            lp = __uint_as_float(0x7FC00000u);
        } else if (target >= 0) {
            lp = empty ? NONE : (fp8::to_f32(x0[target]) - M) - log_s;
        }
        g.logp[row] = lp;
        if (g.entropy) g.entropy[row] = empty ? 0.0f : log_s - Tsum / S;
    }
    if (tid < top) {
        const uint64_t key = best[tid];
        const bool bad = !(S <= 3.4e38f) || key == 0;
        g.top_ids[row * top + tid] = bad ? -1 : int32_t(~uint32_t(key));
        g.top_logp[row * top + tid] =
            bad ? __uint_as_float(0x7FC00000u) : empty ? NONE : (value_of(uint32_t(key >> 32)) - M) - log_s;
    }
}

}  // namespace lp

namespace {

template <typename T, int E>
int launch_rows(const lp::Args& g, cudaStream_t stream) {
    using namespace lp;
    constexpr int kMaxDev = 64;
    static std::atomic<int> room[kMaxDev];   // blocks resident on the whole GPU
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return GPTQ_ERR_CUDA;
    if (room[dev].load() == 0) {
        int sms = 0, per = 0;
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, logprobs_kernel<T, E>, THREADS, 0) != cudaSuccess)
            return GPTQ_ERR_CUDA;
        room[dev].store(std::max(1, sms * per));
    }
    // Blocks of a row: as many as fit beside the other rows', each with at
    // least one batch of BATCH values a thread.
    const int64_t split = std::max<int64_t>(
        1, std::min<int64_t>(std::min<int64_t>(MAX_SPLIT, g.vocab / (THREADS * BATCH)), room[dev].load() / g.n));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(g.n * split));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(split);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, logprobs_kernel<T, E>, g) != cudaSuccess) return GPTQ_ERR_CUDA;
    count_launch();
    return GPTQ_OK;
}

// 16-byte loads where a thread gets at least one of them; below that single
// values, so that every thread of the block has a maximum to offer.
template <typename T>
int launch_type(const lp::Args& g, cudaStream_t stream) {
    constexpr int E = 16 / int(sizeof(T));
    return g.vocab >= 2 * lp::THREADS * E ? launch_rows<T, E>(g, stream) : launch_rows<T, 1>(g, stream);
}

}  // namespace

int launch_token_logprobs(const void* logits, int dtype, int64_t n, int64_t vocab, int64_t ld,
                          const int64_t* targets, float* logp, float* entropy, int top, float* top_logp,
                          int32_t* top_ids, cudaStream_t stream, DevStatus* st) {
    const lp::Args g{logits, targets, n, vocab, ld, logp, entropy, top_logp, top_ids, top, st};
    if (dtype == GPTQ_F32) return launch_type<float>(g, stream);
    if (dtype == GPTQ_BF16) return launch_type<__nv_bfloat16>(g, stream);
    return launch_type<__half>(g, stream);
}

}  // namespace gptq
