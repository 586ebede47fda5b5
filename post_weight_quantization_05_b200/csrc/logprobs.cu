// Log probabilities of given tokens under rows of logits, the entropy of each
// row's distribution, and its k likeliest tokens.
//
//   M = max x;  S = sum e^(x - M);  T = sum e^(x - M) (x - M)
//   logp(v) = (x_v - M) - ln S;  entropy = ln S - T / S
//
// The bound is HBM: each logit is read once.  Rows arrive in pieces of 16 KB
// through a ring of bulk copies that a warp of its own keeps full, the next row's
// first pieces while this row's results are formed.  Each of the other threads
// keeps running sums in base 2,
//   s = sum 2^z;  t = sum 2^z z;  z = x log2 e - k,  k an integer near the maximum's,
// moved to a new k (exactly: a power of two) where a piece's maximum lies well
// above, and the block joins them at the row's end.  A value costs one packed half of
// each of a multiply-add (z, one rounding), an add and a multiply-add, and one ex2.
// A masked value (-inf) makes 2^z z a NaN: the thread then adds that piece again,
// and the row's others, with z bounded.  Rows that base 2 cannot hold (values
// past 1e9, or NaN and infinities) are summed again about their maximum with
// every step guarded.
//
// The k likeliest come out of the same pass: the threads' maxima are distinct
// elements of the row, so the k-th largest of a few of them is a threshold that
// at least k elements reach; each thread's maximum per piece, kept in shared
// memory, tells which values to look at again (L2 still holds them), and the few
// that pass are ranked by (value descending, index ascending).  Where too many
// equal the threshold, those above it and the first that equal it.  All this is
// a row's latency, not its work, so two more warps do it, every other row each,
// while the summing warps are in the next row.
//
// Measured on a B200: 8192 x 50257 bf16 135 us without alternatives (6.1 TB/s), 147
// with five, 171 with twenty (163 and 198 when every found value was appended by a
// ballot of its own; 235 with five when the summing threads did it; finer maxima,
// per half piece, 182); 8192 x 50304 fp32 with five 238 us (6.9 TB/s); one row of
// 128000 fp32 5.2, 7.5 and 12.8 us with none, one and twenty, which is latency: the
// block's joins, the look at the found values again and the cluster's joins.
//
// A row is one block's, or, when there are fewer rows than the GPU has room
// for, a cluster's: its blocks take turns in the row's pieces, and the first joins
// the sums and ranks the others' best through distributed shared memory.  The
// order of every sum is fixed: the same inputs give the same bits.
#include <atomic>
#include <type_traits>

#include "fp8.cuh"
#include "kernels.h"

namespace gptq {
namespace lp {

constexpr int WARPS = 4, THREADS = 32 * WARPS;       // that sum
constexpr int BLOCK = THREADS + 96;                  // and a warp for the copies and two for the results
constexpr int RESIDENT = 5;                          // blocks per SM
constexpr int MAX_TOP = 32;
constexpr int MAX_SPLIT = 8;
constexpr int VECS = 8;                              // 16-byte vectors of a thread per piece
constexpr int PIECE = THREADS * VECS;                // vectors of a piece, 16 KB
constexpr int RING = 2;                              // pieces in flight per block
constexpr int MAX_SLOTS = 32;
template <typename T>                                // bounds kept per thread (of one or more pieces each)
constexpr int SLOTS = 64 / int(sizeof(T));
constexpr int HITS = 128;                            // groups of values to look at again
constexpr int CAND = 256;                            // candidates
constexpr float LOWEST = -3.402823466e38f;
constexpr float FAR = -1e30f;        // x - M from here on counts as this: e^FAR = 0, and 0 * FAR = 0
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.69314718055994531f;

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

// Sums about a maximum m, natural and guarded: the joins, and the rows that
// base 2 cannot hold.
struct Sums {
    float m, s, t;
};
__device__ __forceinline__ void move_to(Sums& a, float m) {
    const float d = fmaxf(a.m - m, FAR), f = exp2_approx(d * LOG2E);
    a.t = f * fmaf(a.s, d, a.t);
    a.s *= f;
    a.m = m;
}
__device__ __forceinline__ void add_one(Sums& a, float x) {
    if (x > a.m) move_to(a, x);
    const float d = max_nan(x - a.m, FAR), e = exp2_approx(d * LOG2E);
    a.s += e;
    a.t = fmaf(e, d, a.t);
}

// Sums in base 2.
constexpr float K_NONE = -1e9f;   // k before any value; below it a row's values count as 0
constexpr float Z_FAR = -1000.0f;  // z from here on counts as this: 2^z = 0
struct Sums2 {
    float k, s, t;
};
__device__ __forceinline__ void move_to(Sums2& a, float k) {
    const float d = fmaxf(a.k - k, -127.0f);                             // 2^d, exactly (0 for -127)
    const float f = __int_as_float((int(d) + 127) << 23);
    a.t = f * fmaf(a.s, a.k - k, a.t);
    a.s *= f;
    a.k = k;
}

// A 16-byte vector of logits.
template <typename T>
struct Vec {
    static constexpr int N = 16 / int(sizeof(T));
    uint32_t w[4];
    __device__ __forceinline__ explicit Vec(uint4 v) : w{v.x, v.y, v.z, v.w} {}
    // values 2 i and 2 i + 1
    __device__ __forceinline__ void pair(int i, float& a, float& b) const {
        if constexpr (sizeof(T) == 4) {
            a = __uint_as_float(w[2 * i]);
            b = __uint_as_float(w[2 * i + 1]);
        } else if constexpr (std::is_same<T, __half>::value) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            a = f.x;
            b = f.y;
        } else {
            a = __uint_as_float(w[i] << 16);
            b = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
};
// The largest of many vectors' values (16-bit types: two lines of maxima). NaN is passed over.
template <typename T>
struct Top {
    uint32_t m;
    __device__ __forceinline__ Top()
        : m(sizeof(T) == 4 ? 0xFF800000u : std::is_same<T, __half>::value ? 0xFC00FC00u : 0xFF80FF80u) {}
    __device__ __forceinline__ void add(const Vec<T>& v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) {
                m = __float_as_uint(fmaxf(__uint_as_float(m), __uint_as_float(v.w[i])));
            } else if constexpr (std::is_same<T, __half>::value) {
                const __half2 r = __hmax2(*reinterpret_cast<const __half2*>(&m),
                                          *reinterpret_cast<const __half2*>(&v.w[i]));
                m = *reinterpret_cast<const uint32_t*>(&r);
            } else {
                const __nv_bfloat162 r = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&m),
                                                 *reinterpret_cast<const __nv_bfloat162*>(&v.w[i]));
                m = *reinterpret_cast<const uint32_t*>(&r);
            }
        }
    }
    __device__ __forceinline__ float value() const {
        Vec<T> v(make_uint4(m, m, m, m));
        float a, b;
        v.pair(0, a, b);
        return fmaxf(a, b);
    }
};
__device__ __forceinline__ void add_guarded(Sums2& a, float x) {   // a.k is not far below x log2 e
    const float z = max_nan(fmaf(x, LOG2E, -a.k), Z_FAR), e = exp2_approx(z);
    a.s += e;
    a.t = fmaf(e, z, a.t);
}
// This thread's `count` vectors of a piece, THREADS apart, into its sums; returns
// their maximum.  t = sum 2^z z loses as many bits as the z of the values that
// count are large, so k follows the maximum: where a piece's lies more than NEAR
// above k, k moves to it once the piece is added, and where it lies RISE above,
// first, the piece added again.  (With k left 60 behind, 50257 equal logits 40 above
// the first piece's had an entropy 1.5e-4 off; 5e-6 at most now.  8192 x 50257 bf16
// with no and with five alternatives: 135 and 147 us; 141 and 153 with NEAR = 0, two
// more with RISE = 8.)  guarded: a masked value has been met.
constexpr float NEAR = 6.0f, RISE = 16.0f;
template <typename T>
__device__ __forceinline__ float add_piece(Sums2& a, bool& guarded, const uint4* at, int count) {
    Top<T> top;
    float m;
    if (a.k == K_NONE) {
        for (int u = 0; u < count; ++u) top.add(Vec<T>(at[u * THREADS]));
        const float k = ceilf(top.value() * LOG2E);
        if (k > a.k) move_to(a, k);
    }
    for (int pass = 0; !guarded; ++pass) {      // two at most
        const uint64_t L = fp8::pack2(LOG2E, LOG2E), minus_k = fp8::pack2(-a.k, -a.k);
        uint64_t s = fp8::pack2(0.0f, 0.0f), t = s;
        auto add = [&](const Vec<T>& v) {
            top.add(v);
#pragma unroll
            for (int i = 0; i < Vec<T>::N / 2; ++i) {
                float x, y;
                v.pair(i, x, y);
                const uint64_t z = fp8::fma2(fp8::pack2(x, y), L, minus_k);
                fp8::unpack2(z, x, y);
                const uint64_t e = fp8::pack2(exp2_approx(x), exp2_approx(y));
                s = fp8::add2(s, e);
                t = fp8::fma2(e, z, t);
            }
        };
        if (count == VECS) {
#pragma unroll
            for (int u = 0; u < VECS; ++u) add(Vec<T>(at[u * THREADS]));
        } else {
            for (int u = 0; u < count; ++u) add(Vec<T>(at[u * THREADS]));
        }
        float t0, t1, s0, s1;
        fp8::unpack2(t, t0, t1);
        fp8::unpack2(s, s0, s1);
        m = top.value();
        const float rise = fmaf(m, LOG2E, -a.k);
        Sums2 piece{a.k, s0 + s1, t0 + t1};
        guarded = piece.t != piece.t;
        if (!guarded && rise <= NEAR) {
            a.s += piece.s;
            a.t += piece.t;
            return m;
        }
        const float k = ceilf(m * LOG2E);
        const bool again = guarded || (pass == 0 && rise >= RISE);
        if (k > a.k) {
            move_to(piece, k);
            move_to(a, k);
        }
        if (again) continue;
        a.s += piece.s;
        a.t += piece.t;
        return m;
    }
    for (int u = 0; u < count; ++u) top.add(Vec<T>(at[u * THREADS]));
    m = top.value();
    const float k = ceilf(m * LOG2E);
    if (k > a.k) move_to(a, k);
    for (int u = 0; u < count; ++u) {
        const Vec<T> v(at[u * THREADS]);
#pragma unroll
        for (int i = 0; i < Vec<T>::N / 2; ++i) {
            float x, y;
            v.pair(i, x, y);
            add_guarded(a, x);
            add_guarded(a, y);
        }
    }
    return m;
}
__device__ __forceinline__ void add_one(Sums2& a, float x) {
    const float k = ceilf(x * LOG2E);
    if (k > a.k) move_to(a, k);
    add_guarded(a, x);
}

// A row's values: those from the first 16-byte boundary on in vectors of E, in
// pieces that the cluster's blocks take in turn, and the few before and behind
// them, one each for the first threads of the first block.  E = 1: no vectors but
// single values, for rows too short to give every thread one.
template <typename T, int E>
struct Row {
    const T* x;
    uint32_t head, nv, pieces, tail, vocab;   // first aligned value; vectors; pieces; first value behind them
    __device__ __forceinline__ Row(const T* r, int64_t n) : x(r), vocab(uint32_t(n)) {
        const uint32_t off = uint32_t(reinterpret_cast<uintptr_t>(r) & 15u);
        head = E == 1 ? 0 : min(vocab, uint32_t(((16u - off) & 15u) / sizeof(T)));
        nv = (vocab - head) / E;
        pieces = (nv + PIECE - 1) / PIECE;
        tail = head + nv * E;
    }
    __device__ __forceinline__ uint32_t vecs(uint32_t p) const { return min(uint32_t(PIECE), nv - p * PIECE); }
    // value `t` of those outside the vectors (all the first block's), or vocab
    __device__ __forceinline__ uint32_t edge(uint32_t t, uint32_t rank) const {
        if (rank != 0) return vocab;
        return t < head ? t : min(vocab, tail + (t - head));
    }
    // f(value, index) for every value of a block, a lane of one warp each
    template <typename F>
    __device__ __forceinline__ void each(uint32_t rank, uint32_t split, uint32_t lane, F f) const {
        const uint32_t e = edge(lane, rank);
        if (e < vocab) f(fp8::to_f32(x[e]), e);
        for (uint32_t p = rank; p < pieces; p += split) {
            const uint32_t first = head + p * PIECE * E, n = vecs(p) * E;
#pragma unroll 8
            for (uint32_t i = lane; i < n; i += 32) f(fp8::to_f32(x[first + i]), first + i);
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

// What the summing warps leave for a row's results.
struct Parts {
    float m[WARPS], k[WARPS], s[WARPS], t[WARPS];
    alignas(16) uint32_t tops[32];           // the largest thread maxima of each warp
};

template <typename T, int E>
struct Finish {
    static constexpr uint32_t ALL = 0xFFFFFFFFu;
    const Args& g;
    const Row<T, E>& row;
    const T* bounds;                         // [slots][THREADS], each thread's maximum in the slot's pieces
    uint64_t *cand, *best;
    uint32_t* hits;
    uint32_t rank, split, mine, per_slot, slots;
    int lane;

    // Appends at list[n] for the lanes that have something (ballots, not
    // atomics: one lane's round trip to shared memory would be everybody's).
    template <typename V>
    __device__ __forceinline__ void append(bool mine_too, V value, V* list, uint32_t room, uint32_t& n) const {
        const uint32_t who = __ballot_sync(ALL, mine_too);
        const uint32_t at = n + __popc(who & ((1u << lane) - 1u));
        if (mine_too && at < room) list[at] = value;
        n += __popc(who);
    }
    // Candidates: the values of at least `least` (strict: above it), if they are
    // at most CAND in at most HITS groups; otherwise -1.
    __device__ __forceinline__ int collect(float least, bool strict) const {
        auto in = [&](float x) { return strict ? x > least : x >= least; };
        uint32_t n = 0, nh = 0;
        const uint32_t e = row.edge(lane, rank);
        const float edge = e < row.vocab ? fp8::to_f32(row.x[e]) : NAN;
        // four threads' bounds per lane and slot; a scan over the lanes' hits for eight slots
        for (uint32_t s0 = 0; s0 < slots; s0 += 8) {
            uint32_t mask = 0;
#pragma unroll
            for (uint32_t s = 0; s < 8; ++s) {
                if (s0 + s >= slots) break;
                T b[4];
                const T* from = bounds + (s0 + s) * THREADS + lane * 4;
                if constexpr (sizeof(T) == 4)
                    *reinterpret_cast<uint4*>(b) = *reinterpret_cast<const uint4*>(from);
                else
                    *reinterpret_cast<uint2*>(b) = *reinterpret_cast<const uint2*>(from);
#pragma unroll
                for (int i = 0; i < 4; ++i) mask |= (in(fp8::to_f32(b[i])) ? 1u : 0u) << (4 * s + i);
            }
            if (!__any_sync(ALL, mask != 0)) continue;
            const uint32_t own = __popc(mask);
            uint32_t upto = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t before = __shfl_up_sync(ALL, upto, o);
                if (lane >= o) upto += before;
            }
            for (uint32_t at = nh + upto - own; mask != 0 && at < HITS; ++at, mask &= mask - 1) {
                const uint32_t bit = __ffs(int(mask)) - 1;
                hits[at] = (s0 + bit / 4) << 16 | (lane * 4 + bit % 4);
            }
            nh += __shfl_sync(ALL, upto, 31);
        }
        if (nh > HITS) return -1;
        __syncwarp();
        append(in(edge), key_of(edge, e), cand, CAND, n);
        // a lane per vector of the groups, FLIGHT of them in flight (three spill)
        const uint32_t units = nh * VECS;
        constexpr int FLIGHT = 2;
        for (uint32_t u0 = 0; u0 < units; u0 += 32 * FLIGHT)
            for (uint32_t q0 = 0; q0 < per_slot; ++q0) {
                uint32_t at[FLIGHT];
                uint4 raw[FLIGHT];
                float one[FLIGHT];
#pragma unroll
                for (int j = 0; j < FLIGHT; ++j) {
                    const uint32_t u = u0 + 32 * j + lane, hit = hits[min(u, units - 1) / VECS];
                    const uint32_t q = (hit >> 16) * per_slot + q0, p = rank + q * split;
                    const uint32_t v = (u % VECS) * THREADS + (hit & 0xFFFFu);
                    const bool live = u < units && q < mine && v < row.vecs(p);
                    at[j] = live ? row.head + (p * PIECE + v) * E : row.vocab;
                    if constexpr (E == 1)
                        one[j] = live ? fp8::to_f32(row.x[at[j]]) : NAN;
                    else if (live)
                        raw[j] = __ldg(reinterpret_cast<const uint4*>(row.x + at[j]));
                }
#pragma unroll
                for (int j = 0; j < FLIGHT; ++j) {
                    if constexpr (E == 1) {
                        append(in(one[j]), key_of(one[j], at[j]), cand, CAND, n);
                    } else {
                        uint32_t pass = 0;                 // bit i: value i is in
                        const Vec<T> v(raw[j]);
                        if (at[j] < row.vocab) {
#pragma unroll
                            for (int i = 0; i < E / 2; ++i) {
                                float x, y;
                                v.pair(i, x, y);
                                pass |= (in(x) ? 1u : 0u) << (2 * i) | (in(y) ? 1u : 0u) << (2 * i + 1);
                            }
                        }
                        while (__any_sync(ALL, pass != 0)) {
                            const int i = pass ? __ffs(int(pass)) - 1 : 0;
                            float x = 0.0f, a, b;
#pragma unroll
                            for (int k = 0; k < E / 2; ++k) {
                                v.pair(k, a, b);
                                x = i == 2 * k ? a : i == 2 * k + 1 ? b : x;
                            }
                            append(pass != 0, key_of(x, at[j] + i), cand, CAND, n);
                            pass &= pass - 1;
                        }
                    }
                }
            }
        __syncwarp();
        return n <= CAND ? int(n) : -1;
    }
    // The candidates' `top` best in order.
    __device__ __forceinline__ void rank_candidates(int n, int top) const {
        if (lane == 0 && (n & 1)) cand[n] = 0;      // read in pairs
        __syncwarp();
        for (int c0 = 0; c0 < n; c0 += 64) {
            const int c = c0 + lane;
            const uint64_t a = c < n ? cand[c] : 0, b = c + 32 < n ? cand[c + 32] : 0;
            int above_a = 0, above_b = 0;
#pragma unroll 2
            for (int i = 0; i < n; i += 2) {
                const ulonglong2 key = *reinterpret_cast<const ulonglong2*>(cand + i);
                above_a += (key.x > a) + (key.y > a);
                above_b += (key.x > b) + (key.y > b);
            }
            if (a != 0 && above_a < top) best[above_a] = a;
            if (b != 0 && above_b < top) best[above_b] = b;
        }
    }
    // best[0 .. top) from the cluster's lists: a lane holds the head of one.
    __device__ __forceinline__ void merge_lists(int top) const {
        const uint64_t* list = cand + lane * top;
        const int have = lane < split ? top : 0;
        uint64_t head = have > 0 ? list[0] : 0, second = have > 1 ? list[1] : 0;
        int next = 2;                                 // behind `second`
        for (int q = 0; q < top; ++q) {
            const uint32_t hi = __reduce_max_sync(ALL, uint32_t(head >> 32));
            const uint32_t lo = __reduce_max_sync(ALL, uint32_t(head >> 32) == hi ? uint32_t(head) : 0u);
            const uint64_t key = uint64_t(hi) << 32 | lo;
            if (lane == 0) best[q] = key;
            if (head == key) {
                head = second;
                second = next < have ? list[next] : 0;
                ++next;
            }
        }
    }
    // best[0 .. top): this block's likeliest.
    __device__ __forceinline__ void likeliest(const uint32_t* tops, int top) const {
        best[lane] = 0;
        const uint32_t o = tops[lane];
        int above = 0;
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            const uint4 other = *reinterpret_cast<const uint4*>(tops + i);
            above += (other.x > o || (other.x == o && i < lane)) + (other.y > o || (other.y == o && i + 1 < lane)) +
                     (other.z > o || (other.z == o && i + 2 < lane)) + (other.w > o || (other.w == o && i + 3 < lane));
        }
        // (0, no value at all, only in rows that have fewer values than threads)
        const uint32_t thr_order = __shfl_sync(ALL, o, __ffs(int(__ballot_sync(ALL, above == top - 1))) - 1);
        const float thr = thr_order ? value_of(thr_order) : -INFINITY;
        __syncwarp();
        int n = collect(thr, false);
        if (n < 0 && (n = collect(thr, true)) >= 0) {
            // Very many equal the threshold: those above it, then the first equal ones.
            auto fill = [&](uint32_t first, uint32_t end) {
                for (uint32_t i0 = first; i0 < end && n < top; i0 += 256) {
                    float x[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t i = i0 + 32 * j + lane;
                        x[j] = i < end ? fp8::to_f32(row.x[i]) : NAN;
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const bool in = x[j] == thr;
                        const uint32_t who = __ballot_sync(ALL, in);
                        const int at = n + __popc(who & ((1u << lane) - 1u));
                        if (in && at < CAND) cand[at] = key_of(x[j], i0 + 32 * j + lane);
                        n = min(CAND, n + __popc(who));
                    }
                }
            };
            for (uint32_t p = rank; n < top && p < row.pieces; p += split) {
                const uint32_t first = row.head + p * PIECE * E;
                fill(p == 0 ? 0 : first, first + row.vecs(p) * E);
            }
            if (rank == 0) fill(row.tail, row.vocab);
            __syncwarp();
        }
        if (n >= 0) {
            rank_candidates(n, top);
        } else {
            // Very many above it as well: the largest key below the last one
            // found, `top` times over the block's values.
            uint64_t last = ~uint64_t(0);
            for (int q = 0; q < top; ++q) {
                uint64_t key = 0;
                row.each(rank, split, lane, [&](float x, uint32_t index) {
                    const uint64_t c = x == x ? key_of(x, index) : 0;
                    if (c < last && c > key) key = c;
                });
#pragma unroll
                for (int o2 = 16; o2 > 0; o2 >>= 1) {
                    const uint64_t other = __shfl_xor_sync(ALL, key, o2);
                    key = other > key ? other : key;
                }
                if (lane == 0) best[q] = key;
                last = key;
            }
        }
        __syncwarp();
    }
    // The block's sums about its maximum, natural.
    __device__ __forceinline__ Sums sums(const Parts& part) const {
        float m = part.m[0], k = part.k[0];
#pragma unroll
        for (int w = 1; w < WARPS; ++w) {
            m = fmaxf(m, part.m[w]);
            k = fmaxf(k, part.k[w]);
        }
        Sums all{fmaxf(m, LOWEST), 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            Sums2 a{part.k[w], part.s[w], part.t[w]};
            move_to(a, k);
            all.s += a.s;
            all.t += a.t;
        }
        if (m != -INFINITY && !(all.s > 0.0f && all.s < 1e30f && all.t == all.t)) {
            // too far out for base 2, or not finite: once more about the maximum
            Sums c{all.m, 0.0f, 0.0f};
            row.each(rank, split, lane, [&](float x, uint32_t) { add_one(c, x); });
            all.s = c.s;
            all.t = c.t;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                all.s += __shfl_xor_sync(ALL, all.s, o);
                all.t += __shfl_xor_sync(ALL, all.t, o);
            }
        } else if (all.s > 0.0f) {
            const float over = fmaf(-m, LOG2E, k);   // k above the maximum
            const float f = exp2_approx(over);
            all.t = fmaf(all.s, over, all.t) * LN2 * f;
            all.s *= f;
        }
        return all;
    }
    __device__ __forceinline__ void write(int64_t r, const Sums& all, int64_t target, float target_x) const {
        // S >= 1 and the entropy >= 0, which roundings may miss by 1e-7 where one token has nearly all
        const float log_s = max_nan(logf(all.s), 0.0f);
        const bool empty = all.s == 0.0f, bad = !(all.s <= 3.4e38f);   // every logit is -inf; one is not a number
        const float nan = __uint_as_float(0x7FC00000u);
        if (lane == 0) {
            if (bad) record_error(g.st, GPTQ_ERR_NONFINITE, int(r));
            float lp = 0.0f;                         // a negative target is not scored
            if (target >= g.vocab) {
                record_error(g.st, GPTQ_ERR_INVALID_ARG, int(r));
                lp = nan;
            } else if (target >= 0) {
                lp = empty ? -INFINITY : (target_x - all.m) - log_s;
            }
            g.logp[r] = lp;
            if (g.entropy) g.entropy[r] = empty ? 0.0f : max_nan(log_s - all.t / all.s, 0.0f);
        }
        if (lane < g.top) {
            const uint64_t key = best[lane];
            const bool none = bad || key == 0;
            g.top_ids[r * g.top + lane] = none ? -1 : int32_t(~uint32_t(key));
            g.top_logp[r * g.top + lane] =
                none ? nan : empty ? -INFINITY : (value_of(uint32_t(key >> 32)) - all.m) - log_s;
        }
    }
};

template <typename T, int E>
__global__ void __launch_bounds__(BLOCK, RESIDENT) logprobs_kernel(const Args g, const uint32_t slot_room) {
    __shared__ alignas(8) uint64_t full[RING], empty[RING];          // pieces landed, pieces read
    __shared__ alignas(8) uint64_t ready[2], taken[2];               // rows summed, rows written out
    __shared__ Parts parts[2];
    __shared__ alignas(16) uint64_t cand_of[2][CAND];
    __shared__ uint64_t best_of[2][MAX_TOP];
    __shared__ uint32_t hits_of[2][HITS];
    __shared__ float total[3];                                       // M, S, T of this block's share
    extern __shared__ __align__(128) uint8_t dynamic[];
    uint4* ring = reinterpret_cast<uint4*>(dynamic);                 // [RING][PIECE]  (E > 1)
    T* bounds =                                                      // [2][slot_room][THREADS]
        reinterpret_cast<T*>(dynamic + (E > 1 ? RING * PIECE * 16 : 0));
    constexpr uint32_t ALL = 0xFFFFFFFFu;
    constexpr float NONE = -INFINITY;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t split;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(split));
    const uint32_t rank = cluster_ctarank();
    const int64_t row0 = blockIdx.x / split, rows = gridDim.x / split;     // rows row0, row0 + rows, ...
    if (tid == 0) {
        for (int s = 0; s < RING; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], WARPS);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&ready[b], WARPS);
            mbar_init(&taken[b], 1);
        }
        fence_mbar_init();
    }
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    // pieces of this block in a row, and how many share a bound
    auto share = [&](const Row<T, E>& row) { return row.pieces > rank ? (row.pieces - rank + split - 1) / split : 0; };

    if (warp == WARPS) {
        // ---------------- copies
        if (E > 1 && lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int64_t r = row0; r < g.n && ok; r += rows) {
                const Row<T, E> row(static_cast<const T*>(g.logits) + r * g.ld, g.vocab);
                for (uint32_t p = rank; p < row.pieces; p += split, ++it) {
                    const uint32_t s = it % RING;
                    if (!mbar_wait(&empty[s], ((it / RING) & 1u) ^ 1u, g.st, 421)) { ok = false; break; }
                    const uint32_t bytes = row.vecs(p) * 16;
                    mbar_arrive_expect_tx(&full[s], bytes);
                    bulk_load(ring + s * PIECE, row.x + row.head + uint64_t(p) * PIECE * E, bytes, &full[s]);
                }
            }
            // the last copies land before the block ends, even where the sums gave up on them
            for (uint32_t i = it < RING ? 0 : it - RING; i < it; ++i)
                mbar_wait(&full[i % RING], (i / RING) & 1u, g.st, 425);
        }
    } else if (warp < WARPS) {
        // ---------------- sums
        uint32_t it = 0, nth = 0;
        bool live = true;    // a wait that ran out: go on without waiting
        for (int64_t r = row0; r < g.n; r += rows, ++nth) {
            const Row<T, E> row(static_cast<const T*>(g.logits) + r * g.ld, g.vocab);
            const uint32_t edge_at = row.edge(tid, rank);
            const float edge = edge_at < row.vocab ? fp8::to_f32(row.x[edge_at]) : NONE;
            const uint32_t mine = share(row), per_slot = (mine + SLOTS<T> - 1) / SLOTS<T>, buf = nth & 1u;
            if (live) live = mbar_wait(&taken[buf], ((nth >> 1) & 1u) ^ 1u, g.st, 423);
            Sums2 a{K_NONE, 0.0f, 0.0f};
            float own_max = NONE, slot_max = NONE;
            bool guarded = false;
            uint32_t in_slot = 0;
            T* bound = bounds + buf * slot_room * THREADS + tid;
            for (uint32_t q = 0; q < mine; ++q) {
                const uint32_t p = rank + q * split, vecs = row.vecs(p);
                float m = NONE;
                if constexpr (E == 1) {
#pragma unroll 4
                    for (uint32_t v = tid; v < vecs; v += THREADS) {
                        const float x = fp8::to_f32(row.x[p * PIECE + v]);
                        m = fmaxf(m, x);
                        add_one(a, x);
                    }
                } else {
                    const uint32_t s = it % RING;
                    if (live) live = mbar_wait(&full[s], (it / RING) & 1u, g.st, 422);
                    m = add_piece<T>(a, guarded, ring + s * PIECE + tid,
                                     vecs == PIECE ? VECS : (int(vecs) - tid + THREADS - 1) / THREADS);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&empty[s]);
                    ++it;
                }
                own_max = fmaxf(own_max, m);
                if (g.top > 0) {
                    slot_max = fmaxf(slot_max, m);
                    if (++in_slot == per_slot || q + 1 == mine) {
                        *bound = fp8::from_f32<T>(slot_max);    // exact: one of the values
                        bound += THREADS;
                        in_slot = 0;
                        slot_max = NONE;
                    }
                }
            }
            if (edge_at < row.vocab) {
                own_max = fmaxf(own_max, edge);
                add_one(a, edge);
            }
            // (all pieces of a row but its last are full, so a thread has values if it has any in the first)
            const bool any = mine > 1 || (mine == 1 && uint32_t(tid) < row.vecs(rank)) || edge_at < row.vocab;
            Parts& part = parts[buf];
            const uint32_t o = any ? order_of(own_max) : 0u;
            const uint32_t ko = __reduce_max_sync(ALL, order_of(a.k));
            move_to(a, value_of(ko));
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) {
                a.s += __shfl_xor_sync(ALL, a.s, d);
                a.t += __shfl_xor_sync(ALL, a.t, d);
            }
            const uint32_t mo = __reduce_max_sync(ALL, o);
            if (lane == 0) {
                part.m[warp] = mo ? value_of(mo) : NONE;
                part.k[warp] = a.k;
                part.s[warp] = a.s;
                part.t[warp] = a.t;
            }
            if (g.top > 0) {
                uint32_t left = o;
#pragma unroll
                for (int q = 0; q < 32 / WARPS; ++q) {
                    uint32_t t = 0;
                    if (q * WARPS < g.top) {
                        t = __reduce_max_sync(ALL, left);
                        const uint32_t who = __ballot_sync(ALL, left == t);
                        if (lane == __ffs(int(who)) - 1) left = 0;
                    }
                    if (lane == 0) part.tops[q * WARPS + warp] = t;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&ready[buf]);
        }
    } else {
        // ---------------- results: the two warps take every other row
        const uint32_t buf = warp - WARPS - 1;
        uint64_t *cand = cand_of[buf], *best = best_of[buf];
        uint32_t* hits = hits_of[buf];
        uint32_t nth = buf;
        bool live = true;
        for (int64_t r = row0 + buf * rows; r < g.n; r += 2 * rows, nth += 2) {
            const Row<T, E> row(static_cast<const T*>(g.logits) + r * g.ld, g.vocab);
            int64_t target = -1;
            float target_x = 0.0f;
            if (rank == 0) {
                target = g.targets[r];
                if (target >= 0 && target < g.vocab) target_x = fp8::to_f32(row.x[target]);
            }
            const uint32_t mine = share(row), per_slot = (mine + SLOTS<T> - 1) / SLOTS<T>;
            const Finish<T, E> finish{g, row, bounds + buf * slot_room * THREADS, cand, best, hits, rank, split, mine,
                                      per_slot, per_slot ? (mine + per_slot - 1) / per_slot : 0, lane};
            if (live) live = mbar_wait(&ready[buf], (nth >> 1) & 1u, g.st, 424);
            Sums all = finish.sums(parts[buf]);
            if (g.top > 0) finish.likeliest(parts[buf].tops, g.top);
            __syncwarp();
            if (lane == 0) mbar_arrive(&taken[buf]);
            if (split == 1) {
                finish.write(r, all, target, target_x);
                __syncwarp();                     // best has been read
                continue;
            }
            // a cluster has one row: the first block joins the sums and lists
            if (lane == 0) {
                total[0] = all.m;
                total[1] = all.s;
                total[2] = all.t;
            }
            __syncwarp();
            cluster_sync();
            if (rank == 0) {
                // a lane per block
                Sums b{LOWEST, 0.0f, 0.0f};
                if (lane < split) {
                    b.m = ld_cluster_f32(&total[0], lane);
                    b.s = ld_cluster_f32(&total[1], lane);
                    b.t = ld_cluster_f32(&total[2], lane);
                }
                float mm = b.m;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(ALL, mm, o));
                move_to(b, mm);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    b.s += __shfl_xor_sync(ALL, b.s, o);
                    b.t += __shfl_xor_sync(ALL, b.t, o);
                }
                all = Sums{mm, b.s, b.t};
                uint64_t keys[MAX_SPLIT];
#pragma unroll
                for (uint32_t q = 0; q < MAX_SPLIT; ++q)
                    if (q < split && lane < g.top) keys[q] = ld_cluster_u64(&best[lane], q);
#pragma unroll
                for (uint32_t q = 0; q < MAX_SPLIT; ++q)
                    if (q < split && lane < g.top) cand[q * g.top + lane] = keys[q];
                __syncwarp();
                finish.merge_lists(g.top);
                __syncwarp();
                finish.write(r, all, target, target_x);
            }
            __syncwarp();
            cluster_sync();                       // the others' shared memory has been read
            return;
        }
    }
    if (split > 1) {
        __syncwarp();
        cluster_sync();
        cluster_sync();
    }
}

}  // namespace lp

namespace {

template <typename T, int E>
int launch_rows(const lp::Args& g, cudaStream_t stream) {
    using namespace lp;
    constexpr int kMaxDev = 64;
    static std::atomic<int> sms[kMaxDev], resident[kMaxDev][MAX_SLOTS + 1];
    auto kernel = logprobs_kernel<T, E>;
    constexpr size_t RING_BYTES = E > 1 ? size_t(RING) * PIECE * 16 : 0;
    constexpr size_t SLOT_BYTES = 2 * THREADS * sizeof(T);     // of two rows
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return GPTQ_ERR_CUDA;
    if (sms[dev].load() == 0) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 int(RING_BYTES + SLOTS<T> * SLOT_BYTES)) != cudaSuccess)
            return GPTQ_ERR_CUDA;
        sms[dev].store(n);
    }
    // Blocks of a row: as many as fit beside the other rows', each with at least one piece.
    const int64_t pieces = (g.vocab / E + PIECE - 1) / PIECE;
    const int64_t split = std::max<int64_t>(
        1, std::min<int64_t>(std::min<int64_t>(MAX_SPLIT, pieces), int64_t(sms[dev].load()) * RESIDENT / g.n));
    const size_t slots = g.top ? size_t(std::min<int64_t>(SLOTS<T>, (pieces + split - 1) / split)) : 0;
    const size_t smem = RING_BYTES + slots * SLOT_BYTES;
    // Otherwise the blocks that the GPU holds at once share the rows.
    int per_sm = resident[dev][slots].load();
    if (per_sm == 0) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, BLOCK, smem) != cudaSuccess)
            return GPTQ_ERR_CUDA;
        per_sm = std::max(1, per_sm);
        resident[dev][slots].store(per_sm);
    }
    const int64_t room = int64_t(sms[dev].load()) * per_sm;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(split > 1 ? g.n * split : std::min(g.n, room)));
    cfg.blockDim = dim3(BLOCK);
    cfg.dynamicSmemBytes = smem;
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
    if (cudaLaunchKernelEx(&cfg, kernel, g, uint32_t(slots)) != cudaSuccess) return GPTQ_ERR_CUDA;
    count_launch();
    return GPTQ_OK;
}

// 16-byte vectors where a thread gets at least one of them; below that single
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
