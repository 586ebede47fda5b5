// Products of e4m3 codes with one fp32 scale per block of 128, on the tcgen05
// tensor cores (kind::f8f6f4).
//
//   y[t][r] = sum_b sx[b][t] sw[r / 128][b] sum_{k in block b} xc[t][k] wc[r][k]
//
// The scales change every 128 values of k, so they cannot wait for the
// epilogue: the MMAs of one block of k (four of K = 32, one 128-byte swizzle
// row of codes) fill a TMEM accumulator of their own, and eight warps then read
// it and add it, times the block's scales, to the tile's sums in fp32 registers.
// A ring of accumulators keeps the tensor cores running meanwhile.  Sums inside
// a block are the tensor core's fp32 accumulation; products of two e4m3
// values are exact there.  A block's scales are two fp32 numbers multiplied: a
// product of scales outside fp32's normal range (2^-126 .. 2^128) loses accuracy
// or overflows.
//
// Few tokens are bound by HBM (the weight's codes), prompts by the accumulators'
// way from TMEM to the sums; either kernel below says how far it gets.
//
// The gated pair runs both products of the same tokens in one kernel, so the
// tokens' codes are read once and neither product is written out:
//   h[t][r] = act(g[t][r]) u[t][r]
// as values, or as the e4m3 codes and scales that the next product takes (a
// tile holds 128 features of a token, exactly one of that product's blocks).
#include <atomic>
#include <cstring>

#include "fp8.cuh"
#include "kernels.h"

namespace gptq {
namespace fp8 {

constexpr int TILE_BYTES = 128 * 128;   // 128 rows of one 128-byte block of k
constexpr int OUT_CODES = 3;            // Args::out beside the gptq_dtype values

struct Maps {
    CUtensorMap w, u, x;   // weight, second weight (gated), tokens
};

struct Args {
    int64_t m, n, lds, ldy, ldys;
    const float *xs, *ws, *us;
    void* y;
    float* ys;
    int nkb, out;
    DevStatus* st;
};

__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// One thread of a converged warp.  The warp that issues the MMAs runs its loop
// whole and elects a thread for the tcgen05 instructions alone: their operands
// stay in uniform registers (one thread looping by itself took 85 clocks per MMA
// to move them there, more than the MMA).
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ int uniform_warp() { return __shfl_sync(0xFFFFFFFFu, int(threadIdx.x >> 5), 0); }

// Instruction descriptor, kind::f8f6f4: e4m3 x e4m3 -> f32, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
    return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// 32 lanes x 16 columns without waiting; tmem_ld_done() before the values are used.
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_ld_x32(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
// N = 16 or 32 columns.
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t* r) {
    if constexpr (N == 16)
        tmem_ld_x16(taddr, r);
    else
        tmem_ld_x32(taddr, r);
}
// Wait for this thread's TMEM loads; the values pass through it so that no
// use of them can be moved in front of the wait.
template <int N>
__device__ __forceinline__ void tmem_ld_done(uint32_t (&r)[N]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// e^x = 2^t e^(r ln 2) with t = RN(x log2 e) and r what that rounding and the
// constant's lost, a number below 2^-16 for every x that matters: 1 + r ln 2
// is exact enough, and ex2's own error (2^-22) is what remains.
__device__ __forceinline__ float exp_of(float x) {
    constexpr float L = 1.44269504f, L_LOW = 1.92596299e-8f;   // log2(e) = L + L_LOW
    const float t = x * L;
    const float r = fmaf(x, L_LOW, fmaf(x, L, -t));
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
    return fmaf(e, r * 0.693147181f, e);
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// act(g): SILU, g / (1 + e^-g); GELU in its exact form, g Phi(g), with Phi
// from erfc so that large negative gates keep their relative accuracy.  Silu of
// gates below -87.3 is 0: the reciprocal is below the normal numbers there (the
// formula's value is below 2^-119).  (The clamps keep exp_of's products finite.)
// 4096 tokens, a pair of 11008 x 4096: 344 us with silu, 407 with gelu, whose erfc is
// in the tiles' output with nothing beside it.
constexpr int SILU = 0, GELU = 1;
template <int ACT>
__device__ __forceinline__ float gate_act(float g) {
    if (ACT == SILU) {
        return g * rcp_approx(1.0f + exp_of(fminf(fmaxf(-g, -127.0f), 88.0f)));
    }
    return 0.5f * g * erfcf(g * -0.70710678118654752f);
}

__device__ __forceinline__ void store_out(void* y, int64_t at, float v, int out) {
    if (out == GPTQ_F32)
        static_cast<float*>(y)[at] = v;
    else if (out == GPTQ_BF16)
        static_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16_rn(v);
    else
        static_cast<__half*>(y)[at] = __float2half_rn(v);
}

// 4-byte asynchronous copy to shared memory; zero if !live (src is not read).
__device__ __forceinline__ void copy4_async(float* dst, const float* src, bool live) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(live ? 4 : 0)
                 : "memory");
}

// 16 bytes of which the first `live` are read, zeros behind them.
__device__ __forceinline__ void copy16_async(float* dst, const float* src, int live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(live) : "memory");
}

// ---------------------------------------------------------------------------
// Weights on the MMA's M side: a tile is 128 weight rows (one row of scale
// blocks) by all the tokens, NT at most, which keeps the tile full for one token
// as for 32.
// The cluster's CTAs share a tile's blocks of k -- a gated pair's even ones the
// gate's, the odd ones the up projection's -- and add their sums through
// distributed shared memory in rank order: no workspace, no atomics, the same
// bits on every call.  Measured: 8192 x 28672, one token 37.6 us (6.24 TB/s);
// a pair of 11008 x 4096 weights, 4 tokens 18.6 us (4.9 TB/s: 13.8 us of reading
// and what start, exchange and codes take).
template <int NT>
struct Narrow {
    static constexpr int BLOCK_BYTES = TILE_BYTES + NT * 128;
    // A stage is a group of blocks of k: the waits, the commit and the sums' start
    // cost about 0.3 us a stage, against the 0.37 us that one SM's share of HBM
    // takes for a block (16 KB).  8192 x 28672, one token: 46 us with one block a
    // stage, 37.6 with two.
    static constexpr int GROUP = 2;
    static constexpr int STAGE_BYTES = GROUP * BLOCK_BYTES;
    static constexpr int SUM_WARPS = 8;                   // two sets of four take every other stage
    static constexpr int THREADS = 32 * (SUM_WARPS + 2);  // and a warp each for loads and MMAs
    static constexpr int MAX_SPLIT = 8;                  // CTAs of a tile: a portable cluster
    static constexpr int AHEAD = 2, RING = 4;            // stages of scales per warp, in flight and kept
    static constexpr int ENTRY = GROUP * (NT + 4);       // floats of one: per block the tokens', then the weights'
    static constexpr int OTHER_BYTES = (SUM_WARPS * RING * ENTRY + 4 * NT) * 4;
    // Two CTAs share an SM's 228 KB (1 KB of them per CTA the driver's): fewer SMs
    // idle than with one.  11008 x 4096, 8 tokens: 11.3 us against 13.7.
    static constexpr int PER_SM = 2;
    static constexpr int STAGES = (233472 / PER_SM - 1024 - 1024 - OTHER_BYTES - 256) / STAGE_BYTES;
    static constexpr int STAGE_COLS = GROUP * NT;  // TMEM columns: an accumulator per block of the stage
    static constexpr int COLS = STAGES * STAGE_COLS <= 64    ? 64
                                : STAGES * STAGE_COLS <= 128 ? 128
                                : STAGES * STAGE_COLS <= 256 ? 256
                                                             : 512;
    static constexpr int READ = 32;                      // accumulator columns read at once
    static constexpr size_t SMEM_BYTES = 1024 + size_t(STAGES) * STAGE_BYTES + OTHER_BYTES + 3 * STAGES * 8 + 16;
    // the sums that the cluster exchanges, and the gated values, reuse the stages
    static_assert(3 * NT * 128 * 4 <= STAGES * STAGE_BYTES, "exchange buffer");
    static_assert(SMEM_BYTES <= 232448, "shared memory");
    static_assert(PER_SM * COLS <= 512 && STAGES * STAGE_COLS <= COLS, "TMEM columns");
    static_assert(STAGES >= 2, "a set of sum warps starts a stage's second round after the other's first");
};

template <int NT, bool GATED, int ACT>
__global__ void __launch_bounds__(Narrow<NT>::THREADS, Narrow<NT>::PER_SM)
    narrow_kernel(const __grid_constant__ Maps maps, const Args g) {
    using C = Narrow<NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* ring_all = reinterpret_cast<float*>(smem + size_t(C::STAGES) * C::STAGE_BYTES);   // [SUM_WARPS][RING][ENTRY]
    uint32_t* amax = reinterpret_cast<uint32_t*>(ring_all + C::SUM_WARPS * C::RING * C::ENTRY);   // [NT][4]
    uint64_t* full = reinterpret_cast<uint64_t*>(amax + 4 * NT);   // [STAGES] TMA landed
    uint64_t* done = full + C::STAGES;                             // [STAGES] MMAs complete
    uint64_t* read = done + C::STAGES;                             // [STAGES] accumulators read by four warps
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(read + C::STAGES);

    uint32_t split;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(split));
    const uint32_t rank = cluster_ctarank();
    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const int tile = int(blockIdx.x / split);
    const int64_t row0 = int64_t(tile) * 128;
    // this CTA's weight and its blocks of k
    const bool up = GATED && (rank & 1u);
    const uint32_t share = GATED ? rank >> 1 : rank, shares = GATED ? split >> 1 : split;
    const int b0 = int(int64_t(g.nkb) * share / shares), blocks = int(int64_t(g.nkb) * (share + 1) / shares) - b0;
    const CUtensorMap* wmap = up ? &maps.u : &maps.w;

    if (threadIdx.x == 0) {
        tma_prefetch_desc(wmap);
        tma_prefetch_desc(&maps.x);
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&done[s], 1);
            mbar_init(&read[s], 4);
        }
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(tmem_slot, C::COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    pdl_wait();
    pdl_trigger();

    float acc[NT];
#pragma unroll
    for (int c = 0; c < NT; ++c) acc[c] = 0.0f;

    const int groups = (blocks + C::GROUP - 1) / C::GROUP;
    if (warp == C::SUM_WARPS) {
        if (lane == 0) {
            int issued = 0;
            for (int i = 0; i < groups; ++i) {
                const int s = i % C::STAGES, count = min(C::GROUP, blocks - i * C::GROUP);
                if (!mbar_wait(&done[s], (uint32_t(i / C::STAGES) & 1u) ^ 1u, g.st, 401)) break;
                mbar_arrive_expect_tx(&full[s], uint32_t(count) * C::BLOCK_BYTES);
                for (int q = 0; q < count; ++q) {
                    uint8_t* base = smem + size_t(s) * C::STAGE_BYTES + q * C::BLOCK_BYTES;
                    const int k = (b0 + i * C::GROUP + q) * 128;
                    tma_load_2d(base, wmap, k, int(row0), &full[s]);
                    tma_load_2d(base + TILE_BYTES, &maps.x, k, 0, &full[s]);
                }
                issued = i + 1;
            }
            // the last copies land before the CTA goes on, even where the MMAs gave up on them
            for (int i = max(0, issued - C::STAGES); i < issued; ++i)
                mbar_wait(&full[i % C::STAGES], uint32_t(i / C::STAGES) & 1u, g.st, 405);
        }
    } else if (warp > C::SUM_WARPS) {
        constexpr uint32_t idesc = idesc_e4m3(128, NT);
        const uint64_t desc0 = sdesc_sw128(smem_u32(smem), 16, 1024);
        for (int i = 0; i < groups; ++i) {
            const int s = i % C::STAGES, count = min(C::GROUP, blocks - i * C::GROUP);
            const uint32_t round = uint32_t(i / C::STAGES) & 1u;
            bool ok = mbar_wait(&read[s], round ^ 1u, g.st, 402);
            ok = ok && mbar_wait(&full[s], round, g.st, 403);
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int q = 0; q < C::GROUP; ++q) {
                    if (q >= count) continue;
                    const uint64_t wd = desc0 + uint32_t(s * C::STAGE_BYTES + q * C::BLOCK_BYTES) / 16;
                    const uint32_t dt = tmem_base + uint32_t(s * C::STAGE_COLS + q * NT);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)   // 32 codes (32 bytes) of the 128-byte swizzle row
                        umma_f8(dt, wd + 2 * kk, wd + TILE_BYTES / 16 + 2 * kk, idesc, kk > 0 ? 1u : 0u);
                }
                umma_commit(&done[s]);               // frees the stage and completes its accumulators
            }
            __syncwarp();
        }
    } else {
        // ---------------- sums: thread = weight row (TMEM lane), registers = tokens
        const int set = warp >> 2;
        float* ring = ring_all + warp * C::RING * C::ENTRY;
        const float* xs = g.xs + int64_t(b0) * g.lds;
        const float* ws = (up ? g.us : g.ws) + int64_t(tile) * g.nkb + b0;
        auto fetch = [&](int i) {
            float* at = ring + ((i >> 1) % C::RING) * C::ENTRY;
#pragma unroll
            for (int c = lane; c < C::GROUP * NT; c += 32) {
                const int q = c / NT, t = c % NT, b = i * C::GROUP + q;
                const bool live = b < blocks && t < g.m;
                copy4_async(at + q * (NT + 4) + t, live ? xs + int64_t(b) * g.lds + t : xs, live);
            }
            if (lane < C::GROUP) copy4_async(at + lane * (NT + 4) + NT, ws + min(i * C::GROUP + lane, blocks - 1), true);
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        for (int i = 0; i < C::AHEAD; ++i) fetch(2 * i + set);
        bool live = true;    // a wait that ran out: go on without waiting
        for (int i = set; i < groups; i += 2) {
            const int s = i % C::STAGES, count = min(C::GROUP, blocks - i * C::GROUP);
            fetch(i + 2 * C::AHEAD);
            asm volatile("cp.async.wait_group %0;" ::"n"(C::AHEAD) : "memory");
            __syncwarp();                     // all lanes' copies of the stage's scales have landed
            const float* scales = ring + ((i >> 1) % C::RING) * C::ENTRY;
            if (live) live = mbar_wait(&done[s], uint32_t(i / C::STAGES) & 1u, g.st, 404);
            live = __all_sync(0xFFFFFFFFu, live);
            tc_fence_after();
            const uint32_t dt = tmem_base + (uint32_t((warp & 3) * 32) << 16) + uint32_t(s * C::STAGE_COLS);
#pragma unroll
            for (int j = 0; j < C::STAGE_COLS; j += C::READ) {
                uint32_t v[C::READ];
#pragma unroll
                for (int c = 0; c < C::READ; c += 32) tmem_ld_x32(dt + j + c, v + c);
                tmem_ld_done(v);
                if (j + C::READ == C::STAGE_COLS) {   // this warp has read the whole stage
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&read[s]);
                }
#pragma unroll
                for (int c = 0; c < C::READ; c += 4) {
                    const int q = (j + c) / NT, t = (j + c) % NT;
                    if (q >= count) continue;         // (blocks behind the last are not written)
                    const float* at = scales + q * (NT + 4);
                    const float4 sx = *reinterpret_cast<const float4*>(at + t);
                    const float w = at[NT];
                    float* sum = acc + t;
                    // (the scales first: a block's sum times one of them may leave fp32's range)
                    sum[0] = fmaf(__uint_as_float(v[c]), sx.x * w, sum[0]);
                    sum[1] = fmaf(__uint_as_float(v[c + 1]), sx.y * w, sum[1]);
                    sum[2] = fmaf(__uint_as_float(v[c + 2]), sx.z * w, sum[2]);
                    sum[3] = fmaf(__uint_as_float(v[c + 3]), sx.w * w, sum[3]);
                }
            }
        }
    }
    // The accumulators are in registers: TMEM goes back before this CTA waits
    // for others, so a CTA that holds TMEM never depends on one that waits for it.
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem_base, C::COLS);

    float* part = reinterpret_cast<float*>(smem);   // [2][NT][128] the sums of this CTA's two sets
    const int set = warp >> 2, r = threadIdx.x & 127;
    if (warp < C::SUM_WARPS) {
#pragma unroll
        for (int c = 0; c < NT; ++c) part[(set * NT + c) * 128 + r] = acc[c];
    }
    __syncwarp();
    cluster_sync();
    const int cols = int(g.m);
    if (warp < C::SUM_WARPS) {
        // tokens (columns) rank, rank + split, ..., every other one to each set
        const int first = int(rank) + set * int(split), step = 2 * int(split);
        const int64_t row = row0 + r;
        float* held = part + 2 * NT * 128;    // gated values until their block's scale is known
        for (int c = first; c < cols; c += step) {
            float v = 0.0f, u = 0.0f;
            for (uint32_t q = 0; q < split; ++q)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float p = ld_cluster_f32(mapa_shared(part + (h * NT + c) * 128 + r, q));
                    if (GATED && (q & 1u))
                        u += p;
                    else
                        v += p;
                }
            if (GATED) v = gate_act<ACT>(v) * u;
            if (GATED && g.out == OUT_CODES) {
                held[c * 128 + r] = v;
                const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v) & 0x7FFFFFFFu);
                if (lane == 0) amax[c * 4 + (warp & 3)] = top;
            } else if (row < g.n) {
                store_out(g.y, c * g.ldy + row, v, g.out);
            }
        }
        if (GATED && g.out == OUT_CODES) {
            named_barrier_sync(1 + set, 128);
            for (int c = first; c < cols; c += step) {
                const uint32_t a = max(max(amax[4 * c], amax[4 * c + 1]), max(amax[4 * c + 2], amax[4 * c + 3]));
                float s = block_scale(a), v = held[c * 128 + r];
                if (r == 0) {
                    g.ys[int64_t(tile) * g.ldys + c] = s;
                    if (a >= INF_BITS) record_error(g.st, GPTQ_ERR_NONFINITE, c);
                }
                if (s < SMALL_SCALE) {
                    s *= SMALL_LIFT;
                    v *= SMALL_LIFT;
                }
                if (row < g.n)
                    static_cast<uint8_t*>(g.y)[c * g.ldy + row] = uint8_t(Coder(s, rcp_approx(s)).one(v));
            }
        }
    }
    __syncwarp();
    cluster_sync();   // peers have read this CTA's sums
}

// ---------------------------------------------------------------------------
// Tokens on the MMA's M side, for prompts: a cluster of two CTAs owns a tile of
// 256 tokens by 256 weight rows (gated: 128 rows of each weight) and runs it as
// cta_group::2 MMAs (M = N = 256, K = 32).  CTA r loads tokens 128 r .. 128 r +
// 127 of the tile and its half of the weight rows (gated: r = 0 the gate's,
// r = 1 the up projection's), 32 KB per block of k, and holds its tokens' 256
// sums: one block fills 256 TMEM columns in 512 clocks, and two accumulators
// take turns.  Eight warps keep the sums, a token per lane and 128 columns per
// thread, so a block's scales are one number per thread (gated: two).  One CTA
// alone would load 48 KB a block for the same MMA work, past the 128 bytes per
// clock that shared memory gives at the tensor cores' e4m3 rate.
//
// Two warps bring the scales: they copy a block's ahead, multiply the tokens' by
// the weights' into a ring in shared memory, and arrive on the same barrier as the
// block's MMAs.  (The sums' warps did it themselves before, 270 of a block's
// clocks: 4096 tokens, a pair of 11008 x 4096, 393 us then, 343 now.)
//
// Measured: 4096 tokens, 8192 x 28672 814 to 847 us from GPU to GPU (2270 to 2360
// TFLOP/s; 948 before the MMAs were issued by an elected thread), 8192 x 4096 128
// us; calls that follow one another without a pause take up to 990 under the power
// cap.  A block takes some 800 clocks, not 512.  What is in the way is the whole
// circle of an accumulator -- MMAs, their arrival, 128 KB read from TMEM and 32768
// multiply-adds, the arrival back -- and power: without the sums' reads and
// multiply-adds the same kernel takes 680 us.  Tried and slower: 128 columns per MMA
// and accumulator, released one by one, with one issuing warp or two (1110 us: A is
// read twice), sixteen warps for the sums.  (Stages: three to six of 32 KB measured
// the same.)
//
// Two variations fit fewer tiles to the GPU: TN = 128 (half the weight rows, four
// accumulators), and SPLIT pairs in a cluster that share a tile's blocks of k
// and add their sums through distributed shared memory, a slice of the columns
// each, in rank order.  A block of 128 columns costs nearly what one of 256 does (590
// clocks, of which 256 are MMAs): the waits, the first TMEM load and the arrivals
// are the same.
template <int TN, int SPLIT>
struct Wide {
    static constexpr int STAGE_BYTES = TILE_BYTES + TN / 2 * 128;
    static constexpr int STAGES = TN == 256 ? 4 : 5;      // some 128 KB
    static constexpr int SLOTS = 512 / TN;
    static constexpr int SUM_WARPS = 8;
    static constexpr int PARTS = SUM_WARPS / 4;           // threads that share a token's columns
    static constexpr int CPT = TN / PARTS;                // columns of a thread
    static constexpr int THREADS = 32 * (SUM_WARPS + 4);  // and one for loads, one for MMAs, two for scales
    // Registers per thread after the split between the sums' two warpgroups and
    // the third; the launch checks that they fit what it was given.  (216 and 72
    // left the sums' loop spilling.)
    static constexpr int SUM_REGS = 232, OTHER_REGS = 40;
    static constexpr int AHEAD = 2;                       // blocks of scales of a warp on their way
    static constexpr int ENTRY = 128 + 4;                 // floats of one: the tokens', two of the weights
    // Blocks of scales kept: four rounds of the stages, each with a barrier on which the
    // sums say once that they have read it.  The scales' warps are at most STAGES
    // blocks ahead of the MMAs, which are at most SLOTS ahead of the sums, so they never
    // wait for room.  (The barriers cost 1% of the long products.  The same arrival
    // behind a branch cost 4%, a wait behind one in the scales' warps 5% of 509 tokens,
    // 11008 x 4096.)
    static constexpr int RING = 4 * STAGES;
    static_assert(SLOTS <= STAGES, "room for the scales ahead");
    static constexpr int RING_BYTES = (RING * 2 * 128 + 2 * AHEAD * ENTRY) * 4; // per token and block: two products of its scale and a weight's
    static constexpr int OUT_BYTES = 32 * 256;            // per warp: 256 bytes of 32 output rows on their way out
    static constexpr size_t SMEM_BYTES = 1024 + size_t(STAGES) * STAGE_BYTES + SUM_WARPS * OUT_BYTES + RING_BYTES +
                                         2 * PARTS * 128 * 4 +
                                         (2 * STAGES + SLOTS + 4) * 8 + 16;
    static_assert(SMEM_BYTES <= 232448, "shared memory");
    static_assert(SMEM_BYTES > 117 * 1024, "a pair that holds its TMEM until its peers are done shares its SM with no other");
    static_assert(SPLIT == 1 || TN * 128 * 4 <= STAGES * STAGE_BYTES, "exchange buffer");
};

// Arrive on a barrier of this CTA where `yes` (predicated, without a branch).
__device__ __forceinline__ void mbar_arrive_if(uint64_t* bar, bool yes) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %1, 0;\n\t"
        "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"(uint32_t(yes))
        : "memory");
}
// Wait for two barriers, with one branch where both phases are complete.
__device__ __forceinline__ bool mbar_wait2(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb, DevStatus* st,
                                           int where) {
    const bool x = mbar_try_wait(a, pa), y = mbar_try_wait(b, pb);
    if (x && y) return true;
    return mbar_wait(a, pa, st, where) && mbar_wait(b, pb, st, where + 1);
}
__device__ __forceinline__ void umma_f8_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// a[0..1] += v[0..1] * s
__device__ __forceinline__ void add_scaled2(float* a, const uint32_t* v, float s) {
    unpack2(fma2(pack2(__uint_as_float(v[0]), __uint_as_float(v[1])), pack2(s, s), pack2(a[0], a[1])), a[0], a[1]);
}
// Arrive on an mbarrier of either CTA without publishing memory: for an
// accumulator that has been read (its loads have returned) nothing else needs
// to be ordered (the scales' ring has barriers of its own), and a release at
// cluster scope would wait for every copy and store this thread has in flight
// (measured: it was the kernel's whole time, 1.9 ms instead of 0.7 at 4096 x 8192
// x 28672).
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// Tile t of tiles_m x tiles_n, in groups of eight tile rows: the tiles that run
// at the same time share few token and weight rows, which L2 then serves.
__device__ __forceinline__ void grouped_tile(uint32_t t, uint32_t tiles_m, uint32_t tiles_n, uint32_t& tm,
                                             uint32_t& tn) {
    constexpr uint32_t G = 8;
    const uint32_t group = t / (G * tiles_n), in = t % (G * tiles_n);
    const uint32_t rows = min(G, tiles_m - group * G);
    tm = group * G + in % rows;
    tn = in / rows;
}

// A warp's 32 output rows of RB bytes (a power of two, 16 .. 256), staged in
// shared memory: lane r writes row r, then the lanes write whole pieces of rows
// to global memory (straight from the registers each 16-byte store of a warp
// would touch 32 lines).  at(): where 16-byte chunk c of row r is kept, so that
// neither side's eight-lane phases meet in a bank.
template <int RB>
struct Stage {
    static constexpr int CHUNKS = RB / 16;
    static __device__ __forceinline__ int at(int r, int c) {
        return r * RB + ((c ^ (CHUNKS >= 8 ? r & 7 : (r * CHUNKS >> 3) & (CHUNKS - 1))) << 4);
    }
    // rows x cols elements of T go to y (row pitch ld elements); vec: y and ld allow 16-byte stores.
    template <typename T>
    static __device__ __forceinline__ void flush(const uint8_t* buf, T* y, int64_t ld, int rows, int cols, bool vec,
                                                 int lane) {
        __syncwarp();
        if (vec && cols == RB / int(sizeof(T))) {
#pragma unroll
            for (int i = 0; i < CHUNKS; ++i) {
                const int r = i * (32 / CHUNKS) + lane / CHUNKS, c = lane % CHUNKS;
                if (r < rows)
                    *reinterpret_cast<uint4*>(y + r * ld + c * (16 / int(sizeof(T)))) =
                        *reinterpret_cast<const uint4*>(buf + at(r, c));
            }
        } else {
            for (int r = 0; r < rows; ++r)
                for (int c = lane; c < cols; c += 32) {
                    const int byte = c * int(sizeof(T));
                    y[r * ld + c] = *reinterpret_cast<const T*>(buf + at(r, byte >> 4) + (byte & 15));
                }
        }
        __syncwarp();
    }
};

// COLS values per lane (one output row each) as T.
template <typename T, int COLS>
__device__ __forceinline__ void store_rows(uint8_t* buf, T* y, int64_t ld, int rows, int64_t left, bool vec, int lane,
                                           const float* v) {
    constexpr int PER = 16 / int(sizeof(T)), RB = COLS * int(sizeof(T)) < 256 ? COLS * int(sizeof(T)) : 256;
    constexpr int PASS = RB / int(sizeof(T));
#pragma unroll
    for (int p = 0; p < COLS; p += PASS) {
#pragma unroll
        for (int j = 0; j < PASS; j += PER) {
            __align__(16) T t[PER];
#pragma unroll
            for (int i = 0; i < PER; ++i) t[i] = from_f32<T>(v[p + j + i]);
            *reinterpret_cast<uint4*>(buf + Stage<RB>::at(lane, j / PER)) = *reinterpret_cast<const uint4*>(t);
        }
        Stage<RB>::flush(buf, y + p, ld, rows, int(max(int64_t(0), min(left - p, int64_t(PASS)))), vec, lane);
    }
}
template <int COLS>
__device__ __forceinline__ void store_rows_as(const Args& g, uint8_t* buf, int64_t tok0, int64_t col, int lane,
                                              const float* v) {
    const int rows = int(max(int64_t(0), min(g.m - tok0, int64_t(32))));
    const int64_t left = g.n - col, at = tok0 * g.ldy + col;
    const bool vec = (reinterpret_cast<uintptr_t>(g.y) & 15u) == 0 && (g.ldy * (g.out == GPTQ_F32 ? 4 : 2)) % 16 == 0;
    if (g.out == GPTQ_F32)
        store_rows<float, COLS>(buf, static_cast<float*>(g.y) + at, g.ldy, rows, left, vec, lane, v);
    else if (g.out == GPTQ_BF16)
        store_rows<__nv_bfloat16, COLS>(buf, static_cast<__nv_bfloat16*>(g.y) + at, g.ldy, rows, left, vec, lane, v);
    else
        store_rows<__half, COLS>(buf, static_cast<__half*>(g.y) + at, g.ldy, rows, left, vec, lane, v);
}

// Arrive on the mbarrier at `bar`'s offset in both CTAs of the pair whose even
// CTA has rank `first` once the pair MMAs issued so far by this thread finish.
__device__ __forceinline__ void umma_commit_pair(uint64_t* bar, uint32_t first) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(uint16_t(3u << first))
        : "memory");
}

template <int TN, bool GATED, int ACT, int SPLIT>
__global__ void __launch_bounds__(Wide<TN, SPLIT>::THREADS, 1)
    wide_kernel(const __grid_constant__ Maps maps, const Args g) {
    using C = Wide<TN, SPLIT>;
    constexpr int TILE_N = GATED ? TN / 2 : TN;           // output columns of a tile
    constexpr int CPT = C::CPT, PARTS = C::PARTS;
    static_assert(!GATED || TN == 256, "a gated tile is one scale block of its output wide");
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* out_all = smem + size_t(C::STAGES) * C::STAGE_BYTES;
    float2* ring = reinterpret_cast<float2*>(out_all + C::SUM_WARPS * C::OUT_BYTES);   // [RING][128]
    float* fetched = reinterpret_cast<float*>(ring + C::RING * 128);                   // [2][AHEAD][ENTRY]
    uint32_t* amax = reinterpret_cast<uint32_t*>(fetched + 2 * C::AHEAD * C::ENTRY);     // [2][PARTS][128]
    uint64_t* full = reinterpret_cast<uint64_t*>(amax + 2 * PARTS * 128);   // even CTA: both CTAs' loads landed
    uint64_t* done = full + C::STAGES;      // both CTAs: the pair's MMAs of the stage's block are complete, its scales there
    uint64_t* tempty = done + C::STAGES;    // even CTA: accumulator read by both CTAs' warps
    uint64_t* taken = tempty + C::SLOTS;    // [4] a round's scales read by this CTA's sums
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(taken + 4);

    const uint32_t rank = cluster_ctarank(), half = rank & 1u, first = rank & ~1u;
    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    // at most 2^16 x 2^15 tiles; with SPLIT > 1 a cluster has one
    const uint32_t cl = blockIdx.x / (2 * SPLIT), ncl = gridDim.x / (2 * SPLIT);
    const uint32_t tiles_m = uint32_t((g.m + 255) / 256), tiles_n = uint32_t((g.n + TILE_N - 1) / TILE_N);
    const uint32_t tiles = tiles_m * tiles_n;
    // this pair's blocks of k
    const uint32_t share = rank >> 1;
    const int b0 = SPLIT == 1 ? 0 : int(int64_t(g.nkb) * share / SPLIT);
    const int blocks = SPLIT == 1 ? g.nkb : int(int64_t(g.nkb) * (share + 1) / SPLIT) - b0;

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&maps.w);
        if (GATED) tma_prefetch_desc(&maps.u);
        tma_prefetch_desc(&maps.x);
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&done[s], 2);
        }
        for (int s = 0; s < C::SLOTS; ++s) mbar_init(&tempty[s], 2 * C::SUM_WARPS);
        for (int s = 0; s < 4; ++s) mbar_init(&taken[s], C::SUM_WARPS);
        fence_mbar_init();
    }
    if (warp == C::SUM_WARPS) {
        tmem_alloc_pair(tmem_slot, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync();          // every CTA's barriers initialized, TMEM allocated
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    pdl_wait();
    pdl_trigger();

    if (warp >= C::SUM_WARPS) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::OTHER_REGS));
        if (warp == C::SUM_WARPS && lane == 0) {
            // ---------------- loads (both CTAs)
            const uint32_t full0 = mapa_shared(&full[0], first);
            const CUtensorMap* wmap = GATED && half == 1 ? &maps.u : &maps.w;
            uint32_t it = 0;     // blocks asked for so far
            bool ok = true;
            for (uint32_t t = cl; t < tiles && ok; t += ncl) {
                uint32_t tm, tn;
                grouped_tile(t, tiles_m, tiles_n, tm, tn);
                const int xr = int(tm * 256 + half * 128), wr = int(tn * TILE_N + (GATED ? 0 : half * (TN / 2)));
                for (int b = 0; b < blocks; ++b, ++it) {
                    const uint32_t s = it % C::STAGES, round = it / C::STAGES;
                    if (!mbar_wait(&done[s], (round & 1u) ^ 1u, g.st, 411)) { ok = false; break; }
                    uint8_t* base = smem + size_t(s) * C::STAGE_BYTES;
                    if (half == 0) mbar_arrive_expect_tx(&full[s], 2 * C::STAGE_BYTES);
                    tma_load_2d_pair(base, &maps.x, (b0 + b) * 128, xr, full0 + s * 8u);
                    tma_load_2d_pair(base + TILE_BYTES, wmap, (b0 + b) * 128, wr, full0 + s * 8u);
                }
            }
            // the pair's last copies land before it goes on, even where the MMAs gave up on them
            if (half == 0)
                for (uint32_t i = it < C::STAGES ? 0 : it - C::STAGES; i < it; ++i)
                    mbar_wait(&full[i % C::STAGES], (i / C::STAGES) & 1u, g.st, 415);
        }
        if (warp == C::SUM_WARPS + 1 && half == 0) {
            // ---------------- MMAs (the even CTA for the pair)
            constexpr uint32_t idesc = idesc_e4m3(256, TN);
            const uint64_t desc0 = sdesc_sw128(smem_u32(smem), 16, 1024);
            uint32_t s = 0, round = 0, d = 0, use = 0;    // stage and accumulator, and their rounds
            bool ok = true;
            for (uint32_t t = cl; t < tiles && ok; t += ncl) {
                for (int b = 0; b < blocks; ++b) {
                    ok = mbar_wait_cluster(&tempty[d], (use & 1u) ^ 1u, g.st, 412);
                    ok = ok && mbar_wait(&full[s], round & 1u, g.st, 413);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
                        const uint64_t xd = desc0 + s * (C::STAGE_BYTES / 16);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_f8_pair(tmem_base + d * TN, xd + 2 * kk, xd + TILE_BYTES / 16 + 2 * kk, idesc,
                                         kk > 0 ? 1u : 0u);
                        umma_commit_pair(&done[s], first);   // frees the stage and completes the accumulator
                    }
                    __syncwarp();
                    if (++s == C::STAGES) { s = 0; ++round; }
                    if (++d == C::SLOTS) { d = 0; ++use; }
                }
            }
        }
        if (warp >= C::SUM_WARPS + 2) {
            // ---------------- scales (both CTAs): every other block each, four tokens a lane
            const uint32_t mine = uint32_t(warp - C::SUM_WARPS - 2);
            const uint32_t total = cl < tiles ? ((tiles - cl + ncl - 1) / ncl) * uint32_t(blocks) : 0;
            float* room = fetched + mine * C::AHEAD * C::ENTRY;
            const float *xs = nullptr, *ws = nullptr, *us = nullptr;   // of tile t
            const bool vec = (reinterpret_cast<uintptr_t>(g.xs) & 15u) == 0 && g.lds % 4 == 0;   // 16-byte copies
            int left = 0;                                              // tokens of t from this lane's on
            uint32_t t = cl, asked = mine, to = 0;
            int next = int(mine);                                      // the next block to fetch, in tile t or behind it
            bool known = false;
            auto fetch = [&] {
                if (asked < total) {
                    for (; next >= blocks; next -= blocks) {
                        t += ncl;
                        known = false;
                    }
                    if (!known) {
                        uint32_t tm, tn;
                        grouped_tile(t, tiles_m, tiles_n, tm, tn);
                        const int64_t tok = int64_t(tm) * 256 + half * 128 + (vec ? 4 * lane : lane);
                        const int64_t row = int64_t(tn) * (GATED || TN == 128 ? 1 : 2);   // of weight scale blocks
                        xs = g.xs + int64_t(b0) * g.lds + tok;
                        ws = g.ws + row * g.nkb + b0;
                        us = GATED ? g.us + row * g.nkb + b0 : g.ws + min(row + 1, (g.n - 1) / 128) * g.nkb + b0;
                        left = int(max(int64_t(0), min(g.m - tok, int64_t(128))));
                        known = true;
                    }
                    float* e = room + to * C::ENTRY;
                    const float* x = xs + next * g.lds;
                    if (vec) {
                        copy16_async(e + 4 * lane, left > 0 ? x : g.xs, min(4 * left, 16));
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            copy4_async(e + 32 * i + lane, left > 32 * i ? x + 32 * i : g.xs, left > 32 * i);
                    }
                    if (lane < 2) copy4_async(e + 128 + lane, (lane == 0 ? ws : us) + next, true);
                    next += 2;
                }
                asked += 2;
                if (++to == C::AHEAD) to = 0;
                asm volatile("cp.async.commit_group;" ::: "memory");
            };
            for (int q = 0; q < C::AHEAD; ++q) fetch();
            uint32_t s = mine, round = 0, from = 0;
            for (uint32_t i = mine; i < total; i += 2) {
                asm volatile("cp.async.wait_group %0;" ::"n"(C::AHEAD - 1) : "memory");
                __syncwarp();                     // all lanes' copies of the block's scales have landed
                const float* e = room + from * C::ENTRY;
                const float w = e[128], u = e[129];
                bool ok = mbar_wait2(&done[s], (round & 1u) ^ 1u, &taken[round & 3u], ((round >> 2) & 1u) ^ 1u, g.st,
                                     417);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float x = e[32 * k + lane];
                    ring[(s + (round & 3u) * C::STAGES) * 128 + 32 * k + lane] = make_float2(x * w, x * u);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&done[s]);
                fetch();                          // into the room that has just been read
                if ((s += 2) >= C::STAGES) { s -= C::STAGES; ++round; }
                if (++from == C::AHEAD) from = 0;
            }
        }
        if (SPLIT > 1) {     // the sums' exchange below
            __syncwarp();
            cluster_sync();
            if (GATED) cluster_sync();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::SUM_REGS));
        // ---------------- sums (both CTAs): lane = token, registers = columns
        const int quad = warp & 3, part = warp >> 2;
        const int r = quad * 32 + lane;       // this thread's token of the CTA's 128
        const uint32_t tempty0 = mapa_shared(&tempty[0], first);
        uint8_t* out_buf = out_all + warp * C::OUT_BYTES;
        // accumulator columns of the two halves of this thread's sums (gated: gate and up)
        const uint32_t c0 = GATED ? (CPT / 2) * part : CPT * part, c1 = GATED ? TN / 2 + c0 : c0 + CPT / 2;
        uint32_t stage = 0, round = 0, slot = 0;
        uint32_t parity = 0;
        bool live = true;     // a wait that ran out: go on without waiting, so that all warps meet at the barriers
        for (uint32_t t = cl; t < tiles; t += ncl, parity ^= 1u) {
            uint32_t tm, tn;
            grouped_tile(t, tiles_m, tiles_n, tm, tn);
            const int64_t tok0 = int64_t(tm) * 256 + half * 128 + quad * 32, tok = tok0 + lane;
            float acc[CPT];
#pragma unroll
            for (int c = 0; c < CPT; ++c) acc[c] = 0.0f;
            for (int b = 0; b < blocks; ++b) {
                if (live) live = mbar_wait(&done[stage], round & 1u, g.st, 414);
                live = __all_sync(0xFFFFFFFFu, live);
                tc_fence_after();
                const uint32_t dt = tmem_base + (uint32_t(quad * 32) << 16) + slot * TN;
                // a chunk of columns at a time, the next one on its way while this is added
                constexpr int CHUNK = TN == 256 ? 32 : 16, STEPS = CPT / CHUNK;
                auto column = [&](int j) {
                    return dt + (j < STEPS / 2 ? c0 + CHUNK * j : c1 + CHUNK * (j - STEPS / 2));
                };
                uint32_t v[2][CHUNK];
                tmem_ld<CHUNK>(column(0), v[0]);
                const float2 f = ring[(stage + (round & 3u) * C::STAGES) * 128 + r];
                const float f0 = GATED || TN == 128 || part == 0 ? f.x : f.y, f1 = GATED ? f.y : f0;
#pragma unroll
                for (int j = 0; j < STEPS; ++j) {
                    tmem_ld_done(v[j & 1]);
                    if (j + 1 < STEPS) {
                        tmem_ld<CHUNK>(column(j + 1), v[(j + 1) & 1]);
                    } else {                  // this warp has read its part of the accumulator
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster_relaxed(tempty0 + slot * 8u);
                    }
#pragma unroll
                    for (int i = 0; i < CHUNK; i += 2)
                        add_scaled2(acc + CHUNK * j + i, v[j & 1] + i, j < STEPS / 2 ? f0 : f1);
                }
                ++stage;
                mbar_arrive_if(&taken[round & 3u], lane == 0 && stage == C::STAGES);
                if (stage == C::STAGES) { stage = 0; ++round; }
                if (++slot == C::SLOTS) slot = 0;
            }
            // This thread's columns of the output: all of its sums, or of the
            // tile's whole sums a slice (gated: of the gate's and of the up's).
            constexpr int MINE = CPT / SPLIT, OC = GATED ? MINE / 2 : MINE;
            float* v = acc;
            if constexpr (SPLIT > 1) {
                float* sums = reinterpret_cast<float*>(smem);     // [TN][128]; every load and MMA is complete
#pragma unroll
                for (int c = 0; c < CPT; ++c) sums[(part * CPT + c) * 128 + r] = acc[c];
                __syncwarp();
                cluster_sync();
#pragma unroll
                for (int c = 0; c < MINE; ++c) {
                    const int column = part * CPT + int(share) * OC + (c < OC ? c : CPT / 2 + c - OC);
                    acc[c] = 0.0f;
#pragma unroll
                    for (uint32_t q = 0; q < SPLIT; ++q)
                        acc[c] += ld_cluster_f32(mapa_shared(sums + column * 128 + r, 2 * q + half));
                }
            }
            const int64_t col = int64_t(tn) * TILE_N + part * (GATED ? CPT / 2 : CPT) + (SPLIT > 1 ? int(share) * OC : 0);
            if constexpr (!GATED) {
                store_rows_as<OC>(g, out_buf, tok0, col, lane, v);
            } else {
                uint32_t top = 0;
#pragma unroll
                for (int c = 0; c < OC; ++c) {
                    v[c] = gate_act<ACT>(v[c]) * v[OC + c];
                    top = max(top, __float_as_uint(v[c]) & 0x7FFFFFFFu);
                }
                // the block's maximum is over this thread's columns and those of the other parts and pairs
                uint32_t* tops = amax + parity * PARTS * 128;
                tops[part * 128 + r] = top;
                if constexpr (SPLIT > 1) {
                    __syncwarp();
                    cluster_sync();
                } else if (g.out == OUT_CODES) {
                    named_barrier_sync(1, 32 * C::SUM_WARPS);
                }
                if (g.out != OUT_CODES) {
                    store_rows_as<OC>(g, out_buf, tok0, col, lane, v);
                    continue;
                }
#pragma unroll
                for (uint32_t q = 0; q < SPLIT; ++q)
#pragma unroll
                    for (int o = 0; o < PARTS; ++o)
                        top = max(top, SPLIT > 1 ? ld_cluster_u32(mapa_shared(tops + o * 128 + r, 2 * q + half))
                                                 : tops[o * 128 + r]);
                float s = block_scale(top);
                if (part == 0 && share == 0 && tok < g.m) {
                    g.ys[int64_t(tn) * g.ldys + tok] = s;
                    if (top >= INF_BITS) record_error(g.st, GPTQ_ERR_NONFINITE, int(tok));
                }
                if (s < SMALL_SCALE) {
                    s *= SMALL_LIFT;
#pragma unroll
                    for (int c = 0; c < OC; ++c) v[c] *= SMALL_LIFT;
                }
                const Coder code(s, rcp_approx(s));
#pragma unroll
                for (int c = 0; c < OC; c += 16)
                    *reinterpret_cast<uint4*>(out_buf + Stage<OC>::at(lane, c / 16)) =
                        make_uint4(code.four(v + c), code.four(v + c + 4), code.four(v + c + 8), code.four(v + c + 12));
                Stage<OC>::flush(out_buf, static_cast<uint8_t*>(g.y) + tok0 * g.ldy + col, g.ldy,
                                 int(max(int64_t(0), min(g.m - tok0, int64_t(32)))),
                                 int(max(int64_t(0), min(g.n - col, int64_t(OC)))), true, lane);
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync();          // no remote arrival, pair MMA or read of a peer's sums is still pending
    if (warp == C::SUM_WARPS) tmem_dealloc_pair(tmem_base, 512);
}

}  // namespace fp8

namespace {

constexpr int kMaxDev = 64;

// Codes [rows, d] with row pitch ld bytes, 128-byte swizzled boxes of box_rows rows.
int make_code_map(PFN_encodeTiled encode, CUtensorMap* tm, const uint8_t* base, int64_t rows, int64_t d, int64_t ld,
                  uint32_t box_rows) {
    const cuuint64_t dims[2] = {cuuint64_t(d), cuuint64_t(rows)};
    const cuuint64_t strides[1] = {cuuint64_t(ld)};
    const cuuint32_t box[2] = {128, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = encode(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(base), dims, strides, box,
                              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? GPTQ_OK : GPTQ_ERR_CUDA;
}

int sm_count(int dev, int* out) {
    static std::atomic<int> sms[kMaxDev];
    if (dev < 0 || dev >= kMaxDev) return GPTQ_ERR_CUDA;
    int n = sms[dev].load();
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return GPTQ_ERR_CUDA;
        sms[dev].store(n);
    }
    *out = n;
    return GPTQ_OK;
}

// How many clusters of `kernel` with `size` CTAs run at once.
template <typename K>
int resident_clusters(std::atomic<int>& cache, K kernel, int threads, size_t smem, int size, int* out) {
    int n = cache.load();
    if (n == 0) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = unsigned(size);
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3(unsigned(size));
        cfg.blockDim = dim3(unsigned(threads));
        cfg.dynamicSmemBytes = smem;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess)
            return GPTQ_ERR_CUDA;
        n = std::max(1, n);
        cache.store(n);
    }
    *out = n;
    return GPTQ_OK;
}

// p.m is at most NT.
template <int NT, bool GATED, int ACT = 0>
int launch_narrow(const Fp8Product& p, cudaStream_t stream, DevStatus* st, PFN_encodeTiled encode) {
    using C = fp8::Narrow<NT>;
    auto kernel = fp8::narrow_kernel<NT, GATED, ACT>;
    static std::atomic<int> resident[kMaxDev][C::MAX_SPLIT + 1];   // clusters of 1 .. MAX_SPLIT CTAs that run at once
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return GPTQ_ERR_CUDA;
    fp8::Maps maps;
    std::memset(&maps, 0, sizeof(maps));
    int rc = make_code_map(encode, &maps.w, p.w, p.n, p.d, p.ldw, 128);
    if (!rc && GATED) rc = make_code_map(encode, &maps.u, p.u, p.n, p.d, p.ldw, 128);
    if (!rc) rc = make_code_map(encode, &maps.x, p.x, p.m, p.d, p.ldx, NT);
    if (rc) return rc;
    const fp8::Args g{p.m, p.n, p.lds, p.ldy, p.ldys, p.xs, p.ws, p.us, p.y, p.ys, int((p.d + 127) / 128), p.out, st};
    const int64_t rows = (p.n + 127) / 128;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    // CTAs per tile: the most whose clusters all run at once (a cluster stays
    // inside one GPC, so that is less than the CTAs that fit).  8192 x 28672, one
    // token: 64 clusters of 4 take 38 us, of 2 47 us, of 5 (too many) 53 us.
    constexpr int STEP = GATED ? 2 : 1;      // a gated pair's CTAs come in twos
    int split = int(std::min<int64_t>(C::MAX_SPLIT, STEP * g.nkb));
    for (; split > 0; split -= STEP) {
        int n = 0;
        if (resident_clusters(resident[dev][split], kernel, C::THREADS, C::SMEM_BYTES, split, &n)) return GPTQ_ERR_CUDA;
        // (the query counts one CTA that uses TMEM per SM)
        if (split == STEP || rows <= int64_t(n) * C::PER_SM) break;
    }
    cfg.gridDim = dim3(unsigned(rows * split));
    attr[0].val.clusterDim.x = unsigned(split);
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kernel, maps, g) != cudaSuccess) return GPTQ_ERR_CUDA;
    count_launch();
    return GPTQ_OK;
}

template <int TN, bool GATED, int ACT, int SPLIT>
int launch_wide(const Fp8Product& p, cudaStream_t stream, DevStatus* st, PFN_encodeTiled encode) {
    using C = fp8::Wide<TN, SPLIT>;
    auto kernel = fp8::wide_kernel<TN, GATED, ACT, SPLIT>;
    static std::atomic<bool> ready[kMaxDev];
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || sm_count(dev, &sms)) return GPTQ_ERR_CUDA;
    if (!ready[dev].load()) {
        cudaFuncAttributes attr;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(C::SMEM_BYTES)) !=
                cudaSuccess ||
            cudaFuncGetAttributes(&attr, kernel) != cudaSuccess)
            return GPTQ_ERR_CUDA;
        // the kernel's warpgroups exchange registers: more than the launch holds would wait for good
        if (attr.numRegs * C::THREADS < 32 * C::SUM_WARPS * C::SUM_REGS + 128 * C::OTHER_REGS) return GPTQ_ERR_CUDA;
        ready[dev].store(true);
    }
    fp8::Maps maps;
    std::memset(&maps, 0, sizeof(maps));
    int rc = make_code_map(encode, &maps.w, p.w, p.n, p.d, p.ldw, TN / 2);
    if (!rc && GATED) rc = make_code_map(encode, &maps.u, p.u, p.n, p.d, p.ldw, TN / 2);
    if (!rc) rc = make_code_map(encode, &maps.x, p.x, p.m, p.d, p.ldx, 128);
    if (rc) return rc;
    const fp8::Args g{p.m, p.n, p.lds, p.ldy, p.ldys, p.xs, p.ws, p.us, p.y, p.ys, int((p.d + 127) / 128), p.out, st};
    const int64_t tile_n = GATED ? TN / 2 : TN;
    const int64_t tiles = (p.m + 255) / 256 * ((p.n + tile_n - 1) / tile_n);
    const int64_t clusters = SPLIT > 1 ? tiles : std::min<int64_t>(tiles, sms / 2);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(2 * SPLIT * clusters));
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2 * SPLIT;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kernel, maps, g) != cudaSuccess) return GPTQ_ERR_CUDA;
    count_launch();
    return GPTQ_OK;
}

// The SM-pair form of a product: the tile width and the pairs per tile with the
// least estimated time,
//   rounds of tiles x (blocks of k per pair x time of a block + time of a tile),
// which is to rank them, not to tell the time: for the first row below it gives 50
// us for the 256-wide tile by 2 and 70 for the 128-wide by 1.  Its constants follow
// these measurements (us; 256-wide tiles by 1 pair, 128-wide by 1, 256 by 2, 128 by
// 2, 128 by 4):
//   256 tokens, 8192 x 28672    94.7   72.7   64.8   81.3   117
//   256 tokens, 4096 x 4096     19.3   13.5   16.0   12.5   29.1
//   512 tokens, 11008 x 4096    36.0   33.5   48.5   68.1   115
//   512 tokens, 768 x 4096      18.0   12.8   14.7   10.6   9.6
//   300 tokens, 11008 x 256     8.9    7.5    26.1   37.9   83.7
//   4096 tokens, 8192 x 4096    123    146    263    359    645
// and for gated pairs (256 by 1, 2 and 4):
//   64 tokens, 11008 x 4096     34.5   47.9   89.0
//   256 tokens, 2048 x 4096     18.4   15.5   28.5
//   64 tokens, 1024 x 8192      30.2   21.3   18.1
struct WideChoice {
    int tn, split, block_ns, tile_ns;
};
int choose_wide(const Fp8Product& p, WideChoice* out) {
    static std::atomic<int> fours[kMaxDev], eights[kMaxDev];
    int dev = 0, sms = 0, four = 0, eight = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || sm_count(dev, &sms)) return GPTQ_ERR_CUDA;
    using C2 = fp8::Wide<128, 2>;
    using C4 = fp8::Wide<128, 4>;
    if (resident_clusters(fours[dev], fp8::wide_kernel<128, false, 0, 2>, C2::THREADS, C2::SMEM_BYTES, 4, &four) ||
        resident_clusters(eights[dev], fp8::wide_kernel<128, false, 0, 4>, C4::THREADS, C4::SMEM_BYTES, 8, &eight))
        return GPTQ_ERR_CUDA;
    const int64_t nkb = (p.d + 127) / 128, tiles_m = (p.m + 255) / 256;
    const WideChoice plain[5] = {
        {256, 1, 390, 4500}, {128, 1, 310, 800}, {256, 2, 390, 6500}, {128, 2, 310, 3500}, {128, 4, 310, 4500}};
    const WideChoice gated[3] = {{256, 1, 390, 4500}, {256, 2, 390, 6500}, {256, 4, 390, 9000}};
    const WideChoice* c = p.u ? gated : plain;
    int64_t best = -1;
    for (int i = 0; i < (p.u ? 3 : 5); ++i) {
        const int64_t tile_n = p.u ? 128 : c[i].tn, tiles = tiles_m * ((p.n + tile_n - 1) / tile_n);
        const int64_t at_once = std::max(1, c[i].split == 1 ? sms / 2 : c[i].split == 2 ? four : eight);
        if (c[i].split > 1 && tiles > at_once) continue;      // such clusters do not follow one another
        const int64_t rounds = (tiles + at_once - 1) / at_once, blocks = (nkb + c[i].split - 1) / c[i].split;
        const int64_t ns = rounds * (blocks * c[i].block_ns + c[i].tile_ns);
        if (best < 0 || ns < best) {
            best = ns;
            *out = c[i];
        }
    }
    return GPTQ_OK;
}

// Up to this many tokens a product runs with the weights on the MMA's M side: 32
// tokens, 8192 x 28672 41 us against 59 on SM pairs, 11008 x 4096 13.8 against 20.
// The next token pays that step.  Tiles of 64 and 128 tokens with the weights on the
// M side were slower than SM pairs except for the largest weight (64 tokens, 8192 x
// 28672: 50 us against 56), measured with one block of k a stage.
constexpr int64_t kNarrowTokens = 32;

template <int ACT>
int launch_gated(const Fp8Product& p, cudaStream_t stream, DevStatus* st, PFN_encodeTiled encode) {
    if (p.m <= 16) return launch_narrow<16, true, ACT>(p, stream, st, encode);
    if (p.m <= kNarrowTokens) return launch_narrow<32, true, ACT>(p, stream, st, encode);
    WideChoice c;
    if (choose_wide(p, &c)) return GPTQ_ERR_CUDA;
    if (c.split == 4) return launch_wide<256, true, ACT, 4>(p, stream, st, encode);
    if (c.split == 2) return launch_wide<256, true, ACT, 2>(p, stream, st, encode);
    return launch_wide<256, true, ACT, 1>(p, stream, st, encode);
}

}  // namespace

int launch_fp8_product(const Fp8Product& p, cudaStream_t stream, DevStatus* st, PFN_encodeTiled encode) {
    if (p.u)
        return p.act == fp8::SILU ? launch_gated<fp8::SILU>(p, stream, st, encode)
                                  : launch_gated<fp8::GELU>(p, stream, st, encode);
    if (p.m <= 16) return launch_narrow<16, false>(p, stream, st, encode);
    if (p.m <= kNarrowTokens) return launch_narrow<32, false>(p, stream, st, encode);
    WideChoice c;
    if (choose_wide(p, &c)) return GPTQ_ERR_CUDA;
    if (c.tn == 128) {
        if (c.split == 4) return launch_wide<128, false, 0, 4>(p, stream, st, encode);
        if (c.split == 2) return launch_wide<128, false, 0, 2>(p, stream, st, encode);
        return launch_wide<128, false, 0, 1>(p, stream, st, encode);
    }
    if (c.split == 2) return launch_wide<256, false, 0, 2>(p, stream, st, encode);
    return launch_wide<256, false, 0, 1>(p, stream, st, encode);
}

}  // namespace gptq
