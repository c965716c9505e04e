// The whole expert layer for few tokens (1 to 32) in two kernels: router logits, then everything else.
// Blog post "Mixture of Experts (MoEs) in Transformers", section "Expert Backend": dispatch tokens to their experts, run the
// projections, apply the routing weights, collect the results in token order. With few tokens nothing is worth sorting or
// copying: the cost is reading the chosen experts' weights once, plus the latency of every launch on the way.
//
//   logits_t = x_t W_r^T + b;  E_t, w_t = top-k;  h_tj = w_tj silu(x_t Wg_e^T) (x_t Wu_e^T), e = E_t[j];  y_t = sum_j Wd_e h_tj
//
// (the routing weight is applied to h before it is rounded to bf16, which the linear down projection lets through; so all
// experts of a token add up in one accumulator). A shared expert is one more expert that every token chose with weight 1.
//
// few_tokens_kernel is one cooperative launch of one CTA per SM:
//   route    every CTA picks the top-k of all tokens itself, from the logits (a warp per token), and lists the active experts
//            and their tokens in shared memory.
//   gate|up  unit = (active expert, 16 columns of h): 2 x (8 gate and 8 up rows) as the 16 rows of mma.m16n8k16, the expert's
//            tokens as its 8 columns (as many MMAs as it takes), K dealt out to the CTA's 16 warps in steps of 32, their sums
//            added through shared memory. A thread's accumulators hold the gate and the up value of the same column: SwiGLU,
//            then h to the workspace.
//   barrier  over the grid, a counter in the workspace (bounded wait). The first loads of W_down go out before it.
//   down     the (32 output columns) x (active expert, K) steps, laid end to end, are cut into equal ranges, one per CTA: no
//            tail, whatever the routing. A block of columns cut between CTAs is finished by the last of them to arrive, which
//            adds their sums in the CTAs' order: no waiting, the same bits every time.
// Loads: a thread's 16 bytes of a weight row are 8 consecutive k; the 4 threads of a row cover 64 bytes. Which k an MMA's
// column stands for does not matter as long as both operands agree, so those 8 values are used as they come, two MMAs' worth,
// against the same 8 of the token's row: no shuffles. Each thread copies its own operands of the coming steps into its own
// shared memory (cp.async, a ring of STAGES steps) and reads them back itself: no barrier, and the ring runs on across the
// units' ends, with up to 128 KB per SM in flight. (Held in registers, in batches of 4 steps, the loads stopped at every
// batch and unit: 66 us instead of 45 for one token on 4 of 32 experts of 2880 x 2880.)
// What bounds it: HBM once the chosen weights are large (8 tokens on 2 of 8 experts of 4096 x 14336: 370-403 us, 0.98 of a copy's
// rate); below that the way there: two launches (the cooperative one starts some 3.5 us behind the logits), picking the experts
// about 3 us, the barrier about 2. One token on 4 of 32 experts of 2880 x 2880: 45-49 us for 199 MB; on 8 of 256 experts of
// 7168 x 2048 with a shared one: 136-141 us for 800 MB (5.7-5.9 TB/s); 2 tokens on a layer of 256 x 512: 18 us, all of it latency.
#pragma once
#include "common.cuh"
#include "gemm.cuh"
#include "route.cuh"
#include "sync.cuh"

namespace moe {

constexpr int FT_MAX_T = 32;
constexpr int FT_WARPS = 16;
constexpr int FT_THREADS = FT_WARPS * 32;
constexpr int FT_MAX_CTAS = 148;
constexpr int FT_KC = 32;     // k values of a step: 64 bytes of a weight row
// Ring of STAGES steps of (4 + NT) x 8 KB, and a buffer for the warps' sums, RB 16-row blocks of NT x 8 KB at a time. What is left
// of the SM's 227 KB holds the tables. (25 to 32 tokens: the MMAs bound it, 16 per 2 KB of weights; three stages with a smaller
// buffer for the sums measured the same as two.)
template <int NT>
struct FewShape {
    static constexpr int STAGES = NT == 1 ? 4 : (NT == 4 ? 2 : 3);
    static constexpr int RB = NT <= 2 ? 2 : 1;
    static constexpr int RING_BYTES = STAGES * (4 + NT) * FT_WARPS * 32 * 16;
    static constexpr int RED_BYTES = FT_WARPS * RB * NT * 32 * 16;
};
constexpr int FT_LOGIT_THREADS = 256;

// ---- logits: one CTA per expert, fp32, 8 tokens at a time; also clears the counters of the kernel behind it ----
__global__ void __launch_bounds__(FT_LOGIT_THREADS) few_tokens_logits_kernel(const __nv_bfloat16* __restrict__ x,
                                                                            const float* __restrict__ w_router,
                                                                            const float* __restrict__ bias, int T, int d, int E,
                                                                            float* __restrict__ logits, int* counters,
                                                                            int n_counters) {
    __shared__ float red[2][FT_LOGIT_THREADS / 32][8];
    grid_dep_wait();
    grid_dep_trigger();
    const int e = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = e * FT_LOGIT_THREADS + threadIdx.x; i < n_counters; i += gridDim.x * FT_LOGIT_THREADS) counters[i] = 0;
    const float4* w = reinterpret_cast<const float4*>(w_router + (size_t)e * d);
    const float b = bias ? bias[e] : 0.f;
    int turn = 0;
    for (int t0 = 0; t0 < T; t0 += 8, turn ^= 1) {
        float acc[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = 0.f;
        for (int v = threadIdx.x; v < d / 8; v += FT_LOGIT_THREADS) {
            const float4 w0 = __ldg(w + 2 * v), w1 = __ldg(w + 2 * v + 1);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (t0 + i >= T) break;
                const uint4 q = __ldg(reinterpret_cast<const uint4*>(x + (size_t)(t0 + i) * d) + v);
                const float2 a0 = unpack_bf16x2(q.x), a1 = unpack_bf16x2(q.y), a2 = unpack_bf16x2(q.z), a3 = unpack_bf16x2(q.w);
                acc[i] = fmaf(a0.x, w0.x, fmaf(a0.y, w0.y, fmaf(a1.x, w0.z, fmaf(a1.y, w0.w, acc[i]))));
                acc[i] = fmaf(a2.x, w1.x, fmaf(a2.y, w1.y, fmaf(a3.x, w1.z, fmaf(a3.y, w1.w, acc[i]))));
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float s = warp_sum(acc[i]);
            if (lane == 0) red[turn][warp][i] = s;
        }
        __syncthreads();
        if (threadIdx.x < 8 && t0 + (int)threadIdx.x < T) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < FT_LOGIT_THREADS / 32; ++i) s += red[turn][i][threadIdx.x];
            logits[(size_t)(t0 + threadIdx.x) * E + e] = s + b;
        }
    }
}

struct FewArgs {
    const __nv_bfloat16* x;         // [T][d]
    const __nv_bfloat16* w_gateup;  // [E][2f][d]
    const __nv_bfloat16* w_down;    // [E][d][f]
    const __nv_bfloat16* s_gateup;  // [2fs][d] or null
    const __nv_bfloat16* s_down;    // [d][fs]
    const float* logits;            // [T][E]
    int32_t* topk_idx;              // [T][k]
    float* topk_w;                  // [T][k]
    __nv_bfloat16* y;               // [T][d]
    __nv_bfloat16* h;               // workspace [T*k + T][ldh]: row t*k+j, or T*k + t for the shared expert
    float* part;                    // workspace [CTAs][2][32 * 8NT]
    int* counters;                  // workspace [1 + ceil(d/32)], zero
    int T, d, f, fs, E, k, mode, ldh;
};

// Shared memory of few_tokens_kernel besides its reduction buffers, in 4-byte words: slots = T * k.
struct FewTables {
    // idx [slots], w [slots], count [E], place [E] (position among the active experts), active [slots + 1],
    // first [slots + 2] (prefix of the active experts' counts), rows [slots] (slots by active expert), 2 flags, tiles
    // [slots + 1], then as 8-bit [slots + 1][8NT]: which of its k choices the token has the active expert as, or -1
    static __host__ __device__ int words(int slots, int E) {
        return 2 * slots + 2 * E + (slots + 1) + (slots + 2) + slots + 2 + (slots + 1);
    }
};

// D (16 x 8, fp32) += A (16 x 16, bf16) B (16 x 8, bf16)
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Asynchronous copy of 16 bytes to this thread's place in shared memory (zeros where `inside` is false: nothing is read).
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, bool inside) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(inside ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

// warp_route_select (route.cuh) for the logits of one token, the same choices and weights bit for bit, with the warp's arg-max by
// two integer reductions instead of ten shuffles a round (every CTA waits for this). A NaN logit counts as the lowest:
// comparisons with it would leave the warp without a common choice.
__device__ __forceinline__ void few_route_select(const float* l, int E, int k, int mode, int32_t* idx_row, float* w_row) {
    const int lane = threadIdx.x & 31;
    const int per = (E + 31) / 32;
    const auto get = [&](int e) {
        const float v = __ldcg(l + e);
        return v == v ? v : -INFINITY;
    };
    // unsigned keys in the order of the values (+0 and -0 alike), above 0, which stands for nothing left
    const auto key_of = [](float v) {
        const uint32_t u = __float_as_uint(v + 0.f);
        return (u & 0x80000000u) ? ~u : u | 0x80000000u;
    };
    constexpr int RPER = 8;  // up to 256 experts stay in registers
    uint32_t keys[RPER];
    if (per <= RPER) {
#pragma unroll
        for (int s = 0; s < RPER; ++s) {
            const int e = s * 32 + lane;
            keys[s] = s < per && e < E ? key_of(get(e)) : 0u;
        }
    }
    uint32_t taken = 0;
    float my_v = 0.f;
    int my_e = -1;
    for (int j = 0; j < k; ++j) {
        uint32_t best = 0u;
        int best_s = 0;
        if (per <= RPER) {
#pragma unroll
            for (int s = 0; s < RPER; ++s) {
                const uint32_t c = (taken >> s) & 1u ? 0u : keys[s];
                if (c > best) best = c, best_s = s;  // ascending ids: '>' keeps the lower one
            }
        } else {
            for (int s = 0; s < per; ++s) {
                const int e = s * 32 + lane;
                const uint32_t c = e < E && !((taken >> s) & 1u) ? key_of(get(e)) : 0u;
                if (c > best) best = c, best_s = s;
            }
        }
        const uint32_t top = __reduce_max_sync(0xffffffffu, best);
        const int e = (int)__reduce_min_sync(0xffffffffu, best == top ? (uint32_t)(best_s * 32 + lane) : 0xffffffffu);
        if ((e & 31) == lane) taken |= 1u << (e >> 5);
        if (lane == j) {
            my_e = e;
            my_v = __uint_as_float(top & 0x80000000u ? top ^ 0x80000000u : ~top);
        }
    }
    const bool mine = lane < k;
    const float vmax = __shfl_sync(0xffffffffu, my_v, 0);
    float w = 0.f;
    if (mode == MOE_ROUTE_SIGMOID_TOPK_NORM) {
        const float s = mine ? 1.f / (1.f + expf(-my_v)) : 0.f;
        w = s / warp_sum(s);
    } else {
        const float ex = mine ? expf(my_v - vmax) : 0.f;
        const float zsel = warp_sum(ex);
        if (mode == MOE_ROUTE_SOFTMAX_TOPK_RENORM) {
            float part = 0.f;
            for (int s = 0; s < per; ++s) {
                const int e = s * 32 + lane;
                if (e < E) part += expf(get(e) - vmax);
            }
            const float zall = warp_sum(part);
            const float p = ex / zall;  // probability under the full softmax
            w = p / warp_sum(p);
        } else {
            w = ex / zsel;
        }
    }
    if (mine) {
        idx_row[lane] = my_e;
        w_row[lane] = w;
    }
}

// Wait until all CTAs of the grid have arrived on *counter (zero at the start). False when the wait ran out.
__device__ __forceinline__ bool grid_barrier(int* counter, int* s_flag) {
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        atomicAdd(counter, 1);
        const uint64_t t0 = globaltimer_ns(), limit = wait_limit_ns();
        // (the test hook moe_test_set_wait: one arrival more than there are)
        const int want = (int)gridDim.x + (*reinterpret_cast<volatile int*>(&g_wait_stall) != 0 ? 1 : 0);
        int ok = 1, seen;
        for (;;) {
            asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(seen) : "l"(counter) : "memory");
            if (seen >= want) break;
            if (globaltimer_ns() - t0 > limit) {
                flag_error(MOE_DEVERR_WAIT_TIMEOUT);
                ok = 0;
                break;
            }
        }
        __threadfence();
        *s_flag = ok;
    }
    __syncthreads();
    return *s_flag != 0;
}

// One element of the down projection over the steps s0 .. s1 of its block of output columns, from the experts that the token chose
// and no others: choice[a * pitch], as which of its k choices it has the active expert a (or -1).
//
// In the MMAs a token without the expert has zeros in its column, and zero times an infinity or NaN among that expert's weights is NaN
// where the formula has no term at all. That always shows as a NaN in the sum (never as an infinity, nor as a wrong number), so a sum
// that is NaN, and only that, is made again here: finite weights cost one comparison per output (46.0 us with and without). One thread, in order, until
// the sum is NaN by itself: at its first term for a token that holds NaN, such as the unused rows of a padded batch.
__device__ __forceinline__ float few_down_of_chosen(const FewArgs& p, const int* active, int A, const int8_t* choice, int pitch, int t,
                                                 int column, int s0, int s1) {
    const int fsteps = (p.f + FT_KC - 1) / FT_KC;
    float sum = 0.f;
    for (int a = min(s0 / fsteps, A); a <= A; ++a) {
        const int first = a * fsteps;  // the expert's first step; the shared one's run on to the block's end
        if (first >= s1) break;
        const int j = choice[a * pitch];
        if (j < 0) continue;
        const int K = a < A ? p.f : p.fs;
        const int k0 = max(s0 - first, 0) * FT_KC, k1 = min((s1 - first) * FT_KC, K);
        const __nv_bfloat16* w = (a < A ? p.w_down + (size_t)active[a] * p.d * p.f : p.s_down) + (size_t)column * K;
        const __nv_bfloat16* h = p.h + (size_t)(a < A ? t * p.k + j : p.T * p.k + t) * p.ldh;
        for (int k = k0; k < k1 && sum == sum; k += 8) {
            const uint4 wv = *reinterpret_cast<const uint4*>(w + k), hv = __ldcg(reinterpret_cast<const uint4*>(h + k));
            const uint32_t wu[4] = {wv.x, wv.y, wv.z, wv.w}, hu[4] = {hv.x, hv.y, hv.z, hv.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 x = unpack_bf16x2(wu[i]), y = unpack_bf16x2(hu[i]);
                sum = fmaf(x.y, y.y, fmaf(x.x, y.x, sum));
            }
        }
    }
    return sum;
}

template <int NT>
__global__ void __launch_bounds__(FT_THREADS, 1) few_tokens_kernel(const __grid_constant__ FewArgs p) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    using S = FewShape<NT>;
    constexpr int STAGES = S::STAGES, RB = S::RB, SLOT_BYTES = FT_THREADS * 16, STAGE_BYTES = (4 + NT) * SLOT_BYTES;
    const uint32_t ring = smem_u32(smem_raw) + threadIdx.x * 16;  // this thread's 16 bytes of slot 0, stage 0
    float4* red = reinterpret_cast<float4*>(smem_raw + S::RING_BYTES);  // [warp][RB][NT][lane]
    int* words = reinterpret_cast<int*>(smem_raw + S::RING_BYTES + S::RED_BYTES);
    const int slots = p.T * p.k;
    int* s_idx = words;
    float* s_w = reinterpret_cast<float*>(s_idx + slots);
    int* s_rank = reinterpret_cast<int*>(red);  // [slots] until the first sums
    int* s_count = s_idx + 2 * slots;
    int* s_place = s_count + p.E;
    int* s_active = s_place + p.E;
    int* s_first = s_active + slots + 1;
    int* s_rows = s_first + slots + 2;
    int* s_n = s_rows + slots;  // number of active experts; flag of the barrier and of the last arrival
    int* s_tiles = s_n + 2;       // [slots + 1] bit n: the active expert has a token among tokens 8n .. 8n + 7
    int8_t* s_choice = reinterpret_cast<int8_t*>(words + FewTables::words(slots, p.E));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t4 = lane & 3;
    const int T = p.T;

    grid_dep_wait();  // the logits

    // ---- route ----
    for (int t = warp; t < T; t += FT_WARPS) few_route_select(p.logits + (size_t)t * p.E, p.E, p.k, p.mode, s_idx + t * p.k, s_w + t * p.k);
    for (int e = threadIdx.x; e < p.E; e += FT_THREADS) s_count[e] = 0;
    for (int i = threadIdx.x; i < (slots + 1) * 8 * NT; i += FT_THREADS) s_choice[i] = -1;
    for (int i = threadIdx.x; i <= slots; i += FT_THREADS) s_tiles[i] = 0;
    __syncthreads();
    for (int s = threadIdx.x; s < slots; s += FT_THREADS) {
        const int e = s_idx[s];
        int rank = 0;
        for (int i = 0; i < s; ++i) rank += s_idx[i] == e;
        s_rank[s] = rank;
        atomicAdd(&s_count[e], 1);
        if (blockIdx.x == 0) {
            p.topk_idx[s] = e;
            p.topk_w[s] = s_w[s];
        }
    }
    __syncthreads();
    if (warp == 0) {  // the active experts, in the order in which the slots name them first
        int n = 0, rows = 0;
        for (int s0 = 0; s0 < slots; s0 += 32) {
            const int s = s0 + lane;
            const bool first = s < slots && s_rank[s] == 0;
            const int e = first ? s_idx[s] : 0;
            const int c = first ? s_count[e] : 0;
            const unsigned m = __ballot_sync(0xffffffffu, first);
            int upto = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += v;
            }
            if (first) {
                const int at = n + __popc(m & lanemask_lt());
                s_active[at] = e;
                s_place[e] = at;
                s_first[at] = rows + upto - c;
            }
            n += __popc(m);
            rows += __shfl_sync(0xffffffffu, upto, 31);
        }
        if (lane == 0) {
            s_first[n] = rows;
            s_n[0] = n;
        }
    }
    __syncthreads();
    const int A = s_n[0];
    for (int s = threadIdx.x; s < slots; s += FT_THREADS) {
        const int at = s_place[s_idx[s]];
        s_rows[s_first[at] + s_rank[s]] = s;
        s_choice[at * 8 * NT + s / p.k] = (int8_t)(s % p.k);
        atomicOr(&s_tiles[at], 1 << (s / p.k / 8));
    }
    if (p.fs)
        for (int t = threadIdx.x; t < T; t += FT_THREADS) {
            s_choice[A * 8 * NT + t] = 0;
            atomicOr(&s_tiles[A], 1 << (t / 8));
        }
    __syncthreads();

    // The operands of a ring stage: A (weights) in slots 2m (MMA rows 0-7 of block m) and 2m + 1 (rows 8-15), B (the tokens'
    // rows) in slot 4 + n.
    float acc[2][NT][4];
    auto clear = [&] {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;
    };
    auto multiply = [&](uint32_t at, int tiles) {  // one step from the stage at `at`
        uint4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = ld_shared_16(at + i * SLOT_BYTES);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (NT > 1 && !((tiles >> n) & 1)) continue;
            const uint4 b = ld_shared_16(at + (4 + n) * SLOT_BYTES);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                mma_bf16(acc[m][n], w[2 * m].x, w[2 * m + 1].x, w[2 * m].y, w[2 * m + 1].y, b.x, b.y);
                mma_bf16(acc[m][n], w[2 * m].z, w[2 * m + 1].z, w[2 * m].w, w[2 * m + 1].w, b.z, b.w);
            }
        }
    };
    auto publish = [&](int tiles, int m0) {  // this warp's sums of RB blocks from m0, for the CTA to add
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
                if (m >= m0 && m < m0 + RB && (NT == 1 || (tiles >> n) & 1))
                    red[((warp * RB + m - m0) * NT + n) * 32 + lane] =
                        make_float4(acc[m][n][0], acc[m][n][1], acc[m][n][2], acc[m][n][3]);
    };
    const float* rf = reinterpret_cast<const float*>(red);
    // MMA row `row` (0-15) and column `col` of the m-th block in `red`, token block n, of warp q
    auto element = [&](int q, int m, int n, int row, int col) {
        return rf[((((q * RB + m) * NT + n) * 32) + (row & 7) * 4 + (col >> 1)) * 4 + (row >> 3) * 2 + (col & 1)];
    };

    // ---- gate|up ----
    {
        const int fb = (p.f + 15) >> 4, sb = (p.fs + 15) >> 4;
        const int units = A * fb + sb;
        const int steps = (p.d + FT_KC - 1) / FT_KC;
        // step i of the CTA's n-th unit goes to warp (n steps + i) mod 16
        auto first_step = [&](int n) { return (warp - n * steps) & (FT_WARPS - 1); };
        // the copies run ahead of the sums: unit pu (the CTA's pn-th), step pc
        int pu = blockIdx.x, pn = 0, pc = first_step(0), p_stage = 0, p_used = 0;
        const __nv_bfloat16 *lo = nullptr, *x_row[NT];
        size_t up = 0;       // from a gate row to its up row
        bool second = false;  // the unit's second 8 columns exist
        bool fresh = true;
        auto issue = [&] {
            while (pu < units && pc >= steps) {
                pu += gridDim.x;
                pc = first_step(++pn);
                fresh = true;
            }
            if (pu < units) {
                if (fresh) {
                    fresh = false;
                    const int a = pu / fb;
                    const bool routed = pu < A * fb;
                    const int j0 = (pu - (routed ? a : A) * fb) * 16, cols = routed ? p.f : p.fs;
                    lo = (routed ? p.w_gateup + (size_t)s_active[a] * 2 * p.f * p.d : p.s_gateup) + (size_t)(j0 + g) * p.d + t4 * 8;
                    up = (size_t)cols * p.d;
                    second = j0 + 8 < cols;
                    const int count = routed ? s_first[a + 1] - s_first[a] : T;
                    p_used = (count + 7) / 8;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const int col = n * 8 + g;
                        x_row[n] = nullptr;
                        if (col < count) x_row[n] = p.x + (size_t)(routed ? s_rows[s_first[a] + col] / p.k : col) * p.d + t4 * 8;
                    }
                }
                const int k0 = pc * FT_KC;
                const bool in = k0 + t4 * 8 < p.d;
                const uint32_t to = ring + p_stage * STAGE_BYTES;
                const __nv_bfloat16* row = lo + (in ? k0 : 0);
                cp_async_16(to, row, in);
                cp_async_16(to + SLOT_BYTES, row + up, in);
                const size_t next8 = second ? (size_t)8 * p.d : 0;
                cp_async_16(to + 2 * SLOT_BYTES, row + next8, in && second);
                cp_async_16(to + 3 * SLOT_BYTES, row + next8 + up, in && second);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    if (n < p_used) cp_async_16(to + (4 + n) * SLOT_BYTES, x_row[n] ? x_row[n] + (in ? k0 : 0) : p.x, in && x_row[n]);
                pc += FT_WARPS;
            }
            cp_async_commit();
            if (++p_stage == STAGES) p_stage = 0;
        };
#pragma unroll
        for (int i = 0; i < STAGES - 1; ++i) issue();
        int stage = 0;
        for (int u = blockIdx.x, n_unit = 0; u < units; u += gridDim.x, ++n_unit) {
            const int a = u / fb;
            const bool routed = u < A * fb;
            const int count = routed ? s_first[a + 1] - s_first[a] : T;
            const int used = (count + 7) / 8, tiles = (1 << used) - 1;
            clear();
            for (int c = first_step(n_unit); c < steps; c += FT_WARPS) {
                issue();  // into the stage of the step before
                cp_async_wait<STAGES - 1>();
                multiply(ring + stage * STAGE_BYTES, tiles);
                if (++stage == STAGES) stage = 0;
            }
#pragma unroll
            for (int m0 = 0; m0 < 2; m0 += RB) {
                publish(tiles, m0);
                __syncthreads();
                for (int i = threadIdx.x; i < 64 * RB * used; i += FT_THREADS) {
                    const int n = i / (64 * RB), m = (i >> 6) % RB, j = (i >> 3) & 7, col = i & 7;
                    const int j0 = (u - (routed ? a : A) * fb) * 16 + (m0 + m) * 8 + j, at = n * 8 + col;
                    if (at >= count || j0 >= (routed ? p.f : p.fs)) continue;
                    float gate = 0.f, upv = 0.f;
#pragma unroll
                    for (int q = 0; q < FT_WARPS; ++q) {
                        gate += element(q, m, n, j, col);
                        upv += element(q, m, n, j + 8, col);
                    }
                    float h = swiglu(gate, upv);
                    int s = slots + at;
                    if (routed) {
                        s = s_rows[s_first[a] + at];
                        h *= s_w[s];
                    }
                    p.h[(size_t)s * p.ldh + j0] = __float2bfloat16_rn(h);
                }
                __syncthreads();
            }
        }
        cp_async_wait<0>();
    }

    // ---- down ----
    {
        const int fsteps = (p.f + FT_KC - 1) / FT_KC, ssteps = (p.fs + FT_KC - 1) / FT_KC;
        const int per = A * fsteps + ssteps;  // steps of a block of 32 output columns
        const int blocks = (p.d + 31) / 32;
        const int all = per * blocks;
        const int r0 = (int)((long)all * blockIdx.x / gridDim.x), r1 = (int)((long)all * (blockIdx.x + 1) / gridDim.x);
        // where step r lies: column block cb, active expert a (A: the shared one), K step c; 16 further on
        struct Place {
            int cb, a, c;
        };
        auto place = [&](int r) {
            Place at;
            at.cb = r / per;
            const int s = r - at.cb * per;
            at.a = min(s / fsteps, A);
            at.c = s - at.a * fsteps;
            return at;
        };
        auto advance = [&](Place& at) {
            at.c += FT_WARPS;
            for (int len = at.a < A ? fsteps : ssteps; at.c >= len; len = at.a < A ? fsteps : ssteps) {
                at.c -= len;
                if (++at.a > A) {  // past the shared expert's (perhaps no) steps
                    at.a = 0;
                    ++at.cb;
                }
            }
        };
        auto issue_weights = [&](const Place& at, int stage) {
            const int K = at.a < A ? p.f : p.fs, k = at.c * FT_KC + t4 * 8, row = at.cb * 32 + g;
            const __nv_bfloat16* m = at.a < A ? p.w_down + (size_t)s_active[at.a] * p.d * p.f : p.s_down;
            const uint32_t to = ring + stage * STAGE_BYTES;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool in = k < K && row + 8 * i < p.d;
                cp_async_16(to + i * SLOT_BYTES, in ? m + (size_t)(row + 8 * i) * K + k : p.x, in);
            }
        };
        auto issue_h = [&](const Place& at, int stage) {
            const int K = at.a < A ? p.f : p.fs, k = at.c * FT_KC + t4 * 8;
            const int tiles = s_tiles[at.a];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (NT > 1 && !((tiles >> n) & 1)) continue;
                const int choice = s_choice[at.a * 8 * NT + n * 8 + g];
                const int slot = at.a < A ? (n * 8 + g) * p.k + choice : slots + n * 8 + g;
                const bool in = choice >= 0 && k < K;
                cp_async_16(ring + stage * STAGE_BYTES + (4 + n) * SLOT_BYTES, in ? p.h + (size_t)slot * p.ldh + k : p.h, in);
            }
        };
        int pr = r0 + warp;
        Place ahead = place(min(pr, all - 1)), at = ahead;
        {
            Place b = ahead;
#pragma unroll
            for (int i = 0; i < STAGES - 1; ++i) {
                if (pr + i * FT_WARPS < r1) {
                    issue_weights(b, i);
                    advance(b);
                }
                cp_async_commit();
            }
        }
        if (!grid_barrier(p.counters, s_n + 1)) {
            cp_async_wait<0>();
            return;
        }
#pragma unroll
        for (int i = 0; i < STAGES - 1; ++i) {
            if (pr < r1) {
                issue_h(ahead, i);
                advance(ahead);
            }
            pr += FT_WARPS;
        }
        cp_async_commit();
        cp_async_wait<0>();
        int stage = 0, p_stage = STAGES - 1;
        int r = r0 + warp;
        const int cb_first = r0 / per;
        for (int cb = cb_first, begin = r0; begin < r1; ++cb) {
            const int end = (int)min((long)r1, (long)(cb + 1) * per);
            clear();
            for (; r < end; r += FT_WARPS) {
                if (pr < r1) {
                    issue_weights(ahead, p_stage);
                    issue_h(ahead, p_stage);
                    advance(ahead);
                }
                cp_async_commit();
                pr += FT_WARPS;
                if (++p_stage == STAGES) p_stage = 0;
                cp_async_wait<STAGES - 1>();
                multiply(ring + stage * STAGE_BYTES, s_tiles[at.a]);
                advance(at);
                if (++stage == STAGES) stage = 0;
            }
            const bool whole = end - begin == per;
            constexpr int OUT = 256 * NT;  // (token, column) values: i = token * 32 + column
            float* mine = p.part + ((size_t)blockIdx.x * 2 + (cb == cb_first ? 0 : 1)) * OUT;
#pragma unroll
            for (int m0 = 0; m0 < 2; m0 += RB) {
                publish((1 << NT) - 1, m0);
                __syncthreads();
                for (int i = threadIdx.x; i < 128 * RB * NT; i += FT_THREADS) {
                    const int t = i / (16 * RB), col = i % (16 * RB), c = m0 * 16 + col;
                    if (t >= T || cb * 32 + c >= p.d) continue;
                    float v = 0.f;
#pragma unroll
                    for (int q = 0; q < FT_WARPS; ++q) v += element(q, col >> 4, t >> 3, col & 15, t & 7);
                    if (v != v) v = few_down_of_chosen(p, s_active, A, s_choice + t, 8 * NT, t, cb * 32 + c, begin - cb * per, end - cb * per);
                    if (whole)
                        p.y[(size_t)t * p.d + cb * 32 + c] = __float2bfloat16_rn(v);
                    else
                        mine[t * 32 + c] = v;
                }
                __syncthreads();
            }
            if (!whole) {  // cut between CTAs: the last one to arrive adds the parts in their order
                const long x0 = (long)cb * per, x1 = x0 + per - 1;
                const int b0 = (int)(((x0 + 1) * gridDim.x - 1) / all), b1 = (int)(((x1 + 1) * gridDim.x - 1) / all);
                __threadfence();
                __syncthreads();
                if (threadIdx.x == 0) s_n[1] = atomicAdd(p.counters + 1 + cb, 1) == b1 - b0;
                __syncthreads();
                if (s_n[1]) {
                    __threadfence();
                    for (int i = threadIdx.x; i < OUT; i += FT_THREADS) {
                        const int t = i >> 5, col = i & 31;
                        if (t >= T || cb * 32 + col >= p.d) continue;
                        float v = 0.f;
                        for (int q = b0; q <= b1; ++q) {
                            const int which = (int)((long)all * q / gridDim.x) / per == cb ? 0 : 1;
                            v += __ldcg(p.part + ((size_t)q * 2 + which) * OUT + i);
                        }
                        p.y[(size_t)t * p.d + cb * 32 + col] = __float2bfloat16_rn(v);
                    }
                }
            }
            __syncthreads();
            begin = end;
        }
        cp_async_wait<0>();
    }
}

}  // namespace moe
