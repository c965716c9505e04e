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
//   gate|up  unit = (active expert, 8 columns of h): 8 gate and 8 up rows as the 16 rows of mma.m16n8k16, the expert's tokens
//            as its 8 columns (as many MMAs as it takes), K split over the CTA's 16 warps, summed through shared memory. A
//            thread's accumulators hold the gate and the up value of the same column: SwiGLU, then h to the workspace.
//   barrier  over the grid, a counter in the workspace (bounded wait). Each warp's first loads of W_down go out before it.
//   down     the (16 output columns) x (active expert, K) steps, laid end to end, are cut into equal ranges, one per CTA: no
//            tail, whatever the routing. A block of columns cut between CTAs is finished by the last of them to arrive, which
//            adds their sums in the CTAs' order: no waiting, the same bits every time.
// Loads: a thread's 16 bytes of a weight row are 8 consecutive k; the 4 threads of a row cover 64 bytes. Which k an MMA's
// column stands for does not matter as long as both operands agree, so those 8 values are used as they come, two MMAs' worth,
// against the same 8 of the token's row: no shuffles, no shared memory for weights. Two batches of 4 such loads x 2 rows per
// thread are in flight (up to 128 KB per SM).
#pragma once
#include "common.cuh"
#include "gemm.cuh"
#include "route.cuh"

namespace moe {

constexpr int FT_MAX_T = 32;
constexpr int FT_WARPS = 16;
constexpr int FT_THREADS = FT_WARPS * 32;
constexpr int FT_MAX_CTAS = 148;
constexpr int FT_KC = 32;     // k values of a step: 64 bytes of a weight row
constexpr int FT_BATCH = 4;   // steps a warp loads together
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
    float* part;                    // workspace [CTAs][2][16 * 8NT]
    int* counters;                  // workspace [1 + ceil(d/16)], zero
    int T, d, f, fs, E, k, mode, ldh;
};

// Shared memory of few_tokens_kernel besides its reduction buffers, in 4-byte words: slots = T * k.
struct FewTables {
    // idx [slots], w [slots], rank [slots], count [E], place [E] (position among the active experts), active [slots + 1],
    // first [slots + 2] (prefix of the active experts' counts), rows [slots] (slots by active expert), then slot_of as 16-bit:
    // [slots + 1][8NT] slot of (active expert, token) or -1
    static __host__ __device__ int words(int slots, int E) { return 3 * slots + 2 * E + (slots + 1) + (slots + 2) + slots + 2; }
};

// D (16 x 8, fp32) += A (16 x 16, bf16) B (16 x 8, bf16)
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Weights are read once: not kept in L1.
__device__ __forceinline__ uint4 ld_weight(const __nv_bfloat16* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Wait until all CTAs of the grid have arrived on *counter (zero at the start). False when the wait ran out.
__device__ __forceinline__ bool grid_barrier(int* counter, int* s_flag) {
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        atomicAdd(counter, 1);
        const uint64_t t0 = globaltimer_ns(), limit = wait_limit_ns();
        int ok = 1, seen;
        for (;;) {
            asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(seen) : "l"(counter) : "memory");
            if (seen >= (int)gridDim.x) break;
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

template <int NT>
__global__ void __launch_bounds__(FT_THREADS, 1) few_tokens_kernel(const FewArgs p) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    constexpr int RED = FT_WARPS * NT * 32;                     // float4 per reduction buffer
    float4* red = reinterpret_cast<float4*>(smem_raw);          // [2][warp][NT][lane]
    int* words = reinterpret_cast<int*>(red + 2 * RED);
    const int slots = p.T * p.k;
    int* s_idx = words;
    float* s_w = reinterpret_cast<float*>(s_idx + slots);
    int* s_rank = s_idx + 2 * slots;
    int* s_count = s_rank + slots;
    int* s_place = s_count + p.E;
    int* s_active = s_place + p.E;
    int* s_first = s_active + slots + 1;
    int* s_rows = s_first + slots + 2;
    int* s_n = s_rows + slots;  // number of active experts; flag of the barrier and of the last arrival
    int16_t* s_slot = reinterpret_cast<int16_t*>(words + FewTables::words(slots, p.E));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t4 = lane & 3;
    const int T = p.T;

    // ---- route ----
    for (int t = warp; t < T; t += FT_WARPS) {
        // a NaN logit counts as the lowest: comparisons with it would leave the warp without a common choice
        const float* l = p.logits + (size_t)t * p.E;
        const auto logit = [=](int e) {
            const float v = l[e];
            return v == v ? v : -INFINITY;
        };
        warp_route_select(logit, p.E, p.k, p.mode, s_idx + t * p.k, s_w + t * p.k);
    }
    for (int e = threadIdx.x; e < p.E; e += FT_THREADS) s_count[e] = 0;
    for (int i = threadIdx.x; i < (slots + 1) * 8 * NT; i += FT_THREADS) s_slot[i] = -1;
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
    if (warp == 0) {  // the active experts in ascending order
        int n = 0, rows = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int c = e0 + lane < p.E ? s_count[e0 + lane] : 0;
            const unsigned m = __ballot_sync(0xffffffffu, c > 0);
            int before = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, before, o);
                if (lane >= o) before += v;
            }
            if (c > 0) {
                const int at = n + __popc(m & lanemask_lt());
                s_active[at] = e0 + lane;
                s_place[e0 + lane] = at;
                s_first[at] = rows + before - c;
            }
            n += __popc(m);
            rows += __shfl_sync(0xffffffffu, before, 31);
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
        s_slot[at * 8 * NT + s / p.k] = (int16_t)s;
    }
    if (p.fs)
        for (int t = threadIdx.x; t < T; t += FT_THREADS) s_slot[A * 8 * NT + t] = (int16_t)(slots + t);
    __syncthreads();

    // ---- gate|up ----
    {
        const int fb = p.f >> 3;
        const int units = A * fb + (p.fs >> 3);
        const int steps = (p.d + FT_KC - 1) / FT_KC;
        // a warp's batches: unit u, steps c, c + 16, c + 32, c + 48
        int u = blockIdx.x, c = warp;
        const __nv_bfloat16 *lo = nullptr, *hi = nullptr;
        auto rows_of = [&](int unit) {
            if (unit < A * fb) {
                const int a = unit / fb;
                lo = p.w_gateup + ((size_t)s_active[a] * 2 * p.f + (unit - a * fb) * 8 + g) * p.d + t4 * 8;
                hi = lo + (size_t)p.f * p.d;
            } else {
                lo = p.s_gateup + ((size_t)(unit - A * fb) * 8 + g) * p.d + t4 * 8;
                hi = lo + (size_t)p.fs * p.d;
            }
        };
        auto fetch = [&](int from, uint4 (&w)[FT_BATCH][2]) {
#pragma unroll
            for (int i = 0; i < FT_BATCH; ++i) {
                const int k0 = (from + i * FT_WARPS) * FT_KC;
                w[i][0] = w[i][1] = make_uint4(0, 0, 0, 0);
                if (k0 + t4 * 8 < p.d) {
                    w[i][0] = ld_weight(lo + k0);
                    w[i][1] = ld_weight(hi + k0);
                }
            }
        };
        uint4 w[FT_BATCH][2], wn[FT_BATCH][2];
        float acc[NT][4];
        int turn = 0;
        if (u < units) {
            rows_of(u);
            fetch(c, w);
        }
        bool fresh = true;
        int count = 0, nt_used = 0;
        const __nv_bfloat16* xr[NT];
        while (u < units) {
            if (fresh) {
                const int a = u / fb;
                const bool routed = u < A * fb;
                count = routed ? s_first[a + 1] - s_first[a] : T;
                nt_used = (count + 7) / 8;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int col = n * 8 + g;
                    xr[n] = nullptr;
                    if (col < count) xr[n] = p.x + (size_t)(routed ? s_rows[s_first[a] + col] / p.k : col) * p.d + t4 * 8;
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
                }
            }
            const int u0 = u, c0 = c;
            c += FT_BATCH * FT_WARPS;
            if (c >= steps) {
                u += gridDim.x;
                c = warp;
                if (u < units) rows_of(u);
            }
            if (u < units) fetch(c, wn);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (n >= nt_used) break;
                uint4 b[FT_BATCH];
#pragma unroll
                for (int i = 0; i < FT_BATCH; ++i) {
                    const int k0 = (c0 + i * FT_WARPS) * FT_KC;
                    b[i] = make_uint4(0, 0, 0, 0);
                    if (xr[n] && k0 + t4 * 8 < p.d) b[i] = __ldg(reinterpret_cast<const uint4*>(xr[n] + k0));
                }
#pragma unroll
                for (int i = 0; i < FT_BATCH; ++i) {
                    mma_bf16(acc[n], w[i][0].x, w[i][1].x, w[i][0].y, w[i][1].y, b[i].x, b[i].y);
                    mma_bf16(acc[n], w[i][0].z, w[i][1].z, w[i][0].w, w[i][1].w, b[i].z, b[i].w);
                }
            }
            fresh = u != u0;
            if (fresh) {  // the unit's sums: through shared memory, then SwiGLU
                float4* r = red + turn * RED;
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    if (n < nt_used) r[(warp * NT + n) * 32 + lane] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
                __syncthreads();
                const float* rf = reinterpret_cast<const float*>(r);
                for (int i = threadIdx.x; i < 64 * nt_used; i += FT_THREADS) {
                    const int n = i >> 6, j = (i >> 3) & 7, col = i & 7;
                    if (n * 8 + col >= count) continue;
                    float gate = 0.f, up = 0.f;
#pragma unroll
                    for (int q = 0; q < FT_WARPS; ++q) {
                        const float* v = rf + (((q * NT + n) * 32) + j * 4 + (col >> 1)) * 4 + (col & 1);
                        gate += v[0];
                        up += v[2];
                    }
                    const int a = u0 / fb;
                    if (u0 < A * fb) {
                        const int s = s_rows[s_first[a] + n * 8 + col];
                        p.h[(size_t)s * p.ldh + (u0 - a * fb) * 8 + j] = __float2bfloat16_rn(s_w[s] * swiglu(gate, up));
                    } else {
                        p.h[(size_t)(slots + n * 8 + col) * p.ldh + (u0 - A * fb) * 8 + j] = __float2bfloat16_rn(swiglu(gate, up));
                    }
                }
                turn ^= 1;
            }
#pragma unroll
            for (int i = 0; i < FT_BATCH; ++i) {
                w[i][0] = wn[i][0];
                w[i][1] = wn[i][1];
            }
        }
    }

    // ---- down ----
    const int fsteps = (p.f + FT_KC - 1) / FT_KC, ssteps = (p.fs + FT_KC - 1) / FT_KC;
    const int per = A * fsteps + ssteps;  // steps of a block of 16 output columns
    const int blocks = (p.d + 15) / 16;
    const long all = (long)per * blocks;
    const long r0 = all * blockIdx.x / gridDim.x, r1 = all * (blockIdx.x + 1) / gridDim.x;
    // step s of column block cb -> this thread's weight pointers (null past the matrix) and k
    auto fetch = [&](int cb, int s, int s_end, uint4 (&w)[FT_BATCH][2]) {
#pragma unroll
        for (int i = 0; i < FT_BATCH; ++i) {
            const int st = s + i * FT_WARPS;
            w[i][0] = w[i][1] = make_uint4(0, 0, 0, 0);
            if (st < s_end) {
                const int a = min(st / fsteps, A);
                const int K = a < A ? p.f : p.fs;
                const int k = (st - a * fsteps) * FT_KC + t4 * 8;
                if (k < K) {
                    const __nv_bfloat16* m = a < A ? p.w_down + (size_t)s_active[a] * p.d * p.f : p.s_down;
                    const int row = cb * 16 + g;
                    w[i][0] = ld_weight(m + (size_t)row * K + k);
                    if (row + 8 < p.d) w[i][1] = ld_weight(m + (size_t)(row + 8) * K + k);
                }
            }
        }
    };
    uint4 w[FT_BATCH][2], wn[FT_BATCH][2];
    int cb = (int)(r0 / per);
    int s_begin = (int)(r0 - (long)cb * per), s_end = (int)min((long)per, s_begin + (r1 - r0));
    const int cb_first = cb;
    if (r0 < r1) fetch(cb, s_begin + warp, s_end, w);
    if (!grid_barrier(p.counters, s_n + 1)) return;
    int turn = 0;
    int s = s_begin + warp;
    float acc[NT][4] = {};
    long left = r1 - r0;  // steps of the CTA's range from s_begin on
    while (left > 0) {
        // the next batch: of this column block, or the first of the next one
        const int cb0 = cb, s0 = s, s_end0 = s_end, s_begin0 = s_begin;
        const bool last = s_begin + FT_BATCH * FT_WARPS * ((s - s_begin) / (FT_BATCH * FT_WARPS) + 1) >= s_end;
        s += FT_BATCH * FT_WARPS;
        if (last) {
            left -= s_end - s_begin;
            ++cb;
            s_begin = 0;
            s_end = (int)min((long)per, left);
            s = warp;
        }
        if (left > 0) fetch(cb, s, s_end, wn);
        uint4 b[FT_BATCH];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < FT_BATCH; ++i) {
                const int st = s0 + i * FT_WARPS;
                b[i] = make_uint4(0, 0, 0, 0);
                if (st < s_end0) {
                    const int a = min(st / fsteps, A);
                    const int k = (st - a * fsteps) * FT_KC + t4 * 8;
                    const int slot = s_slot[a * 8 * NT + n * 8 + g];
                    if (slot >= 0 && k < (a < A ? p.f : p.fs))
                        b[i] = *reinterpret_cast<const uint4*>(p.h + (size_t)slot * p.ldh + k);
                }
            }
#pragma unroll
            for (int i = 0; i < FT_BATCH; ++i) {
                mma_bf16(acc[n], w[i][0].x, w[i][1].x, w[i][0].y, w[i][1].y, b[i].x, b[i].y);
                mma_bf16(acc[n], w[i][0].z, w[i][1].z, w[i][0].w, w[i][1].w, b[i].z, b[i].w);
            }
        }
        if (last) {
            float4* r = red + turn * RED;
            turn ^= 1;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                r[(warp * NT + n) * 32 + lane] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
            }
            __syncthreads();
            const float* rf = reinterpret_cast<const float*>(r);
            const bool whole = s_begin0 == 0 && s_end0 == per;
            constexpr int OUT = 128 * NT;  // (column, token) values: i = token * 16 + column
            float* mine = p.part + ((size_t)blockIdx.x * 2 + (cb0 == cb_first ? 0 : 1)) * OUT;
            for (int i = threadIdx.x; i < OUT; i += FT_THREADS) {
                const int t = i >> 4, col = i & 15;
                float v = 0.f;
#pragma unroll
                for (int q = 0; q < FT_WARPS; ++q)
                    v += rf[(((q * NT + (t >> 3)) * 32) + (col & 7) * 4 + ((t & 7) >> 1)) * 4 + (col >> 3) * 2 + (t & 1)];
                if (!whole)
                    mine[i] = v;
                else if (t < T && cb0 * 16 + col < p.d)
                    p.y[(size_t)t * p.d + cb0 * 16 + col] = __float2bfloat16_rn(v);
            }
            if (!whole) {  // cut between CTAs: the last one to arrive adds the parts in their order
                const long x0 = (long)cb0 * per, x1 = x0 + per - 1;
                const int b0 = (int)(((x0 + 1) * gridDim.x - 1) / all), b1 = (int)(((x1 + 1) * gridDim.x - 1) / all);
                __threadfence();
                __syncthreads();
                if (threadIdx.x == 0) s_n[1] = atomicAdd(p.counters + 1 + cb0, 1) == b1 - b0;
                __syncthreads();
                if (s_n[1]) {
                    __threadfence();
                    for (int i = threadIdx.x; i < OUT; i += FT_THREADS) {
                        const int t = i >> 4, col = i & 15;
                        float v = 0.f;
                        for (int q = b0; q <= b1; ++q) {
                            const int which = (int)(all * q / gridDim.x / per) == cb0 ? 0 : 1;
                            v += __ldcg(p.part + ((size_t)q * 2 + which) * OUT + i);
                        }
                        if (t < T && cb0 * 16 + col < p.d) p.y[(size_t)t * p.d + cb0 * 16 + col] = __float2bfloat16_rn(v);
                    }
                }
                __syncthreads();
            }
        }
#pragma unroll
        for (int i = 0; i < FT_BATCH; ++i) {
            w[i][0] = wn[i][0];
            w[i][1] = wn[i][1];
        }
    }
}

}  // namespace moe
