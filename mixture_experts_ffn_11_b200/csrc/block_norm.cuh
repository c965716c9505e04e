// RMS norms around a block, and their gradients. The blog post "Mixture of Experts (MoEs) in Transformers" keeps "the
// Transformer backbone" around the expert layer (section "From Dense to Sparse"): what enters the layer is a norm of the
// residual stream, what leaves it is added back to the stream. With r the stream [T][d] and y the block's output [T][d]:
//
//   in front of the block   xn = r * rstd * w,                      rstd[t] = (mean_i r[t][i]^2 + eps)^(-1/2)
//   behind it               out = alpha r + g * (y * rstd * w)      rstd of y; g: a gate row per gate_rows tokens, or none
//   and, in the same pass   xn' = out * rstd' * w'                  rstd' of out as it is stored: the next block's input
//
// Each is one pass over its arrays (a few flops per element, so HBM bounds it). A row belongs to one CTA, whose threads
// hold VPT vectors of 8 columns each, the same columns for every row: the gains stay in registers, and the gradients of
// gains and gate, sums over rows, are kept there too until the CTA's rows are done. Sums are in fp32.
//
// Many rows: they arrive in shared memory by bulk copies that run BN stages ahead (RowRing), so HBM does not wait for a row's
// reductions; a stage is refilled as soon as the CTA has its row in registers. Few rows (at most one per CTA): plain loads, without
// the copies' extra latency.
//
// Measured (HBM's floor at a copy's rate in brackets): behind the block with the next norm, 4096 rows of 2880 in bf16, 25 us (14.4; its
// output mostly stays in L2, a row's reductions and stores set the pace); its gradient with a gate, 8192 rows of 4096 with an fp32 stream,
// 107 us (92), in bf16 88 us (62); the gradient in front, 4096 rows of 2880, 25 us (14.4), in two kernels, the second, launched ahead,
// adding the CTAs' partial sums in a fixed order, four rows of them at a time (launched behind the first 30.4 us); in front, 64 rows of
// 7168, 1.9 us (0.3), a launch. Rows by plain loads, one thread for all of a row's columns: 28.9, 238, -, 42.3.
#pragma once
#include "common.cuh"
#include "fp8_quant.cuh"
#include "sync.cuh"

namespace moe {

__device__ __forceinline__ void unpair(const uint64_t (&v)[4], float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("mov.b64 {%0, %1}, %2;" : "=f"(f[2 * i]), "=f"(f[2 * i + 1]) : "l"(v[i]));
}
__device__ __forceinline__ float sum2(uint64_t v) {
    float lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
    return lo + hi;
}

// 8 consecutive elements as they lie in memory
template <typename E>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
    uint4 q;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { q = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void zero() { q = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack_bf16x2(u[i]);
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
    __device__ __forceinline__ void put(const float (&v)[8]) {
        q = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = q; }
    __device__ __forceinline__ void pairs(uint64_t (&v)[4]) const {
        const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = pair2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
    }
    __device__ __forceinline__ void put_pairs(const uint64_t (&v)[4]) {
        float f[8];
        unpair(v, f);
        put(f);
    }
    // from here on the values are what this register holds: their fp32 forms are made again, not kept
    __device__ __forceinline__ void keep_packed() { asm volatile("" : "+r"(q.x), "+r"(q.y), "+r"(q.z), "+r"(q.w)); }
};
template <>
struct Vec8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = reinterpret_cast<const float4*>(p)[0];
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
    __device__ __forceinline__ void put(const float (&v)[8]) {
        a = make_float4(v[0], v[1], v[2], v[3]);
        b = make_float4(v[4], v[5], v[6], v[7]);
    }
    __device__ __forceinline__ void store(float* p) const {
        reinterpret_cast<float4*>(p)[0] = a;
        reinterpret_cast<float4*>(p)[1] = b;
    }
    __device__ __forceinline__ void pairs(uint64_t (&v)[4]) const {
        v[0] = pair2(a.x, a.y), v[1] = pair2(a.z, a.w), v[2] = pair2(b.x, b.y), v[3] = pair2(b.z, b.w);
    }
    __device__ __forceinline__ void put_pairs(const uint64_t (&v)[4]) {
        float f[8];
        unpair(v, f);
        put(f);
    }
    __device__ __forceinline__ void keep_packed() {}
};

constexpr int BN_MAX_THREADS = 512;
constexpr int BN_MAX_WARPS = BN_MAX_THREADS / 32;
constexpr int BN_MAX_D = BN_MAX_THREADS * 4 * 8;  // 4 vectors per thread
constexpr int BN_MAX_STAGES = 8;
constexpr int BN_MAX_CLUSTER = 8;
constexpr int BN_GRAD_CTAS = 592;  // rows of a backward pass are cut into at most so many ranges (4 per SM)

// One of the arrays that make up a row's input: elements of `size` bytes (0: no such array); row t is row t / per of it (per > 1: a gate
// row shared by consecutive tokens).
struct RowArray {
    const void* base;
    int size, per;
};

// Ring of rows in shared memory. RING = false: the same interface on the arrays themselves. SPREAD: every warp up to the number
// of arrays issues one array's copy, else thread 0 all of them (which of the two is
// faster was measured kernel by kernel: 4096 rows of 8192 in fp32 in two CTAs 192 us by one thread, 147 us spread; 8192 rows of 4096 in
// bf16 in one CTA 94 and 103 us).
//
// When a wait runs out, no row is copied any more, and what is under way is waited for before the CTA leaves. The warps of a SPREAD ring
// have to agree on which row is the first that is not copied (its barrier counts all their copies): thread 0 decides, in advance(),
// and leaves the decision for the others to read behind the barrier that every row has between its advance() and its release().
template <bool RING, int NARR, bool SPREAD = false>
struct RowRing {
    RowArray arr[NARR];
    uint64_t* full;
    int cols, col0, n;  // columns of the arrays, the first one taken, how many
    uint32_t row_bytes;
    int stages, stage, step, end, next;  // next: the row to copy next
    uint32_t phase;
    int row;

    // columns c0 .. c0 + n_cols of d, rows first, first + step, ... < end
    __device__ __forceinline__ void start(uint8_t* smem, int n_stages, int d, int c0, int n_cols, int first, int step_, int end_) {
        cols = d;
        col0 = c0;
        n = n_cols;
        step = step_;
        end = end_;
        row = first - step_;
        next = first;
        if constexpr (RING) {
            full = reinterpret_cast<uint64_t*>(smem);
            stages = n_stages;
            stage = -1;
            phase = 1;
            row_bytes = 0;
#pragma unroll
            for (int i = 0; i < NARR; ++i) row_bytes += (uint32_t)(n * arr[i].size);
            if (threadIdx.x == 0) {
                for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
                mbar_init(never(), 1);
                *abort_flag() = 0;
                *limit() = wait_limit_ns();
                fence_mbar_init();
            }
            __syncthreads();
            for (int s = 0; s < stages; ++s) copy(s, false);
            // (the test hook moe_test_set_wait: a wait that nothing ends)
            if (*reinterpret_cast<volatile int*>(&g_wait_stall) != 0) mbar_wait_within(never(), 0, abort_flag(), limit());
        }
    }
    // [3]: raised when a wait ran out; thread 0's decisions for even and odd rows (SPREAD, consecutive rows)
    __device__ __forceinline__ volatile int* abort_flag() const { return reinterpret_cast<volatile int*>(full + BN_MAX_STAGES); }
    __device__ __forceinline__ uint8_t* data() const { return reinterpret_cast<uint8_t*>(full) + 128; }
    __device__ __forceinline__ volatile uint64_t* limit() const { return full + BN_MAX_STAGES + 3; }
    __device__ __forceinline__ uint64_t* never() const { return full + BN_MAX_STAGES + 2; }  // a barrier that nothing arrives on
    __device__ __forceinline__ void copy(int s, bool stopped) {  // the next row into stage s
        if (next >= end || stopped) return;
        const int warp = threadIdx.x >> 5;
        if (SPREAD ? (threadIdx.x & 31) == 0 : threadIdx.x == 0) {
            if (warp == 0) mbar_arrive_expect_tx(&full[s], row_bytes);
            uint8_t* to = data() + (size_t)s * row_bytes;
#pragma unroll
            for (int i = 0; i < NARR; ++i) {
                const uint32_t bytes = (uint32_t)(n * arr[i].size);
                if (arr[i].size != 0 && (!SPREAD || warp == i)) {
                    const int r = arr[i].per > 1 ? next / arr[i].per : next;
                    bulk_load(to, reinterpret_cast<const uint8_t*>(arr[i].base) + ((size_t)r * cols + col0) * arr[i].size, bytes, &full[s]);
                }
                to += bytes;
            }
        }
        next += step;
    }
    // Go on to the next row, once it has arrived; false behind the last. (A wait that runs out sets the error bit and the rows
    // that follow are computed from whatever is there: no thread leaves alone.)
    __device__ __forceinline__ bool advance() {
        row += step;
        if (row >= end) return false;
        if constexpr (RING) {
            if (++stage == stages) stage = 0;
            if (stage == 0) phase ^= 1u;
            if (!mbar_wait_within(&full[stage], phase, abort_flag(), limit()) && threadIdx.x == 0 && row < next)
                mbar_wait_drain(&full[stage], phase);  // no copy is in flight when the CTA leaves
            if (SPREAD && threadIdx.x == 0) abort_flag()[1 + (row & 1)] = *abort_flag();
        }
        return true;
    }
    // Where the current row lies, for get() and release() now or some rows later (until it is released)
    __device__ __forceinline__ int here() const { return RING ? stage : row; }
    // Where the row `back` rows before that one lies (back at most 2 and below the number of stages)
    __device__ __forceinline__ int here_before(int back) const {
        if constexpr (!RING) return row - back;
        const int s = stage - back;
        return s < 0 ? s + stages : s;
    }
    // Elements of array i of the current row, or of the row that was at `at`
    template <typename E>
    __device__ __forceinline__ const E* get(int i) const {
        return get<E>(i, here());
    }
    template <typename E>
    __device__ __forceinline__ const E* get(int i, int at_row) const {
        if constexpr (RING) {
            uint32_t at = 0;
#pragma unroll
            for (int j = 0; j < NARR; ++j)
                if (j < i) at += (uint32_t)(n * arr[j].size);
            return reinterpret_cast<const E*>(data() + (size_t)at_row * row_bytes + at);
        } else {
            const int r = arr[i].per > 1 ? at_row / arr[i].per : at_row;
            return reinterpret_cast<const E*>(reinterpret_cast<const uint8_t*>(arr[i].base) + ((size_t)r * cols + col0) * arr[i].size);
        }
    }
    // The CTA is done with a row (all its threads are past a barrier since they read it): its stage takes another
    __device__ __forceinline__ void release() { release(here()); }
    __device__ __forceinline__ void release(int at_row) {
        if constexpr (RING) {
            copy(at_row, abort_flag()[SPREAD ? 1 + (row & 1) : 0] != 0);
        }
    }
};

// Sum over the CTA, given to every thread. `red` is one of two alternating buffers, so one barrier per call suffices: a thread that is
// a call ahead writes the other buffer, and two calls ahead is past the next barrier.
__device__ __forceinline__ float block_sum(float v, float* red) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0) red[warp] = v;
    __syncthreads();
    float s = (lane & 15) < warps ? red[lane & 15] : 0.f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}
// Three sums in 12 shuffles instead of 27: in the first two steps half of the lanes
// pass on one value and keep another, so that lanes 8 j .. 8 j + 7 end up adding value j; behind the barrier a lane takes value
// lane % 4 of warps lane / 4 and lane / 4 + 8.
__device__ __forceinline__ void block_sums(float (&v)[3], float* red) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const bool hi = lane & 16, odd = lane & 8;
    float x = hi ? v[2] : v[0], y = hi ? 0.f : v[1];
    x += __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[2], 16);
    y += __shfl_xor_sync(0xffffffffu, hi ? v[1] : 0.f, 16);
    float z = odd ? y : x;
    z += __shfl_xor_sync(0xffffffffu, odd ? x : y, 8);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    if ((lane & 7) == 0) red[warp * 4 + (lane >> 3)] = z;
    __syncthreads();
    z = (lane >> 2) < warps ? red[lane] : 0.f;
    if ((lane >> 2) + 8 < warps) z += red[lane + 32];
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
#pragma unroll
    for (int j = 0; j < 3; ++j) v[j] = __shfl_sync(0xffffffffu, z, j);
}

// Rows wider than a CTA's threads hold are cut by columns over the CTAs of a cluster. Each sends its sums of a row to all of them (st.async
// into shared memory, counted by the receiver's barrier) and adds what it got in the order of the CTAs, one row later: about 1 us on
// the way, in which the CTA takes up the next row. Four slots: a CTA sends row m only with every other's sums of row m - 2,
// which that one sends once all its threads have taken those of row m - 4. A CTA whose wait ran out sends no more and expects no
// more (its barrier may still be waiting for an earlier row); the others' waits then run out too.
struct ClusterSums {
    float4 slot[4][BN_MAX_CLUSTER];
    uint64_t bar[4];
    uint64_t limit;
    uint32_t expect;  // bytes of a row
    int abort_flag;
};
__device__ __forceinline__ void cluster_sums_init(ClusterSums& x, uint32_t ctas) {
    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; ++i) mbar_init(&x.bar[i], 1);
        // (the test hook moe_test_set_wait: one CTA's sums more than there are)
        x.expect = (ctas + (*reinterpret_cast<volatile int*>(&g_wait_stall) != 0 ? 1u : 0u)) * 16u;
        x.abort_flag = 0;
        x.limit = wait_limit_ns();
        fence_mbar_init();
    }
    cluster_sync();
}
// n: how many rows came before
__device__ __forceinline__ void cluster_sums_send(ClusterSums& x, int n, uint32_t ctas, uint32_t rank, const float (&v)[3]) {
    const int turn = n & 3;
    const int i = (int)threadIdx.x - (int)blockDim.x + 32;  // the last warp
    if (i < 0 || *reinterpret_cast<volatile int*>(&x.abort_flag)) return;
    if (i == 0) mbar_arrive_expect_tx(&x.bar[turn], x.expect);
    if (i < (int)ctas)
        store_remote(mapa_shared(smem_u32(&x.slot[turn][rank]), i), make_float4(v[0], v[1], v[2], 0.f),
                     mapa_shared(smem_u32(&x.bar[turn]), i));
}
__device__ __forceinline__ void cluster_sums_take(ClusterSums& x, int n, uint32_t ctas, float (&v)[3]) {
    const int turn = n & 3;
    mbar_wait_within(&x.bar[turn], (uint32_t)(n >> 2) & 1u, &x.abort_flag, static_cast<const volatile uint64_t*>(&x.limit));
    v[0] = v[1] = v[2] = 0.f;
    for (uint32_t r = 0; r < ctas; ++r) {
        const float4 q = x.slot[turn][r];
        v[0] += q.x, v[1] += q.y, v[2] += q.z;
    }
}

template <int VPT>
__device__ __forceinline__ void load_gains(const float* w, int nvec, float (&g)[VPT][8]) {
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
        const int v = threadIdx.x + u * blockDim.x;
        Vec8<float> q;
        q.zero();
        if (v < nvec) q.load(w + (size_t)v * 8);
        q.get(g[u]);
    }
}

__device__ __forceinline__ void load_gains(const float* w, int nvec, uint64_t (&g)[4]) {
    Vec8<float> q;
    q.zero();
    if (threadIdx.x < nvec) q.load(w + (size_t)threadIdx.x * 8);
    q.pairs(g);
}

// ---- forward ----------------------------------------------------------------------------------------

template <typename R, int VPT, bool RING>
__global__ void __launch_bounds__(BN_MAX_THREADS) block_norm_in_kernel(const R* __restrict__ x, const float* __restrict__ w, int T,
                                                             int d, float eps, __nv_bfloat16* __restrict__ xn,
                                                             float* __restrict__ rstd, int stages) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float red[2][BN_MAX_WARPS];
    grid_dep_wait();
    grid_dep_trigger();
    const int nvec = d >> 3;
    RowRing<RING, 1> rows;
    rows.arr[0] = {x, sizeof(R), 1};
    rows.start(smem, stages, d, 0, d, blockIdx.x, gridDim.x, T);
    float g[VPT][8];
    load_gains<VPT>(w, nvec, g);
    int turn = 0;
    for (; rows.advance(); turn ^= 1) {
        const int t = rows.row;
        const R* x_row = rows.template get<R>(0);
        Vec8<R> q[VPT];
        float s[1] = {0.f};
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const int v = threadIdx.x + u * blockDim.x;
            q[u].zero();
            if (v < nvec) q[u].load(x_row + v * 8);
        }
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            float f[8];
            q[u].get(f);
#pragma unroll
            for (int i = 0; i < 8; ++i) s[0] = fmaf(f[i], f[i], s[0]);
        }
        s[0] = block_sum(s[0], red[turn]);
        rows.release();
        const float rs = rsqrtf(s[0] / (float)d + eps);
        if (threadIdx.x == 0) rstd[t] = rs;
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const int v = threadIdx.x + u * blockDim.x;
            if (v >= nvec) continue;
            float f[8];
            q[u].get(f);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = f[i] * rs * g[u][i];
            Vec8<__nv_bfloat16> o;
            o.put(f);
            o.store(xn + (size_t)t * d + (size_t)v * 8);
        }
    }
}

struct NormOutArgs {
    const __nv_bfloat16* y;     // [T][d]
    const void* r;              // [T][d] bf16 or fp32; out may be the same memory
    const float* w;             // [d]
    const __nv_bfloat16* gate;  // [ceil(T / gate_rows)][d] or null
    const float* w_next;        // [d] or null
    void* out;                  // [T][d], type of r
    float* rstd;                // [T]
    __nv_bfloat16* xn;          // [T][d] (with w_next)
    float* rstd_next;           // [T] (with w_next)
    int T, d, gate_rows;
    float alpha, eps;
};

template <typename R, int VPT, bool NEXT, bool RING>
__global__ void __launch_bounds__(BN_MAX_THREADS) block_norm_out_kernel(const NormOutArgs a, int stages) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float red[2][BN_MAX_WARPS];
    grid_dep_wait();
    grid_dep_trigger();
    const int nvec = a.d >> 3;
    RowRing<RING, 3> rows;
    rows.arr[0] = {a.y, 2, 1};
    rows.arr[1] = {a.r, sizeof(R), 1};
    rows.arr[2] = {a.gate, a.gate ? 2 : 0, a.gate_rows};
    rows.start(smem, stages, a.d, 0, a.d, blockIdx.x, gridDim.x, a.T);
    float g[VPT][8], gn[NEXT ? VPT : 1][8];
    load_gains<VPT>(a.w, nvec, g);
    if constexpr (NEXT) load_gains<VPT>(a.w_next, nvec, gn);
    R* out = reinterpret_cast<R*>(a.out);
    int turn = 0;
    while (rows.advance()) {
        const int t = rows.row;
        Vec8<__nv_bfloat16> y[VPT], gt[VPT];
        Vec8<R> q[VPT];
        float s[1] = {0.f};
        const __nv_bfloat16 *y_row = rows.template get<__nv_bfloat16>(0), *gate_row = rows.template get<__nv_bfloat16>(2);
        const R* r_row = rows.template get<R>(1);
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const int v = threadIdx.x + u * blockDim.x;
            y[u].zero();
            q[u].zero();
            gt[u].zero();
            if (v < nvec) {
                y[u].load(y_row + v * 8);
                q[u].load(r_row + v * 8);
                if (a.gate) gt[u].load(gate_row + v * 8);
            }
        }
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            float f[8];
            y[u].get(f);
#pragma unroll
            for (int i = 0; i < 8; ++i) s[0] = fmaf(f[i], f[i], s[0]);
        }
        s[0] = block_sum(s[0], red[turn]);
        rows.release();
        turn ^= 1;
        const float rs = rsqrtf(s[0] / (float)a.d + a.eps);
        if (threadIdx.x == 0) a.rstd[t] = rs;
        s[0] = 0.f;
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const int v = threadIdx.x + u * blockDim.x;
            float f[8], o[8], m[8];
            y[u].get(f);
            q[u].get(o);
            gt[u].get(m);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float n = f[i] * rs * g[u][i];
                o[i] = fmaf(a.alpha, o[i], a.gate ? n * m[i] : n);
            }
            q[u].put(o);  // the stream as it is stored: what the next norm, and a backward pass, read
            if (v < nvec) q[u].store(out + (size_t)t * a.d + (size_t)v * 8);
            if constexpr (NEXT) {
                q[u].get(o);
                if (v < nvec) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) s[0] = fmaf(o[i], o[i], s[0]);
                }
            }
        }
        if constexpr (NEXT) {
            s[0] = block_sum(s[0], red[turn]);
            turn ^= 1;
            const float rn = rsqrtf(s[0] / (float)a.d + a.eps);
            if (threadIdx.x == 0) a.rstd_next[t] = rn;
#pragma unroll
            for (int u = 0; u < VPT; ++u) {
                const int v = threadIdx.x + u * blockDim.x;
                if (v >= nvec) continue;
                float o[8];
                q[u].get(o);
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = o[i] * rn * gn[u][i];
                Vec8<__nv_bfloat16> n;
                n.put(o);
                n.store(a.xn + (size_t)t * a.d + (size_t)v * 8);
            }
        }
    }
}

// ---- backward ---------------------------------------------------------------------------------------
// CTA b takes the rows [T b / B, T (b + 1) / B) (contiguous, so that a gate row's tokens meet in few CTAs) and leaves its
// sums over them in the workspace, [B][d] fp32 per sum; block_norm_reduce_kernel adds those in the order of b. No atomics:
// the same bits every time. A gate row whose tokens all lie in one CTA is written there; of the others a CTA can only
// have its first and its last (slots 0 and 1).

__host__ __device__ __forceinline__ int norm_first_row(int T, int B, int b) { return (int)((long)T * b / B); }

struct NormInGradArgs {
    const __nv_bfloat16* dxn;  // [T][d]
    const void* dres;          // [T][d] or null, type of x
    const void* x;             // [T][d]
    const float* w;            // [d]
    const float* rstd;         // [T]
    void* dx;                  // [T][d], type of x; may be dres
    float* part_w;             // [B][d]
    int T, d;
};

template <typename R, int VPT, bool RING>
__global__ void __launch_bounds__(BN_MAX_THREADS) block_norm_in_grad_kernel(const NormInGradArgs a, int stages) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float red[2][BN_MAX_WARPS];
    const int nvec = a.d >> 3;
    const float inv_d = 1.f / (float)a.d;
    RowRing<RING, 3> rows;
    rows.arr[0] = {a.dxn, 2, 1};
    rows.arr[1] = {a.x, sizeof(R), 1};
    rows.arr[2] = {a.dres, a.dres ? (int)sizeof(R) : 0, 1};
    grid_dep_wait();
    grid_dep_trigger();
    rows.start(smem, stages, a.d, 0, a.d, norm_first_row(a.T, gridDim.x, blockIdx.x), 1, norm_first_row(a.T, gridDim.x, blockIdx.x + 1));
    float g[VPT][8], acc[VPT][8];
    load_gains<VPT>(a.w, nvec, g);
#pragma unroll
    for (int u = 0; u < VPT; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[u][i] = 0.f;
    R* dx = reinterpret_cast<R*>(a.dx);
    int turn = 0;
    for (; rows.advance(); turn ^= 1) {
        const int t = rows.row;
        const __nv_bfloat16* dxn_row = rows.template get<__nv_bfloat16>(0);
        const R *x_row = rows.template get<R>(1), *dres_row = rows.template get<R>(2);
        Vec8<__nv_bfloat16> dn[VPT];
        Vec8<R> q[VPT], res[VPT];
        float s[1] = {0.f};
        const float rs = a.rstd[t];
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const int v = threadIdx.x + u * blockDim.x;
            dn[u].zero();
            q[u].zero();
            res[u].zero();
            if (v < nvec) {
                dn[u].load(dxn_row + v * 8);
                q[u].load(x_row + v * 8);
                if (a.dres) res[u].load(dres_row + v * 8);
            }
        }
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            float f[8], m[8];
            q[u].get(f);
            dn[u].get(m);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float hat = f[i] * rs;
                acc[u][i] = fmaf(m[i], hat, acc[u][i]);
                s[0] = fmaf(m[i] * g[u][i], hat, s[0]);
            }
        }
        s[0] = block_sum(s[0], red[turn]);
        rows.release();
        const float mean = s[0] * inv_d;
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const int v = threadIdx.x + u * blockDim.x;
            if (v >= nvec) continue;
            float f[8], m[8], o[8];
            q[u].get(f);
            dn[u].get(m);
            res[u].get(o);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = fmaf(rs, fmaf(-f[i] * rs, mean, m[i] * g[u][i]), o[i]);
            q[u].put(o);
            q[u].store(dx + (size_t)t * a.d + (size_t)v * 8);
        }
    }
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
        const int v = threadIdx.x + u * blockDim.x;
        if (v >= nvec) continue;
        Vec8<float> o;
        o.put(acc[u]);
        o.store(a.part_w + (size_t)blockIdx.x * a.d + (size_t)v * 8);
    }
}

struct NormOutGradArgs {
    const void* dout;           // [T][d], type of out
    const __nv_bfloat16* dxn;   // [T][d] or null
    const __nv_bfloat16* y;     // [T][d]
    const void* out;            // [T][d] (with dxn)
    const float* w;             // [d]
    const __nv_bfloat16* gate;  // [groups][d] or null
    const float* w_next;        // [d] (with dxn)
    const float* rstd;          // [T]
    const float* rstd_next;     // [T] (with dxn)
    void* dr;                   // [T][d]; may be dout
    __nv_bfloat16* dy;          // [T][d]
    float* dgate;               // [groups][d] or null
    float* part_w;              // [B][d]
    float* part_next;           // [B][d] (with dxn)
    float* part_gate;           // [B][2][d] (with gate)
    int T, d, gate_rows;
    float alpha;
};

// With dR the gradient that reaches `out` by both ways (along the stream, and through the next norm):
//   dR = dout + rstd' (dxn w' - out rstd'^2 S1 / d),   S1 = sum dxn w' out
//   dy = rstd (dR g w - yhat S2 / d),                  S2 = sum dR g w yhat,  yhat = y rstd
// S2 needs dR, which needs S1; but it is linear in it: S2 = SA - (rstd'^3 S1 / d) SB with SA = sum (dout + rstd' dxn w') g w
// yhat and SB = sum out g w yhat, so one reduction over the row gives all three. dR is never rounded.
//
// A thread keeps one vector of 8 columns: gains, sums and a row's values are up to 80 registers for it. Rows of more columns than
// a CTA's threads hold are cut over the CTAs of a cluster. (With two or four vectors per thread they spilled: 4096 rows of 8192 in
// bf16 202 us instead of 137, 2048 of 16384 in fp32 921 us instead of 151.) Instructions and the steps from row to row bound it there, HBM
// for one CTA per row in fp32 (8192 rows of 4096 with gate and next norm: 107 us, floor 92; bf16 88 us, floor 62).
template <typename R, bool NEXT, bool GATE, bool RING, bool CLUSTER>
__global__ void __launch_bounds__(BN_MAX_THREADS) block_norm_out_grad_kernel(const NormOutGradArgs a, int stages) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float red[2][4 * BN_MAX_WARPS];
    __shared__ __align__(16) ClusterSums across;
    const uint32_t ctas = CLUSTER ? cluster_nctarank() : 1, rank = CLUSTER ? cluster_ctarank() : 0;
    const int range = CLUSTER ? blockIdx.x / ctas : blockIdx.x, ranges = CLUSTER ? gridDim.x / ctas : gridDim.x;
    const int per_cta = ((a.d >> 3) + (int)ctas - 1) / (int)ctas;  // vectors
    const int c0 = (int)rank * per_cta * 8;                        // this CTA's columns: c0 .. c0 + 8 nvec
    const int nvec = min(per_cta, (a.d - c0) >> 3);
    const float inv_d = 1.f / (float)a.d;
    const int t0 = norm_first_row(a.T, ranges, range), t1 = norm_first_row(a.T, ranges, range + 1);
    RowRing<RING, 5, CLUSTER> rows;  // (a cluster's CTAs have more than 5 warps)
    rows.arr[0] = {a.dout, sizeof(R), 1};
    rows.arr[1] = {a.y, 2, 1};
    rows.arr[2] = {a.out, NEXT ? (int)sizeof(R) : 0, 1};
    rows.arr[3] = {a.dxn, NEXT ? 2 : 0, 1};
    rows.arr[4] = {a.gate, GATE ? 2 : 0, a.gate_rows};
    grid_dep_wait();
    grid_dep_trigger();
    rows.start(smem, stages, a.d, c0, nvec * 8, t0, 1, t1);
    if constexpr (CLUSTER) cluster_sums_init(across, ctas);
    // two columns to an operation throughout (fp32 pairs): a row's instructions weigh as much as its bytes
    uint64_t g[4], gn[4], acc[4], acc_next[4], acc_gate[4];
    load_gains(a.w + c0, nvec, g);
    if constexpr (NEXT) load_gains(a.w_next + c0, nvec, gn);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = acc_next[i] = acc_gate[i] = 0;
    const int v = threadIdx.x;
    const bool mine = v < nvec;
    const uint64_t alpha2 = pair2(a.alpha, a.alpha);
    R* dr = reinterpret_cast<R*>(a.dr) + c0 + v * 8;
    __nv_bfloat16* dy = a.dy + c0 + v * 8;
    struct Row {
        Vec8<__nv_bfloat16> dn, y, gt;
        Vec8<R> up, o;
    };
    const auto load = [&](Row& q, int at) {
        q.up.zero();
        q.y.zero();
        if constexpr (NEXT) q.o.zero(), q.dn.zero();
        if constexpr (GATE) q.gt.zero();
        if (!mine) return;
        q.up.load(rows.template get<R>(0, at) + v * 8);
        q.y.load(rows.template get<__nv_bfloat16>(1, at) + v * 8);
        if constexpr (NEXT) {
            q.o.load(rows.template get<R>(2, at) + v * 8);
            q.dn.load(rows.template get<__nv_bfloat16>(3, at) + v * 8);
        }
        if constexpr (GATE) q.gt.load(rows.template get<__nv_bfloat16>(4, at) + v * 8);
    };
    // a row's sums over the CTA's columns; n: how many rows came before
    const auto sums = [&](const Row& q, float rs, float rn, int n, float (&s)[3]) {
        const uint64_t rs2 = pair2(rs, rs), rn2 = pair2(rn, rn);
        uint64_t fu[4], fy[4], fo[4], fd[4], fg[4], s2[3] = {0, 0, 0};
        q.up.pairs(fu);
        q.y.pairs(fy);
        if constexpr (NEXT) q.o.pairs(fo), q.dn.pairs(fd);
        if constexpr (GATE) q.gt.pairs(fg);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint64_t k = mul2(mul2(fy[i], rs2), g[i]);
            if constexpr (GATE) k = mul2(k, fg[i]);
            if constexpr (NEXT) {
                const uint64_t m = mul2(fd[i], gn[i]);
                s2[0] = fma2(fma2(rn2, m, fu[i]), k, s2[0]);
                s2[1] = fma2(m, fo[i], s2[1]);
                s2[2] = fma2(fo[i], k, s2[2]);
                acc_next[i] = fma2(fd[i], mul2(fo[i], rn2), acc_next[i]);
            } else {
                s2[0] = fma2(fu[i], k, s2[0]);
            }
        }
        if constexpr (NEXT) {
#pragma unroll
            for (int j = 0; j < 3; ++j) s[j] = sum2(s2[j]);
            block_sums(s, red[n & 1]);
        } else {
            s[0] = block_sum(sum2(s2[0]), red[n & 1]);
            s[1] = s[2] = 0.f;
        }
    };
    // its gradients, from the sums over all columns
    const auto finish = [&](Row& q, int t, float rs, float rn, const float (&s)[3]) {
        // dR = dout + rstd' (dxn w' - c out), S2 = SA - rstd' c SB. Factors in an order that keeps the products of rstd' and of out near 1
        // (rstd'^3 alone leaves fp32's range for rows of rms 1e-13 or 1e15)
        float c = 0.f;
        if constexpr (NEXT) c = rn * (rn * s[1] * inv_d);
        const float mean = (NEXT ? s[0] - rn * (c * s[2]) : s[0]) * inv_d;
        if (!mine) return;
        q.up.keep_packed();
        q.y.keep_packed();
        if constexpr (NEXT) q.o.keep_packed(), q.dn.keep_packed();
        if constexpr (GATE) q.gt.keep_packed();
        uint64_t fu[4], fy[4], fo[4], fd[4], fg[4];
        q.up.pairs(fu);
        q.y.pairs(fy);
        if constexpr (NEXT) q.o.pairs(fo), q.dn.pairs(fd);
        if constexpr (GATE) q.gt.pairs(fg);
        const uint64_t rs2 = pair2(rs, rs), rn2 = pair2(rn, rn), minus_c = pair2(-c, -c), minus_mean = pair2(-mean, -mean);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint64_t dR = fu[i];
            if constexpr (NEXT) dR = fma2(rn2, fma2(minus_c, fo[i], mul2(gn[i], fd[i])), dR);
            const uint64_t hat = mul2(fy[i], rs2), e = mul2(dR, hat);
            uint64_t dn = mul2(dR, g[i]);
            if constexpr (GATE) {
                acc_gate[i] = fma2(e, g[i], acc_gate[i]);
                acc[i] = fma2(e, fg[i], acc[i]);
                dn = mul2(dn, fg[i]);
            } else {
                acc[i] = add2(acc[i], e);
            }
            fy[i] = mul2(rs2, fma2(hat, minus_mean, dn));
            fu[i] = mul2(alpha2, dR);
        }
        q.up.put_pairs(fu);
        q.up.store(dr + (size_t)t * a.d);
        q.y.put_pairs(fy);
        q.y.store(dy + (size_t)t * a.d);
        if constexpr (GATE) {
            if (t + 1 == t1 || (t + 1) % a.gate_rows == 0) {  // the last of a gate row's tokens here
                const int group = t / a.gate_rows;
                const long g0 = (long)group * a.gate_rows;
                const bool whole = g0 >= t0 && (t + 1 == a.T || t + 1 == g0 + a.gate_rows);
                float* to = whole ? a.dgate + (size_t)group * a.d
                                  : a.part_gate + ((size_t)range * 2 + (group == t0 / a.gate_rows ? 0 : 1)) * a.d;
                Vec8<float> o;
                o.put_pairs(acc_gate);
                o.store(to + c0 + v * 8);
#pragma unroll
                for (int i = 0; i < 4; ++i) acc_gate[i] = 0;
            }
        }
    };
    if constexpr (!CLUSTER) {
        for (int n = 0; rows.advance(); ++n) {
            const int t = rows.row;
            const float rs = a.rstd[t], rn = NEXT ? a.rstd_next[t] : 0.f;
            Row q;
            float s[3];
            load(q, rows.here());
            sums(q, rs, rn, n, s);
            rows.release();
            finish(q, t, rs, rn, s);
        }
    } else {
        float rs_before = 0.f, rn_before = 0.f;
        for (int n = 0;; ++n) {
            const bool more = rows.advance();
            float rs = 0.f, rn = 0.f, s[3];
            Row q;
            if (more) {
                rs = a.rstd[rows.row], rn = NEXT ? a.rstd_next[rows.row] : 0.f;
                load(q, rows.here());
                sums(q, rs, rn, n, s);
                cluster_sums_send(across, n, ctas, rank, s);
                if (n > 1) rows.release(rows.here_before(2));
            }
            if (n > 0) {
                load(q, RING && !more ? rows.here() : rows.here_before(1));  // (behind the last row the ring has not moved)
                cluster_sums_take(across, n - 1, ctas, s);
                finish(q, t0 + n - 1, rs_before, rn_before, s);
            }
            if (!more) break;
            rs_before = rs, rn_before = rn;
        }
    }
    if (mine) {
        Vec8<float> q;
        q.put_pairs(acc);
        q.store(a.part_w + (size_t)range * a.d + c0 + v * 8);
        if constexpr (NEXT) {
            q.put_pairs(acc_next);
            q.store(a.part_next + (size_t)range * a.d + c0 + v * 8);
        }
    }
    if constexpr (CLUSTER) cluster_sync();  // no CTA leaves while another's sums may still arrive in it
}

// Adds up what the CTAs left: blockIdx.y = 0: dw, 1: dw_next (with part_next), then the gate rows that lie in several CTAs, each by
// the first CTA whose last row is one of its tokens but not the last (edge: that CTA). 32 columns per block; 8 lanes cover them
// with 16-byte loads, so a warp adds four partial rows at a time (warp i: rows 4i .. 4i + 3, then 64 further on), all in a fixed
// order: the rows of a lane, the four lanes of a column, the sixteen warps.
struct NormReduceArgs {
    const float *part_w, *part_next, *part_gate;
    float *dw, *dw_next, *dgate;
    int T, d, gate_rows, B, sums;  // sums: 1, or 2 with part_next
    int16_t edge[BN_GRAD_CTAS];
};

constexpr int BNR_WARPS = 16;

__global__ void __launch_bounds__(BNR_WARPS * 32) block_norm_reduce_kernel(const __grid_constant__ NormReduceArgs a) {
    __shared__ __align__(16) float sums[BNR_WARPS][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int col = blockIdx.x * 32 + lane;
    const int job = blockIdx.y;
    int b0 = 0, b1 = a.B;  // CTAs to add
    const float* from = job == 0 ? a.part_w : a.part_next;
    float* to = job == 0 ? a.dw : a.dw_next;
    size_t pitch = a.d;
    int slot0 = 0;  // of a gate row in the first CTA: 1 if that CTA has an earlier gate row in part too
    if (job >= a.sums) {
        b0 = a.edge[job - a.sums];
        const long group = (norm_first_row(a.T, a.B, b0 + 1) - 1) / a.gate_rows;
        const long last = min((group + 1) * a.gate_rows, (long)a.T) - 1;
        b1 = (int)(((last + 1) * a.B - 1) / a.T) + 1;  // one past the CTA of the last token
        slot0 = norm_first_row(a.T, a.B, b0) / a.gate_rows == group ? 0 : 1;
        from = a.part_gate;
        to = a.dgate + group * a.d;
        pitch *= 2;
    }
    grid_dep_wait();
    grid_dep_trigger();
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    const int col4 = blockIdx.x * 32 + (lane & 7) * 4;
    if (col4 < a.d) {
#pragma unroll 5
        for (int b = b0 + warp * 4 + (lane >> 3); b < b1; b += BNR_WARPS * 4) {
            const float4 v = *reinterpret_cast<const float4*>(from + b * pitch + (b == b0 ? (size_t)slot0 * a.d : 0) + col4);
            s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
    }
#pragma unroll
    for (int o = 8; o < 32; o <<= 1) {
        s.x += __shfl_xor_sync(0xffffffffu, s.x, o);
        s.y += __shfl_xor_sync(0xffffffffu, s.y, o);
        s.z += __shfl_xor_sync(0xffffffffu, s.z, o);
        s.w += __shfl_xor_sync(0xffffffffu, s.w, o);
    }
    if (lane < 8) *reinterpret_cast<float4*>(&sums[warp][lane * 4]) = s;
    __syncthreads();
    if (warp == 0 && col < a.d) {
        float all = sums[0][lane];
#pragma unroll
        for (int i = 1; i < BNR_WARPS; ++i) all += sums[i][lane];
        to[col] = all;
    }
}

}  // namespace moe
