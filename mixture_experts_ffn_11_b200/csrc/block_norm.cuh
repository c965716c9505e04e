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
#pragma once
#include "common.cuh"

namespace moe {

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
};

constexpr int BN_MAX_THREADS = 512;
constexpr int BN_MAX_WARPS = BN_MAX_THREADS / 32;
constexpr int BN_MAX_D = BN_MAX_THREADS * 4 * 8;  // 4 vectors per thread
constexpr int BN_GRAD_CTAS = 296;  // rows of a backward pass are cut into at most so many ranges (2 per SM)

// Sums of NS values over the CTA, given to every thread. `red` is one of two alternating buffers, so one barrier per call
// suffices: a thread that is a call ahead writes the other buffer, and two calls ahead is past the next barrier.
template <int NS>
__device__ __forceinline__ void block_sums(float (&v)[NS], float (*red)[BN_MAX_WARPS]) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        if (lane == 0) red[i][warp] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        float s = lane < warps ? red[i][lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        v[i] = s;
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

// ---- forward ----------------------------------------------------------------------------------------

template <typename R, int VPT>
__global__ void __launch_bounds__(BN_MAX_THREADS) block_norm_in_kernel(const R* __restrict__ x, const float* __restrict__ w, int T,
                                                             int d, float eps, __nv_bfloat16* __restrict__ xn,
                                                             float* __restrict__ rstd) {
    __shared__ float red[2][1][BN_MAX_WARPS];
    grid_dep_wait();
    grid_dep_trigger();
    const int nvec = d >> 3;
    float g[VPT][8];
    load_gains<VPT>(w, nvec, g);
    int turn = 0;
    for (int t = blockIdx.x; t < T; t += gridDim.x, turn ^= 1) {
        Vec8<R> q[VPT];
        float s[1] = {0.f};
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const int v = threadIdx.x + u * blockDim.x;
            q[u].zero();
            if (v < nvec) q[u].load(x + (size_t)t * d + (size_t)v * 8);
        }
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            float f[8];
            q[u].get(f);
#pragma unroll
            for (int i = 0; i < 8; ++i) s[0] = fmaf(f[i], f[i], s[0]);
        }
        block_sums<1>(s, red[turn]);
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

template <typename R, int VPT, bool NEXT>
__global__ void __launch_bounds__(BN_MAX_THREADS) block_norm_out_kernel(const NormOutArgs a) {
    __shared__ float red[2][1][BN_MAX_WARPS];
    grid_dep_wait();
    grid_dep_trigger();
    const int nvec = a.d >> 3;
    float g[VPT][8], gn[NEXT ? VPT : 1][8];
    load_gains<VPT>(a.w, nvec, g);
    if constexpr (NEXT) load_gains<VPT>(a.w_next, nvec, gn);
    const R* r = reinterpret_cast<const R*>(a.r);
    R* out = reinterpret_cast<R*>(a.out);
    int turn = 0;
    for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
        Vec8<__nv_bfloat16> y[VPT], gt[VPT];
        Vec8<R> q[VPT];
        float s[1] = {0.f};
        const size_t grow = a.gate ? (size_t)(t / a.gate_rows) * a.d : 0;
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const int v = threadIdx.x + u * blockDim.x;
            y[u].zero();
            q[u].zero();
            gt[u].zero();
            if (v < nvec) {
                y[u].load(a.y + (size_t)t * a.d + (size_t)v * 8);
                q[u].load(r + (size_t)t * a.d + (size_t)v * 8);
                if (a.gate) gt[u].load(a.gate + grow + (size_t)v * 8);
            }
        }
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            float f[8];
            y[u].get(f);
#pragma unroll
            for (int i = 0; i < 8; ++i) s[0] = fmaf(f[i], f[i], s[0]);
        }
        block_sums<1>(s, red[turn]);
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
            block_sums<1>(s, red[turn]);
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

__device__ __forceinline__ int norm_first_row(int T, int B, int b) { return (int)((long)T * b / B); }

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

template <typename R, int VPT>
__global__ void __launch_bounds__(BN_MAX_THREADS) block_norm_in_grad_kernel(const NormInGradArgs a) {
    __shared__ float red[2][1][BN_MAX_WARPS];
    const int nvec = a.d >> 3;
    const float inv_d = 1.f / (float)a.d;
    float g[VPT][8], acc[VPT][8];
    load_gains<VPT>(a.w, nvec, g);
#pragma unroll
    for (int u = 0; u < VPT; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[u][i] = 0.f;
    const R* x = reinterpret_cast<const R*>(a.x);
    const R* dres = reinterpret_cast<const R*>(a.dres);
    R* dx = reinterpret_cast<R*>(a.dx);
    int turn = 0;
    const int t1 = norm_first_row(a.T, gridDim.x, blockIdx.x + 1);
    for (int t = norm_first_row(a.T, gridDim.x, blockIdx.x); t < t1; ++t, turn ^= 1) {
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
                const size_t at = (size_t)t * a.d + (size_t)v * 8;
                dn[u].load(a.dxn + at);
                q[u].load(x + at);
                if (dres) res[u].load(dres + at);
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
        block_sums<1>(s, red[turn]);
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
template <typename R, int VPT, bool NEXT, bool GATE>
__global__ void __launch_bounds__(BN_MAX_THREADS) block_norm_out_grad_kernel(const NormOutGradArgs a) {
    constexpr int NS = NEXT ? 3 : 1;
    __shared__ float red[2][NS][BN_MAX_WARPS];
    const int nvec = a.d >> 3;
    const float inv_d = 1.f / (float)a.d;
    float g[VPT][8], gn[NEXT ? VPT : 1][8];
    float acc[VPT][8], acc_next[NEXT ? VPT : 1][8], acc_gate[GATE ? VPT : 1][8];
    load_gains<VPT>(a.w, nvec, g);
    if constexpr (NEXT) load_gains<VPT>(a.w_next, nvec, gn);
#pragma unroll
    for (int u = 0; u < VPT; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            acc[u][i] = 0.f;
            if constexpr (NEXT) acc_next[u][i] = 0.f;
            if constexpr (GATE) acc_gate[u][i] = 0.f;
        }
    const R* dout = reinterpret_cast<const R*>(a.dout);
    const R* out = reinterpret_cast<const R*>(a.out);
    R* dr = reinterpret_cast<R*>(a.dr);
    int turn = 0;
    const int t0 = norm_first_row(a.T, gridDim.x, blockIdx.x), t1 = norm_first_row(a.T, gridDim.x, blockIdx.x + 1);
    for (int t = t0; t < t1; ++t, turn ^= 1) {
        Vec8<__nv_bfloat16> dn[NEXT ? VPT : 1], y[VPT], gt[GATE ? VPT : 1];
        Vec8<R> up[VPT], o[NEXT ? VPT : 1];
        float s[NS] = {};
        const float rs = a.rstd[t];
        const float rn = NEXT ? a.rstd_next[t] : 0.f;
        const int group = GATE ? t / a.gate_rows : 0;
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const int v = threadIdx.x + u * blockDim.x;
            up[u].zero();
            y[u].zero();
            if constexpr (NEXT) o[u].zero(), dn[u].zero();
            if constexpr (GATE) gt[u].zero();
            if (v < nvec) {
                const size_t at = (size_t)t * a.d + (size_t)v * 8;
                up[u].load(dout + at);
                y[u].load(a.y + at);
                if constexpr (NEXT) {
                    o[u].load(out + at);
                    dn[u].load(a.dxn + at);
                }
                if constexpr (GATE) gt[u].load(a.gate + (size_t)group * a.d + (size_t)v * 8);
            }
        }
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            float fu[8], fy[8], fo[8], fd[8], fg[8];
            up[u].get(fu);
            y[u].get(fy);
            if constexpr (NEXT) o[u].get(fo), dn[u].get(fd);
            if constexpr (GATE) gt[u].get(fg);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float k = fy[i] * rs * g[u][i] * (GATE ? fg[i] : 1.f);
                if constexpr (NEXT) {
                    const float n = fd[i] * gn[u][i];
                    s[0] = fmaf(fmaf(rn, n, fu[i]), k, s[0]);
                    s[1] = fmaf(n, fo[i], s[1]);
                    s[2] = fmaf(fo[i], k, s[2]);
                    acc_next[u][i] = fmaf(fd[i], fo[i] * rn, acc_next[u][i]);
                } else {
                    s[0] = fmaf(fu[i], k, s[0]);
                }
            }
        }
        block_sums<NS>(s, red[turn]);
        float c = 0.f;  // dR = dout + rstd' dxn w' - c out
        if constexpr (NEXT) c = rn * rn * rn * s[1] * inv_d;
        const float mean = (NEXT ? s[0] - c * s[NS - 1] : s[0]) * inv_d;
        const bool last_of_group = GATE && (t + 1 == t1 || (t + 1) % a.gate_rows == 0);
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const int v = threadIdx.x + u * blockDim.x;
            if (v >= nvec) continue;
            const size_t at = (size_t)t * a.d + (size_t)v * 8;
            float fu[8], fy[8], fo[8], fd[8], fg[8];
            up[u].get(fu);
            y[u].get(fy);
            if constexpr (NEXT) o[u].get(fo), dn[u].get(fd);
            if constexpr (GATE) gt[u].get(fg);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float dR = fu[i];
                if constexpr (NEXT) dR = fmaf(-c, fo[i], fmaf(rn * gn[u][i], fd[i], dR));
                const float hat = fy[i] * rs;
                const float e = dR * hat;
                if constexpr (GATE) {
                    acc_gate[u][i] = fmaf(e, g[u][i], acc_gate[u][i]);
                    acc[u][i] = fmaf(e, fg[i], acc[u][i]);
                    fy[i] = rs * fmaf(-hat, mean, dR * fg[i] * g[u][i]);
                } else {
                    acc[u][i] += e;
                    fy[i] = rs * fmaf(-hat, mean, dR * g[u][i]);
                }
                fu[i] = a.alpha * dR;
            }
            up[u].put(fu);
            up[u].store(dr + at);
            y[u].put(fy);
            y[u].store(a.dy + at);
            if constexpr (GATE) {
                if (last_of_group) {
                    const long g0 = (long)group * a.gate_rows;
                    const bool whole = g0 >= t0 && (t + 1 == a.T || t + 1 == g0 + a.gate_rows);
                    float* to = whole ? a.dgate + (size_t)group * a.d
                                      : a.part_gate + ((size_t)blockIdx.x * 2 + (group == t0 / a.gate_rows ? 0 : 1)) * a.d;
                    Vec8<float> q;
                    q.put(acc_gate[u]);
                    q.store(to + (size_t)v * 8);
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc_gate[u][i] = 0.f;
                }
            }
        }
    }
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
        const int v = threadIdx.x + u * blockDim.x;
        if (v >= nvec) continue;
        Vec8<float> q;
        q.put(acc[u]);
        q.store(a.part_w + (size_t)blockIdx.x * a.d + (size_t)v * 8);
        if constexpr (NEXT) {
            q.put(acc_next[u]);
            q.store(a.part_next + (size_t)blockIdx.x * a.d + (size_t)v * 8);
        }
    }
}

// Adds up what the CTAs left: blockIdx.y = 0: dw, 1: dw_next, 2 + b: the gate row that holds the boundary between the
// rows of CTA b and CTA b + 1, unless an earlier boundary lies in it too. 32 columns per block; warp i adds the partial
// rows i, i + 8, ..., then warp 0 adds the eight sums in order.
struct NormReduceArgs {
    const float *part_w, *part_next, *part_gate;
    float *dw, *dw_next, *dgate;
    int T, d, gate_rows, B;
};

constexpr int BNR_WARPS = 8;

__global__ void __launch_bounds__(BNR_WARPS * 32) block_norm_reduce_kernel(const NormReduceArgs a) {
    __shared__ float sums[BNR_WARPS][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int col = blockIdx.x * 32 + lane;
    const int job = blockIdx.y;
    int b0 = 0, b1 = a.B;  // CTAs to add
    long group = 0;
    float* to;
    if (job == 0) {
        to = a.dw;
    } else if (job == 1) {
        if (!a.part_next) return;
        to = a.dw_next;
    } else {
        const int b = job - 2;
        const int edge = norm_first_row(a.T, a.B, b + 1);
        group = edge / a.gate_rows;
        const long g0 = group * a.gate_rows, g1 = min(g0 + a.gate_rows, (long)a.T);
        if (edge == g0 || norm_first_row(a.T, a.B, b) > g0) return;  // no tokens before the edge; an earlier edge's group
        b0 = b;
        b1 = b + 2;
        while (b1 < a.B && norm_first_row(a.T, a.B, b1) < g1) ++b1;
        to = a.dgate + group * a.d;
    }
    float s = 0.f;
    if (col < a.d) {
#pragma unroll 4
        for (int b = b0 + warp; b < b1; b += BNR_WARPS) {
            const float* from;
            if (job == 0)
                from = a.part_w + (size_t)b * a.d;
            else if (job == 1)
                from = a.part_next + (size_t)b * a.d;
            else
                from = a.part_gate + ((size_t)b * 2 + (norm_first_row(a.T, a.B, b) / a.gate_rows == group ? 0 : 1)) * a.d;
            s += from[col];
        }
    }
    sums[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && col < a.d) {
        float all = sums[0][lane];
#pragma unroll
        for (int i = 1; i < BNR_WARPS; ++i) all += sums[i][lane];
        to[col] = all;
    }
}

}  // namespace moe
