// e4m3 values with one fp32 scale per block of 128: activations per row and 128 columns, weights per 128 x 128 block.
//
// With top the largest magnitude of a block: scale = top / 448 (1 for a block of zeros), value = 448 x / top rounded to the
// nearest e4m3 (ties to even). The quotient is decided exactly: x is a bf16 value, so 448 x is a whole number of at most 11
// bits times a power of two and top one of 8 bits; their quotient either is a number of few bits (perhaps a tie between two
// e4m3 values) or differs from every such number by more than 2^-17 of itself. A quotient q0 = a * (1 / m) corrected once by its
// exactly computed remainder (a - q0 m, one fma) is within an ulp of a / m and is a / m itself where that is a fp32 number, so
// the rounding to e4m3 comes out as that of the exact quotient. (Residual correction: Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990.)
// HBM bounds both encoders: 16384 rows of 2880, 29 us (94 MB read, 47 MB written: 22 us at a copy's rate); the same number of rows
// gathered from 4096, which stay in L2, 23 us (11).
#pragma once
#include <cuda_fp8.h>

#include "common.cuh"

namespace moe {

constexpr int F8_BLOCK = 128;
constexpr float F8_MAX = 448.f;

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair2(float lo, float hi) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
    return v;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t v;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t v;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
    return v;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t v;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}

struct F8Scaler {
    uint64_t c, minus_m, r;  // each twice
    float scale;
    __device__ __forceinline__ explicit F8Scaler(float top) {
        const bool some = top > 0.f;
        // p = 2^k with top * p near 1 (its exponent kept where p, 448 p and 1 / (top p) are normal numbers)
        const int e = min(max((int)(__float_as_uint(top) >> 23) & 255, 16), 252);
        const float p = __uint_as_float((uint32_t)(254 - e) << 23);
        const float m = some ? top * p : 1.f;
        const float rcp = __frcp_rn(m);
        c = pair2(p * F8_MAX, p * F8_MAX);
        minus_m = pair2(-m, -m);
        r = pair2(rcp, rcp);
        scale = some ? __fdiv_rn(top, F8_MAX) : 1.f;
    }
    // two bf16 values -> two e4m3 bytes
    __device__ __forceinline__ uint32_t two(uint32_t v) const {
        const uint64_t a = mul2(pair2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u)), c);
        const uint64_t q = mul2(a, r);
        const uint64_t out = fma2(fma2(q, minus_m, a), r, q);
        float lo, hi;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(out));
        return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
    }
    __device__ __forceinline__ uint2 eight(const uint4& v) const {
        return make_uint2(two(v.x) | two(v.y) << 16, two(v.z) | two(v.w) << 16);
    }
};

// The largest magnitude of 8 bf16 values (a NaN counts only beside another).
__device__ __forceinline__ float top_of(const uint4& v) {
    const auto abs2 = [](uint32_t u) {
        u &= 0x7fff7fffu;
        return *reinterpret_cast<const __nv_bfloat162*>(&u);
    };
    const __nv_bfloat162 m = __hmax2(__hmax2(abs2(v.x), abs2(v.y)), __hmax2(abs2(v.z), abs2(v.w)));
    return fmaxf(__low2float(m), __high2float(m));
}

// Rows of x (row r of the output is row row_src[r] of x [T][K], or row r without row_src): q [R][K], s [ceil(K/128)][R].
// A warp takes F8_CHUNK_VEC vectors of a row (blockIdx.y: which), 4 lanes a block of 128; the 8 warps of a CTA take 8 consecutive
// rows, so their scales fill a 32-byte sector. HBM-bound: 3 bytes moved per element; the next row's loads go out before this
// row's arithmetic. (With 16 lanes to a block the reciprocal and the scale, some 60 instructions, came to every 8 values
// instead of every 32: 32 us instead of 23 for 16,384 rows of 2880 gathered from 4096.)
constexpr int F8_CHUNK_VEC = 128;  // 16-byte vectors: 4 per lane

__global__ void __launch_bounds__(256) fp8_row_quantize_kernel(const __nv_bfloat16* __restrict__ x,
                                                               const int32_t* __restrict__ row_src, int T, int K, int R,
                                                               uint8_t* __restrict__ q, float* __restrict__ s) {
    grid_dep_wait();
    grid_dep_trigger();
    const int lane = threadIdx.x & 31;
    const int nvec = K >> 3, v0 = blockIdx.y * F8_CHUNK_VEC + (lane >> 2) * 16 + (lane & 3);
    const int step = gridDim.x * 8;
    const auto load = [&](int row, uint4 (&v)[4]) {
        int src = row;
        if (row_src) {
            src = __ldg(row_src + row);
            if (src < 0 || src >= T) {
                if (lane == 0) flag_error(MOE_DEVERR_ROW_RANGE);
                src = -1;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = make_uint4(0, 0, 0, 0);
            if (src >= 0 && v0 + 4 * i < nvec) v[i] = __ldg(reinterpret_cast<const uint4*>(x + (size_t)src * K) + v0 + 4 * i);
        }
    };
    uint4 v[4], next[4];
    int row = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row < R) load(row, v);
    for (; row < R; row += step) {
        if (row < R - step) load(row + step, next);
        float top = fmaxf(fmaxf(top_of(v[0]), top_of(v[1])), fmaxf(top_of(v[2]), top_of(v[3])));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const F8Scaler f(top);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (v0 + 4 * i < nvec) *reinterpret_cast<uint2*>(q + (size_t)row * K + (size_t)(v0 + 4 * i) * 8) = f.eight(v[i]);
            v[i] = next[i];
        }
        if ((lane & 3) == 0 && v0 < nvec) s[(size_t)(v0 >> 4) * R + row] = f.scale;
    }
}

// Weights w [G][N][K]: one CTA per 128 x 128 block. q [G][N][K], s [G][ceil(N/128)][ceil(K/128)]. Once per layer.
__global__ void __launch_bounds__(256) fp8_block_quantize_kernel(const __nv_bfloat16* __restrict__ w, int N, int K,
                                                                 long blocks, uint8_t* __restrict__ q, float* __restrict__ s) {
    __shared__ float red[2][8];
    grid_dep_wait();
    grid_dep_trigger();
    const int kb = (K + F8_BLOCK - 1) / F8_BLOCK, nb = (N + F8_BLOCK - 1) / F8_BLOCK;
    int turn = 0;
    for (long b = blockIdx.x; b < blocks; b += gridDim.x, turn ^= 1) {
        const int k0 = (int)(b % kb) * F8_BLOCK + (threadIdx.x & 15) * 8;
        const long row0 = b / kb;
        const long g = row0 / nb;
        const int n0 = (int)(row0 - g * nb) * F8_BLOCK + (threadIdx.x >> 4);
        uint4 v[8];
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = make_uint4(0, 0, 0, 0);
            if (n0 + 16 * i < N && k0 < K)
                v[i] = *reinterpret_cast<const uint4*>(w + ((size_t)g * N + n0 + 16 * i) * K + k0);
            top = fmaxf(top, top_of(v[i]));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if ((threadIdx.x & 31) == 0) red[turn][threadIdx.x >> 5] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, red[turn][i]);
        const F8Scaler f(top);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (n0 + 16 * i < N && k0 < K)
                *reinterpret_cast<uint2*>(q + ((size_t)g * N + n0 + 16 * i) * K + k0) = f.eight(v[i]);
        if (threadIdx.x == 0) s[b] = f.scale;
    }
}

}  // namespace moe
