// Grouped GEMM on e4m3 operands with a scale for each block of 128, on CTA pairs: the expert products of the layer with
// 8-bit weights and activations ("Expert Backend" of the blog post: one grouped GEMM over all experts).
//
//   out[r][c] = epilogue( sum_b sa[b][r] * sw[c / 128][b] * ( sum_{k in block b} A[r][k] * W[g][c][k] ) )
//
// The inner sums run on the tensor cores (tcgen05.mma kind::f8f6f4, fp32 accumulators in tensor memory), the outer sum in
// registers: fp32 scales are not powers of two, so an accumulator cannot stay in tensor memory from one K block to the next.
// As in gemm_swap.cuh the weight rows are the MMA's M dimension (256 per pair, 128 per CTA) and the group's token rows its N
// dimension (a multiple of 32, up to MAXN), so ragged groups cost little padding. TMEM lane = weight row, TMEM column = token.
//
// Roles (384 threads per CTA, both CTAs):
//   warp 0      TMA producer: per 128-wide K block (one ring stage) this CTA's 128 weight rows (one box) and its half of the
//               token rows (one box); completion is counted on the leader's full[stage].
//   warp 1      TMEM allocation; in the leader the MMA issuer: per K block four MMAs (K = 32 each) into the next of NBUF
//               TMEM buffers, so the tensor cores run ahead of the warps that read them.
//   warps 2, 3  scales: sa of the tile's tokens and sw of this CTA's weight rows into a ring by asynchronous copies (warp 2),
//               their products into another (warp 3). (Loaded through registers two K blocks ahead, the loads' latency set the
//               pace: 1.2 us per K block at any tile size.)
//   warps 4-11  two warpgroups, each the four lane quarters of half the tile's tokens: read a K block's sums from TMEM
//               (tcgen05.ld 16x256b: the layout of an MMA fragment, thread = 2 rows x 2 tokens of each 16 x 8 block),
//               multiply by the scales, add to the tile's sums in registers (MAXN / 2 per thread); after the last K block
//               round to bf16, transpose 8 x 8 blocks with stmatrix into [token][column] staging blocks, 16-byte stores.
//   gate|up: each quarter of 32 lanes holds 16 gate rows and the 16 up rows of the same columns (one TMA box over the weights
//   viewed as [G][f/16][2][16][K]), which the 16-lane loads bring into the same thread's registers: SwiGLU needs no exchange.
// What bounds it. Many rows: reading the sums back. A K block of 256 tokens is 512 cycles of MMA, but its sums leave TMEM, meet their
// scales and free the buffer after some 880 cycles in the warps, and the two buffers' hand-overs and the operands' arrival bring a step
// to 0.69 us. 4096 tokens on 4 of 32 experts of 2880 x 2880: gate|up 414-420 us (1.30 PFLOP/s), down 219 us (1.24 PFLOP/s); the
// same with no operand copies 286 / 140 us, with copies and no multiply-adds 358 / 195 us (the copies then run at 8 TB/s from L2).
// Each warpgroup's half of a buffer as MMAs and barriers of its own (four hand-overs in flight) measured the same, 419 / 225 us; a
// ring of six stages and TMEM loads two batches ahead gave nothing. Few rows: HBM, the weights streamed once (16 tokens on 8 of 64
// experts of 7168 x 2048: 199 us and 100 us, 6.5 and 6.4 TB/s), and where the tiles are few, their last round (4 tokens on 4 of 32
// experts of 2880 x 2880: 299 tiles on 74 pairs, five rounds for 4.04: 46 us, 4.7 TB/s; down 156 tiles, three for 2.1: 30 us).
#pragma once
#include <type_traits>

#include "common.cuh"
#include "fp8_quant.cuh"
#include "gemm.cuh"
#include "gemm_swap.cuh"
#include "sync.cuh"

namespace moe {

constexpr int G8_THREADS = 384;
constexpr int G8_SCALE_STAGES = 4;  // ring of products sa * sw
constexpr int G8_RAW_STAGES = 8;    // ring of scales as they arrive from memory

struct Gemm8Args {
    const int32_t* group_offsets;  // [G+1], device
    const float* sa;               // [ceil(K/128)][M]
    const float* sw;               // gate|up [G][2][ceil(f/128)][KB], down [G][ceil(n_out/128)][KB]
    int G, M, K, n_out, wblocks;   // wblocks: weight blocks (TILE_W output columns each) per group
    __nv_bfloat16* out;            // [M][n_out]
};

template <bool GATEUP, int MAXN>
struct Gemm8Shape {
    static constexpr int W_BYTES = 128 * F8_BLOCK;
    static constexpr int X_BYTES = MAXN / 2 * F8_BLOCK;
    static constexpr int STAGE_BYTES = W_BYTES + X_BYTES;
    static constexpr int STAGES = MAXN == 256 ? 5 : (MAXN == 128 ? 7 : 8);
    static constexpr int NBUF = 512 / MAXN;
    static constexpr int TILE_W = GATEUP ? 128 : 256;
    static constexpr int SCALE_BYTES = (GATEUP ? 2 : 1) * MAXN * 4;
    static constexpr int RAW_FLOATS = MAXN + 4;
    static constexpr int EPI_BYTES = 8 * 2 * 2048;  // two staging blocks per warp
    static constexpr int BAR_BYTES = 512;
    static constexpr int TABLE_BYTES = (2 * (GG_MAX_GROUPS + 1) * 4 + 127) / 128 * 128;
    static constexpr int SMEM_BYTES =
        1024 + STAGES * STAGE_BYTES + EPI_BYTES + G8_SCALE_STAGES * SCALE_BYTES +
        G8_RAW_STAGES * RAW_FLOATS * 4 + BAR_BYTES + TABLE_BYTES;
    static_assert(STAGE_BYTES % 1024 == 0, "stage bases stay 1024-byte aligned");
    static_assert(SMEM_BYTES <= 232448, "shared memory");
    static_assert((2 * STAGES + 2 * NBUF + 2 * G8_SCALE_STAGES + 2 * G8_RAW_STAGES + 2) * 8 + 8 <= BAR_BYTES, "barrier area");
};

// token boxes of 128, 64, 32, 16 rows
struct Fp8Maps {
    CUtensorMap x[4];
};

// D (256 rows) (+)= A B^T over 32 K elements of e4m3, fp32 accumulator; CTA pair, as umma_bf16_ss_pair.
__device__ __forceinline__ void umma_e4m3_ss_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                  uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Instruction descriptor for kind::f8f6f4, A and B e4m3 (format 0), both K-major, fp32 accumulator (fields as idesc_bf16_f32).
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
    return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// Start loading 16 lanes x 32 columns of fp32 from TMEM. Thread t gets, for each block j of 8 columns, lane t / 4 and
// columns 2 (t % 4), + 1 in r[4j], r[4j + 1], and lane t / 4 + 8 in r[4j + 2], r[4j + 3]. The registers are valid after
// tmem_wait_ld on them.
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, float (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
        : "r"(taddr)
        : "memory");
}
// Wait for this warp's TMEM loads; the registers they write pass through, so nothing reads them earlier.
__device__ __forceinline__ void tmem_wait_ld(float (&a)[16], float (&b)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(a[0]), "+f"(a[1]), "+f"(a[2]), "+f"(a[3]), "+f"(a[4]), "+f"(a[5]), "+f"(a[6]), "+f"(a[7]), "+f"(a[8]),
                   "+f"(a[9]), "+f"(a[10]), "+f"(a[11]), "+f"(a[12]), "+f"(a[13]), "+f"(a[14]), "+f"(a[15]), "+f"(b[0]),
                   "+f"(b[1]), "+f"(b[2]), "+f"(b[3]), "+f"(b[4]), "+f"(b[5]), "+f"(b[6]), "+f"(b[7]), "+f"(b[8]), "+f"(b[9]),
                   "+f"(b[10]), "+f"(b[11]), "+f"(b[12]), "+f"(b[13]), "+f"(b[14]), "+f"(b[15])
                 :
                 : "memory");
}

// acc += {v0, v1} * s
__device__ __forceinline__ void fma2_acc(float2& acc, float v0, float v1, const float2& s) {
    const uint64_t r = fma2(pair2(v0, v1), pair2(s.x, s.y), pair2(acc.x, acc.y));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(acc.x), "=f"(acc.y) : "l"(r));
}

// Register shares of the warpgroups (setmaxnreg): the block is launched with 384 x 168 = 64,512 registers, which the
// 128 x 72 of warps 0-3 and the 256 x 216 of the others use up exactly.
template <int R>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}

// Asynchronous copy of one float (zero where `inside` is false: nothing is read), and an arrival on `bar` once every such copy
// of this thread so far has landed (counted among the barrier's expected arrivals).
__device__ __forceinline__ void cp_async_f32(float* dst, const float* src, bool inside) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(inside ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_mbar_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Four 8 x 8 blocks of 16-bit elements, each stored transposed: lane 8 m + i gives the address of row i of block m.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t saddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(saddr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}

// Send a staged block of 32 rows (row0 .. row0 + 31 of out [M][ld]) x COLS columns from col0: 16-byte stores of the rows
// < row_end and columns < col_end. The staging rows are COLS * 2 bytes, their 16-byte units XORed so that the 8 rows of
// an 8 x 8 block fall in different banks. (Plain stores: a TMA store per block made the warps wait for the engine to read the
// staging buffers, about 1000 cycles per 32 tokens.)
template <int COLS>
__device__ __forceinline__ uint32_t staged_unit(int row, int unit) {
    return (uint32_t)(row * COLS * 2 + ((unit ^ (COLS == 32 ? (row >> 1) & 3 : (row >> 2) & 1)) << 4));
}
template <int COLS>
__device__ __forceinline__ void store_staged_rows(const uint8_t* stage, int lane, __nv_bfloat16* out, int ld, int row0, int row_end,
                                                  int col0, int col_end) {
    constexpr int UNITS = COLS / 8, ROWS = 32 / UNITS;  // rows per store instruction
    __syncwarp();
    const int u = lane % UNITS;
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
        const int row = i * ROWS + lane / UNITS;
        const uint4 val = *reinterpret_cast<const uint4*>(stage + staged_unit<COLS>(row, u));
        if (row0 + row < row_end && col0 + u * 8 < col_end)
            *reinterpret_cast<uint4*>(out + (size_t)(row0 + row) * ld + col0 + u * 8) = val;
    }
}

template <bool GATEUP, int MAXN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(G8_THREADS, 1)
    grouped_gemm_fp8_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ Fp8Maps tmX,
                            const Gemm8Args args, int weights_streamed_once) {
    using S = Gemm8Shape<GATEUP, MAXN>;
    constexpr int STAGES = S::STAGES, NBUF = S::NBUF;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* stages = smem;
    uint8_t* epi = smem + STAGES * S::STAGE_BYTES;
    uint8_t* scales = epi + S::EPI_BYTES;
    float* raw = reinterpret_cast<float*>(scales + G8_SCALE_STAGES * S::SCALE_BYTES);
    uint64_t* full_bar = reinterpret_cast<uint64_t*>(raw + G8_RAW_STAGES * S::RAW_FLOATS);  // used in the leader
    uint64_t* empty_bar = full_bar + STAGES;
    uint64_t* tfull_bar = empty_bar + STAGES;  // [NBUF]
    uint64_t* tempty_bar = tfull_bar + NBUF;   // [NBUF], used in the leader
    uint64_t* sfull_bar = tempty_bar + NBUF;   // [G8_SCALE_STAGES]
    uint64_t* sempty_bar = sfull_bar + G8_SCALE_STAGES;
    uint64_t* rfull_bar = sempty_bar + G8_SCALE_STAGES;  // [G8_RAW_STAGES]
    uint64_t* rempty_bar = rfull_bar + G8_RAW_STAGES;
    uint64_t* final_bar = rempty_bar + G8_RAW_STAGES;
    uint64_t* never_bar = final_bar + 1;  // nothing arrives on it (test_stall)
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(never_bar + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int32_t* s_off = reinterpret_cast<int32_t*>(reinterpret_cast<uint8_t*>(full_bar) + S::BAR_BYTES);
    int32_t* s_tp = s_off + (GG_MAX_GROUPS + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int cluster = blockIdx.x >> 1, n_clusters = gridDim.x >> 1;
    const int G = args.G;
    const int KB = (args.K + F8_BLOCK - 1) / F8_BLOCK;
    const int wblocks = args.wblocks;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full_bar[s], 1);
            mbar_init(&empty_bar[s], 1);
        }
        for (int b = 0; b < NBUF; ++b) {
            mbar_init(&tfull_bar[b], 1);
            mbar_init(&tempty_bar[b], 16);  // the warps that read it, of both CTAs
        }
        for (int s = 0; s < G8_SCALE_STAGES; ++s) {
            mbar_init(&sfull_bar[s], 32);
            mbar_init(&sempty_bar[s], 8);
        }
        for (int s = 0; s < G8_RAW_STAGES; ++s) {
            mbar_init(&rfull_bar[s], 32);
            mbar_init(&rempty_bar[s], 32);
        }
        mbar_init(final_bar, 1);
        mbar_init(never_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmW);
#pragma unroll
        for (int i = 0; i < 4; ++i) tma_prefetch_desc(&tmX.x[i]);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, 512);
        tmem_relinquish_pair();
    }
    grid_dep_wait();  // inputs below come from earlier kernels in the stream
    grid_dep_trigger();
    for (int g = threadIdx.x; g <= G; g += G8_THREADS) {
        int v = args.group_offsets[g];
        if (v < 0 || v > args.M) {
            flag_error(MOE_DEVERR_GROUP_RANGE);
            v = min(max(v, 0), args.M);
        }
        s_off[g] = v;
    }
    __syncthreads();
    if (warp == 0) {  // tile prefix over groups: tiles(g) = ceil(rows / MAXN) * wblocks
        const int per = (G + 31) / 32;
        const int g0 = lane * per, g1 = min(g0 + per, G);
        int local = 0;
        for (int g = g0; g < g1; ++g) {
            const int n = s_off[g + 1] - s_off[g];
            if (n < 0) flag_error(MOE_DEVERR_GROUP_RANGE);
            local += (max(n, 0) + MAXN - 1) / MAXN * wblocks;
        }
        int incl = local;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        int run = incl - local;
        for (int g = g0; g < g1; ++g) {
            s_tp[g] = run;
            run += (max(s_off[g + 1] - s_off[g], 0) + MAXN - 1) / MAXN * wblocks;
        }
        if (lane == 31) s_tp[G] = incl;
    }
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers are initialised before any cross-CTA arrive or TMA signal
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;
    const int total = s_tp[G];
    const uint64_t limit = wait_limit_ns();

    // tile -> group g, weight block wb, first token row r0 (absolute), rows in the tile (<= MAXN)
    auto locate = [&](int tile, int& g, int& wb, int& r0, int& rows) {
        int lo = 0, hi = G - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s_tp[mid] <= tile)
                lo = mid;
            else
                hi = mid - 1;
        }
        g = lo;
        const int n = s_off[g + 1] - s_off[g];
        const int tt = (n + MAXN - 1) / MAXN;
        const int local = tile - s_tp[g];
        wb = local / tt;
        const int ti = local - wb * tt;
        r0 = s_off[g] + ti * MAXN;
        rows = min(MAXN, n - ti * MAXN);
    };

    if (warp < 4) {
        if constexpr (MAXN == 256) fewer_registers<72>();
        if (warp == 0) {
            // ---------------- TMA producer (both CTAs) ----------------
            const uint64_t pol_x = l2_policy_evict_last();
            const uint64_t pol_w = weights_streamed_once ? l2_policy_evict_first() : l2_policy_evict_normal();
            int stage = 0;
            uint32_t phase = 0;
            long issued = 0;
            bool ok = true;
            for (int tile = cluster; tile < total && ok; tile += n_clusters) {
                int g, wb, r0, rows;
                locate(tile, g, wb, r0, rows);
                const int half = (rows + 31) / 32 * 16;  // token rows per CTA (N / 2), in the smallest box that holds them
                const int bi = swap_box_index(half);
                const int xrow0 = r0 + (int)rank * half;
                const uint32_t tx = 2u * (uint32_t)(S::W_BYTES + (128 >> bi) * F8_BLOCK);
                for (int kb = 0; kb < KB; ++kb) {
                    if (lane == 0) {
                        ok = mbar_wait_within(&empty_bar[stage], phase ^ 1u, abort_flag, limit);
                        if (ok) {
                            uint8_t* sw = stages + stage * S::STAGE_BYTES;
                            const uint32_t bar = mapa_shared(smem_u32(&full_bar[stage]), 0);
                            if (leader) mbar_arrive_expect_tx(&full_bar[stage], tx);
                            if constexpr (GATEUP)
                                tma_load_5d_pair(sw, &tmW, bar, kb * F8_BLOCK, 0, 0, wb * 8 + 4 * (int)rank, g, pol_w);
                            else
                                tma_load_3d_pair(sw, &tmW, bar, kb * F8_BLOCK, wb * 256 + 128 * (int)rank, g, pol_w);
                            tma_load_2d_pair(sw + S::W_BYTES, &tmX.x[bi], bar, kb * F8_BLOCK, xrow0, pol_x);
                        }
                    }
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (!ok) break;
                    ++issued;
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // the leader's full barriers count both CTAs' copies: it waits for the last ones (bounded)
            if (lane == 0 && leader) {
                for (long n = issued > STAGES ? issued - STAGES : 0; n < issued; ++n)
                    mbar_wait_drain(&full_bar[n % STAGES], (uint32_t)((n / STAGES) & 1));
            }
            __syncwarp();
        } else if (warp == 1) {
            // ---------------- MMA issuer (leader only) ----------------
            // This warp's own time per K block has to stay below the MMAs' (512 cycles at 256 tokens): the whole warp runs the
            // loop, so that descriptors and addresses stay in uniform registers, and the next K block's barriers are polled
            // between this one's MMAs and commits.
            if (leader) {
                int stage = 0, buf = 0;
                uint32_t phase = 0, buf_phase = 0;
                const bool elected = elect_one();
                bool ok = __all_sync(0xffffffffu, test_stall(never_bar, abort_flag));
                bool ready = false;  // the coming K block's barriers were seen complete
                for (int tile = cluster; tile < total && ok; tile += n_clusters) {
                    int g, wb, r0, rows;
                    locate(tile, g, wb, r0, rows);
                    const uint32_t idesc = idesc_e4m3_f32(256, (rows + 31) / 32 * 32);
                    for (int kb = 0; kb < KB; ++kb) {
                        if (!ready) {
                            ok = mbar_wait_within(&tempty_bar[buf], buf_phase ^ 1u, abort_flag, limit) &&
                                 mbar_wait_within(&full_bar[stage], phase, abort_flag, limit);
                            ok = __all_sync(0xffffffffu, ok);
                            if (!ok) break;
                        }
                        tc_fence_after_sync();
                        const uint32_t sa = smem_u32(stages + stage * S::STAGE_BYTES);
                        const uint64_t wdesc = smem_desc_sw128(sa), xdesc = smem_desc_sw128(sa + S::W_BYTES);
                        const uint32_t d_tmem = tmem_base + (uint32_t)(buf * MAXN);
                        uint64_t* const tfull = &tfull_bar[buf];
                        uint64_t* const empty = &empty_bar[stage];
                        if (elected) {
#pragma unroll
                            for (int k = 0; k < F8_BLOCK / 32; ++k)
                                umma_e4m3_ss_pair(d_tmem, wdesc + 2 * k, xdesc + 2 * k, idesc, k != 0 ? 1u : 0u);
                        }
                        if (++stage == STAGES) {
                            stage = 0;
                            phase ^= 1u;
                        }
                        if (++buf == NBUF) {
                            buf = 0;
                            buf_phase ^= 1u;
                        }
                        const bool te = mbar_test_wait(smem_u32(&tempty_bar[buf]), buf_phase ^ 1u);
                        const bool fu = mbar_test_wait(smem_u32(&full_bar[stage]), phase);
                        if (elected) {
                            umma_commit_pair_multicast(tfull, 0x3);
                            umma_commit_pair_multicast(empty, 0x3);
                        }
                        ready = __all_sync(0xffffffffu, te && fu);
                    }
                }
                if (elected) umma_commit_pair(final_bar);
            }
            __syncwarp();
        } else {
            // ---------------- scales (both CTAs) ----------------
            // warp 2: raw scales of each step (tile, K block) into a ring, by asynchronous 4-byte copies (rows start anywhere):
            // sa of the tile's tokens, then the one or two sw of this CTA's weight rows. Nothing waits for a copy here, so a ring's
            // depth of them is in flight. warp 3: their products into the ring the sums read.
            constexpr int PER = MAXN / 32;
            const int nblk = (args.n_out + F8_BLOCK - 1) / F8_BLOCK;
            int slot = 0, cslot = 0;
            uint32_t phase = 0, c_phase = 0;
            bool ok = true;
            for (int tile = cluster; tile < total && ok; tile += n_clusters) {
                int g, wb, r0, rows;
                locate(tile, g, wb, r0, rows);
                if (warp == 2) {
                    const float* w0;
                    if constexpr (GATEUP)
                        w0 = args.sw + (((size_t)g * 2 + (lane & 1)) * nblk + wb) * KB;
                    else
                        w0 = args.sw + ((size_t)g * nblk + min(2 * wb + (int)rank, nblk - 1)) * KB;
                    const float* a0 = args.sa + r0;
                    for (int kb = 0; kb < KB; ++kb) {
                        ok = mbar_wait_within(&rempty_bar[slot], phase ^ 1u, abort_flag, limit);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        float* to = raw + slot * S::RAW_FLOATS;
#pragma unroll
                        for (int i = 0; i < PER; ++i) {
                            const int t = lane + 32 * i;
                            cp_async_f32(to + t, a0 + (size_t)kb * args.M + (t < rows ? t : 0), t < rows);
                        }
                        if (lane < 2) cp_async_f32(to + MAXN + lane, w0 + kb, true);
                        cp_async_mbar_arrive(&rfull_bar[slot]);
                        if (++slot == G8_RAW_STAGES) {
                            slot = 0;
                            phase ^= 1u;
                        }
                    }
                } else {
                    bool ready = false;
                    for (int kb = 0; kb < KB; ++kb) {
                        if (!ready) {
                            ok = mbar_wait_within(&rfull_bar[slot], phase, abort_flag, limit) &&
                                 mbar_wait_within(&sempty_bar[cslot], c_phase ^ 1u, abort_flag, limit);
                            ok = __all_sync(0xffffffffu, ok);
                            if (!ok) break;
                        }
                        const float* from = raw + slot * S::RAW_FLOATS;
                        float* to = reinterpret_cast<float*>(scales + cslot * S::SCALE_BYTES);
                        uint64_t* const r_freed = &rempty_bar[slot];
                        uint64_t* const filled = &sfull_bar[cslot];
                        if (++slot == G8_RAW_STAGES) {
                            slot = 0;
                            phase ^= 1u;
                        }
                        if (++cslot == G8_SCALE_STAGES) {
                            cslot = 0;
                            c_phase ^= 1u;
                        }
                        const bool next = mbar_test_wait(smem_u32(&rfull_bar[slot]), phase) &
                                          mbar_test_wait(smem_u32(&sempty_bar[cslot]), c_phase ^ 1u);
                        const float b0 = from[MAXN], b1 = from[MAXN + 1];
#pragma unroll
                        for (int i = 0; i < PER; ++i) {
                            // gate|up: the gate's products of two tokens, then the up rows', so that one load brings all four
                            const int t = lane + 32 * i;
                            const float a = from[t];
                            if constexpr (GATEUP) {
                                to[4 * (t >> 1) + (t & 1)] = a * b0;
                                to[4 * (t >> 1) + 2 + (t & 1)] = a * b1;
                            } else {
                                to[t] = a * b0;
                            }
                        }
                        mbar_arrive(r_freed);
                        mbar_arrive(filled);
                        ready = kb + 1 < KB && __all_sync(0xffffffffu, next);
                    }
                }
            }
            if (warp == 2) cp_async_wait_all();  // no copy is in flight when the CTA leaves
            __syncwarp();
        }
    } else {
        // ---------------- scaled sums and epilogue (warps 4-11, both CTAs) ----------------
        if constexpr (MAXN == 256) more_registers<216>();
        constexpr int CHUNKS = MAXN / 32;  // 16-token chunks of this warpgroup's half
        const int q = warp & 3, hw = (warp - 4) >> 2;
        const uint32_t tempty_leader = mapa_shared(smem_u32(tempty_bar), 0);
        bool ready = false;  // the coming K block's sums and scales were seen complete
        uint8_t* stage_base = epi + (warp - 4) * 4096;
        int buf = 0, slot = 0;
        uint32_t buf_phase = 0, s_phase = 0;
        bool ok = true;
        for (int tile = cluster; tile < total && ok; tile += n_clusters) {
            int g, wb, r0, rows;
            locate(tile, g, wb, r0, rows);
            const int nh = (rows + 31) / 32 * 16, first = hw * nh;  // this warpgroup's tokens
            float2 acc[CHUNKS][2][4];
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[c][0][i] = acc[c][1][i] = make_float2(0.f, 0.f);
            // The K blocks, straight through for each number of 32-token batches (the last may reach past this half's tokens:
            // columns nothing is stored from). A look at a barrier takes some 200 cycles here, also when it is complete, so the
            // next K block's are looked at behind this one's last loads and the multiply-adds in their shadow.
            const auto mainloop = [&](auto batches) {
                constexpr int NB = decltype(batches)::value;
                for (int kb = 0; kb < KB; ++kb) {
                    if (!ready) {
                        ok = mbar_wait_within(&sfull_bar[slot], s_phase, abort_flag, limit) &&
                             mbar_wait_within(&tfull_bar[buf], buf_phase, abort_flag, limit);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                    }
                    tc_fence_after_sync();
                    const uint32_t t0 = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * MAXN + first);
                    const float* sc = reinterpret_cast<const float*>(scales + slot * S::SCALE_BYTES) + (GATEUP ? 2 : 1) * (first + 2 * (lane & 3));
                    const uint32_t freed = tempty_leader + (uint32_t)(buf * 8);
                    uint64_t* const s_freed = &sempty_bar[slot];
                    if (++buf == NBUF) {
                        buf = 0;
                        buf_phase ^= 1u;
                    }
                    if (++slot == G8_SCALE_STAGES) {
                        slot = 0;
                        s_phase ^= 1u;
                    }
                    bool next = false;
                    float v[2][2][16];
                    tmem_ld_16x32(t0, v[0][0]);
                    tmem_ld_16x32(t0 + (16u << 16), v[0][1]);
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        float2 s0[4], s1[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if constexpr (GATEUP) {
                                const float4 both = *reinterpret_cast<const float4*>(sc + 64 * b + 16 * j);
                                s0[j] = make_float2(both.x, both.y);
                                s1[j] = make_float2(both.z, both.w);
                            } else {
                                s0[j] = s1[j] = *reinterpret_cast<const float2*>(sc + 32 * b + 8 * j);
                            }
                        }
                        tmem_wait_ld(v[b & 1][0], v[b & 1][1]);
                        if (b + 1 < NB) {
                            tmem_ld_16x32(t0 + (uint32_t)(32 * (b + 1)), v[(b + 1) & 1][0]);
                            tmem_ld_16x32(t0 + (uint32_t)(32 * (b + 1)) + (16u << 16), v[(b + 1) & 1][1]);
                        } else {  // everything of this K block is in registers
                            tc_fence_before_sync();
                            __syncwarp();
                            if (lane == 0) {
                                mbar_arrive_remote(freed);
                                mbar_arrive(s_freed);
                            }
                            next = mbar_test_wait(smem_u32(&sfull_bar[slot]), s_phase) &
                                   mbar_test_wait(smem_u32(&tfull_bar[buf]), buf_phase);
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const int r = 4 * j + 2 * i;
                                fma2_acc(acc[2 * b + (j >> 1)][0][2 * (j & 1) + i], v[b & 1][0][r], v[b & 1][0][r + 1], s0[j]);
                                fma2_acc(acc[2 * b + (j >> 1)][1][2 * (j & 1) + i], v[b & 1][1][r], v[b & 1][1][r + 1], s1[j]);
                            }
                    }
                    ready = kb + 1 < KB && __all_sync(0xffffffffu, next);
                }
            };
            if constexpr (MAXN == 64) {
                mainloop(std::integral_constant<int, 1>());
            } else if (MAXN == 128 || nh <= 64) {
                if (nh <= 32)
                    mainloop(std::integral_constant<int, 1>());
                else
                    mainloop(std::integral_constant<int, 2>());
            } else {
                if (nh <= 96)
                    mainloop(std::integral_constant<int, 3>());
                else
                    mainloop(std::integral_constant<int, MAXN == 256 ? 4 : 2>());
            }
            if (!ok) break;
            const int row_first = r0 + first, row_end = min(r0 + rows, row_first + nh);
            const int col0 = GATEUP ? wb * 128 + 64 * (int)rank + 16 * q : wb * 256 + 128 * (int)rank + 32 * q;
            if (col0 >= args.n_out) continue;
#pragma unroll
            for (int cc = 0; cc < CHUNKS; cc += 2) {  // blocks of 32 tokens
                if (row_first + 16 * cc >= row_end) break;
                uint8_t* my_stage = stage_base + (cc / 2 & 1) * 2048;
#pragma unroll
                for (int c = cc; c < cc + 2; ++c) {
                    if constexpr (GATEUP) {
                        float h[8];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            h[2 * i] = swiglu(acc[c][0][i].x, acc[c][1][i].x);
                            h[2 * i + 1] = swiglu(acc[c][0][i].y, acc[c][1][i].y);
                        }
                        // blocks (columns 0-7 | 8-15) of tokens 0-7, then of tokens 8-15
                        const int row = 16 * (c - cc) + (lane & 7) + ((lane >> 4) << 3);
                        stmatrix_x4_trans(smem_u32(my_stage) + staged_unit<16>(row, (lane >> 3) & 1), pack_bf16x2(h[0], h[1]),
                                          pack_bf16x2(h[2], h[3]), pack_bf16x2(h[4], h[5]), pack_bf16x2(h[6], h[7]));
                    } else {
#pragma unroll
                        for (int j = 0; j < 2; ++j) {  // 8 tokens, 32 columns
                            const int row = 16 * (c - cc) + 8 * j + (lane & 7);
                            stmatrix_x4_trans(smem_u32(my_stage) + staged_unit<32>(row, lane >> 3),
                                              pack_bf16x2(acc[c][0][2 * j].x, acc[c][0][2 * j].y),
                                              pack_bf16x2(acc[c][0][2 * j + 1].x, acc[c][0][2 * j + 1].y),
                                              pack_bf16x2(acc[c][1][2 * j].x, acc[c][1][2 * j].y),
                                              pack_bf16x2(acc[c][1][2 * j + 1].x, acc[c][1][2 * j + 1].y));
                        }
                    }
                }
                store_staged_rows<GATEUP ? 16 : 32>(my_stage, lane, args.out, args.n_out, row_first + 16 * cc, row_end, col0,
                                                    args.n_out);
            }
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1 && leader) {
        if (lane == 0) mbar_wait_drain(final_bar, 0);  // the pair's MMAs have finished
        __syncwarp();
    }
    cluster_sync();  // no CTA leaves while its peer may still signal its barriers or read its smem
    tc_fence_after_sync();
    if (warp == 1) tmem_dealloc_pair(tmem_base, 512);
}

}  // namespace moe
