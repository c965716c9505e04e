// The library's translation unit: the layer (moe.cu) and the operators that stand beside its calls: the few-token layer, the e4m3
// products, the norms around a block (declared in include/moe.h). One unit, so that the device error word, the wait limit and the
// host helpers have a single definition.
#include "moe.cu"

#include "block_norm.cuh"
#include "few_tokens.cuh"
#include "fp8_quant.cuh"
#include "gemm_fp8.cuh"

namespace {
// fp32 and int32 arrays (null ones are the caller's to allow)
template <typename... P>
bool aligned4(const P*... p) {
    return ((reinterpret_cast<uintptr_t>(p) | ...) & 3u) == 0;
}
}  // namespace

// ---- the whole layer for few tokens ----
namespace {

constexpr size_t kFewMaxSmem = 232448;  // 227 KB: the most a CTA can have

// Shared-memory limits of the kernels below, set once per device (as device_info does for the layer's own kernels), and the device.
moe_status_t operator_device(DeviceInfo& di) {
    moe_status_t st = device_info(di);
    if (st != MOE_OK) return st;
    static bool ready[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    std::lock_guard<std::mutex> lock(g_mu);
    if (e == cudaSuccess && !ready[dev]) {
        const cudaFuncAttribute a = cudaFuncAttributeMaxDynamicSharedMemorySize;
        e = cudaFuncSetAttribute(grouped_gemm_fp8_kernel<true, 256>, a, Gemm8Shape<true, 256>::SMEM_BYTES);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(grouped_gemm_fp8_kernel<false, 256>, a, Gemm8Shape<false, 256>::SMEM_BYTES);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(grouped_gemm_fp8_kernel<true, 128>, a, Gemm8Shape<true, 128>::SMEM_BYTES);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(grouped_gemm_fp8_kernel<false, 128>, a, Gemm8Shape<false, 128>::SMEM_BYTES);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(grouped_gemm_fp8_kernel<true, 64>, a, Gemm8Shape<true, 64>::SMEM_BYTES);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(grouped_gemm_fp8_kernel<false, 64>, a, Gemm8Shape<false, 64>::SMEM_BYTES);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(few_tokens_kernel<1>, a, (int)kFewMaxSmem);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(few_tokens_kernel<2>, a, (int)kFewMaxSmem);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(few_tokens_kernel<3>, a, (int)kFewMaxSmem);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(few_tokens_kernel<4>, a, (int)kFewMaxSmem);
        ready[dev] = e == cudaSuccess;
    }
    if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    return MOE_OK;
}

struct FewWorkspace {  // byte offsets: counters | h | parts
    size_t h, part, bytes;
    int n_counters, ldh;
};
FewWorkspace few_workspace(int T, int d, int f, int fs, int k) {
    FewWorkspace w;
    w.n_counters = 1 + (d + 31) / 32;
    w.ldh = f > fs ? f : fs;
    w.h = ((size_t)w.n_counters * 4 + 255) / 256 * 256;
    w.part = w.h + ((size_t)(T * k + (fs ? T : 0)) * w.ldh * 2 + 255) / 256 * 256;
    w.bytes = w.part + (size_t)FT_MAX_CTAS * 2 * 32 * (T <= 8 ? 8 : (T <= 16 ? 16 : 32)) * 4;
    return w;
}

template <int NT>
size_t few_smem(int slots, int E) {
    using S = FewShape<NT>;
    return (size_t)S::RING_BYTES + S::RED_BYTES + (size_t)FewTables::words(slots, E) * 4 + (size_t)(slots + 1) * 8 * NT;
}

// One CTA per SM, all of them resident at once (they meet at a barrier): a cooperative launch.
template <int NT>
cudaError_t launch_few(const FewArgs& a, int grid, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(FT_THREADS);
    cfg.dynamicSmemBytes = few_smem<NT>(a.T * a.k, a.E);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // as launch_pdl
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, few_tokens_kernel<NT>, a);
}

}  // namespace

// ---- e4m3 operands with a scale per block of 128 ----
namespace {

template <bool GATEUP, int MAXN>
moe_status_t launch_fp8(const uint8_t* a, const float* sa, const uint8_t* w, const float* sw, const int32_t* offsets, int G, int M,
                        int d, int f, moe_bf16_t* out, int sms, cudaStream_t stream) {
    using S = Gemm8Shape<GATEUP, MAXN>;
    CUtensorMap tw;
    Fp8Maps tx;
    const int K = GATEUP ? d : f, n_out = GATEUP ? f : d;
    const cuuint64_t k = (cuuint64_t)K, n = (cuuint64_t)n_out, g = (cuuint64_t)G;
    const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    moe_status_t st;
    if (GATEUP) {  // [G][2][f][K] as [G][f/16][2][16][K]: one box = four times 16 gate rows and the 16 up rows of their columns
        const cuuint64_t dims[5] = {k, 16, 2, n / 16, g};
        const cuuint64_t str[4] = {k, n * k, 16 * k, 2 * n * k};
        const cuuint32_t box[5] = {F8_BLOCK, 16, 2, 4, 1};
        st = make_tmap(&tw, w, 5, dims, str, box, u8);
    } else {
        const cuuint64_t dims[3] = {k, n, g};
        const cuuint64_t str[2] = {k, n * k};
        const cuuint32_t box[3] = {F8_BLOCK, 128, 1};
        st = make_tmap(&tw, w, 3, dims, str, box, u8);
    }
    const cuuint64_t xdims[2] = {k, (cuuint64_t)M};
    const cuuint64_t xstr[1] = {k};
    for (int i = 0; i < 4 && st == MOE_OK; ++i) {
        const cuuint32_t box[2] = {F8_BLOCK, (cuuint32_t)(128 >> i)};
        st = make_tmap(&tx.x[i], a, 2, xdims, xstr, box, u8);
    }
    if (st != MOE_OK) return st;
    Gemm8Args args;
    args.group_offsets = offsets;
    args.sa = sa;
    args.sw = sw;
    args.G = G;
    args.M = M;
    args.K = K;
    args.n_out = n_out;
    args.wblocks = (n_out + S::TILE_W - 1) / S::TILE_W;
    args.out = reinterpret_cast<__nv_bfloat16*>(out);
    const long upper = ((long)M / MAXN + G) * (long)args.wblocks;  // >= the real tile count
    const int clusters = (int)(upper < sms / 2 ? upper : sms / 2);
    const int streamed_once = (long)M <= (long)G * MAXN ? 1 : 0;
    const cudaError_t e = launch_pdl(grouped_gemm_fp8_kernel<GATEUP, MAXN>, dim3(2 * clusters), dim3(G8_THREADS), S::SMEM_BYTES,
                                     stream, tw, tx, args, streamed_once);
    return check_launch(GATEUP ? "grouped_gemm_gateup_fp8" : "grouped_gemm_down_fp8", e);
}

// Arguments of both products, then the launch. A tile covers up to 64, 128 or 256 token rows of a group: narrow tiles leave room for
// more ring stages, wide ones read a group's weights fewer times. Which is decided by the average rows per group, the only
// thing the host knows of the groups. Measured, groups within half of the average either way, gate|up / down in us:
//   32 groups, d = f = 2880       average 32: 64 rows 87 / 52, 128 rows 88 / 53      48: 64 rows 108 / 60, 128 rows 94 / 54
//                                 average 96: 128 rows 123 / 67, 256 rows 137 / 75   112: 128 rows 136 / 70, 256 rows 143 / 83
//                                 average 128: 128 rows 153 / 79, 256 rows 146 / 78
//   128 groups, d 2048, f 768     average 96: 128 rows 104 / 68, 256 rows 117 / 71   112: 128 rows 115 / 76, 256 rows 116 / 72
//                                 average 128: 128 rows 123 / 80, 256 rows 126 / 75
//   8 groups, d 4096, f 14336     average 96: 128 rows 193 / 92, 256 rows 220 / 112  112: 128 rows 231 / 133, 256 rows 235 / 115
//                                 average 128: 128 rows 275 / 133, 256 rows 245 / 118
// At 112 both products together are 20 us apart for 32 groups (128 rows the faster), 3 and 15 the other way for 128 and 8: 112 takes 128.
template <bool GATEUP>
moe_status_t gemm_fp8(const uint8_t* a, const float* sa, const uint8_t* w, const float* sw, const int32_t* offsets, int G, int M,
                      int d, int f, moe_bf16_t* out, cudaStream_t stream) {
    if (!w || !sw || !offsets || (M > 0 && (!a || !sa || !out))) return fail(MOE_ERR_INVALID_ARG, "null pointer argument");
    if (!aligned16(a) || !aligned16(w) || !aligned16(out))
        return fail(MOE_ERR_INVALID_ARG, "value and output pointers must be 16-byte aligned");
    if (!aligned4(offsets, sa, sw)) return fail(MOE_ERR_INVALID_ARG, "offsets or scales misaligned");
    if (G < 1 || G > GG_MAX_GROUPS) return fail(MOE_ERR_INVALID_ARG, "G=%d outside [1, %d]", G, GG_MAX_GROUPS);
    if (M < 0) return fail(MOE_ERR_INVALID_ARG, "M=%d < 0", M);
    if (d < 16 || f < 16 || d % 16 || f % 16)
        return fail(MOE_ERR_INVALID_ARG, "d=%d and f=%d must be positive multiples of 16 (16-byte rows of e4m3)", d, f);
    DeviceInfo di;
    moe_status_t st = operator_device(di);
    if (st != MOE_OK) return st;
    if (di.sms < 2) return fail(MOE_ERR_UNSUPPORTED, "the fp8 GEMM needs CTA pairs");
    if (M == 0) return MOE_OK;
    if ((long)M <= 32L * G) return launch_fp8<GATEUP, 64>(a, sa, w, sw, offsets, G, M, d, f, out, di.sms, stream);
    if ((long)M <= 112L * G) return launch_fp8<GATEUP, 128>(a, sa, w, sw, offsets, G, M, d, f, out, di.sms, stream);
    return launch_fp8<GATEUP, 256>(a, sa, w, sw, offsets, G, M, d, f, out, di.sms, stream);
}

}  // namespace

// ---- block norms ----
namespace {

// Launch shape for T rows of d columns, row_bytes of input each: vectors per thread, threads, CTAs and stages of the row ring
// (0: no ring). Up to two rows per SM: a row per CTA by plain loads, one vector per thread where that fits, for the shortest path
// through a row. More: rings that fill about 200 KB of shared memory per SM between `per_sm` CTAs, or as many more (up to `most`) as
// 512 threads make, so that narrow rows too have some 16 warps' work under way (behind the block, 8192 rows of 1024 in bf16: two CTAs of
// 128 threads per SM 34 us, four 22 us).
struct NormShape {
    int vpt, threads, grid, stages;
    size_t smem;
};
constexpr size_t kNormRingBytes = 204 * 1024;
// the widest row, of the gradient in front with an fp32 stream and dres, has a stage
static_assert(BN_MAX_D * (2 + 4 + 4) <= kNormRingBytes - 256, "stages");
NormShape norm_shape(int T, int d, int sms, size_t row_bytes, int vpt1_max, int per_sm, int most) {
    const int nvec = d / 8;
    NormShape s{};
    const bool ring = T > 2 * sms;
    s.vpt = nvec <= vpt1_max ? 1 : (nvec <= 2 * BN_MAX_THREADS ? 2 : 4);
    if (!ring && nvec <= BN_MAX_THREADS) s.vpt = 1;
    s.threads = (nvec + s.vpt * 32 - 1) / (s.vpt * 32) * 32;
    if (!ring) {
        s.grid = T;
        return s;
    }
    int m = std::max(per_sm, std::min(BN_MAX_THREADS / s.threads, most));
    while (m > 1 && (m * s.threads > 1536 || 2 * row_bytes > kNormRingBytes / m)) --m;
    s.grid = m * sms < T ? m * sms : T;
    s.stages = (int)std::min<size_t>(BN_MAX_STAGES, (kNormRingBytes / m - 256) / row_bytes);
    s.smem = 128 + (size_t)s.stages * row_bytes;
    return s;
}

// Limits of the kernels' dynamic shared memory: the most that any ring takes, whatever the call, so that no call depends on another and no
// thread lowers what another is about to use. (Without it the limit of 48 KB holds for static and dynamic memory together.)
template <typename... Kernels>
cudaError_t norm_ring_limit(Kernels... kernels) {
    cudaError_t e = cudaSuccess;
    ((e = e == cudaSuccess ? cudaFuncSetAttribute(kernels, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kNormRingBytes) : e), ...);
    return e;
}
template <typename R, int VPT>
cudaError_t norm_ring_limits() {
    return norm_ring_limit(block_norm_in_kernel<R, VPT, true>, block_norm_out_kernel<R, VPT, false, true>,
                           block_norm_out_kernel<R, VPT, true, true>, block_norm_in_grad_kernel<R, VPT, true>);
}
template <typename R, bool NEXT, bool GATE>
cudaError_t norm_grad_ring_limits() {
    return norm_ring_limit(block_norm_out_grad_kernel<R, NEXT, GATE, true, false>, block_norm_out_grad_kernel<R, NEXT, GATE, true, true>);
}
template <typename R>
cudaError_t norm_ring_limits() {
    cudaError_t e = norm_ring_limits<R, 1>();
    if (e == cudaSuccess) e = norm_ring_limits<R, 2>();
    if (e == cudaSuccess) e = norm_ring_limits<R, 4>();
    if (e == cudaSuccess) e = norm_grad_ring_limits<R, false, false>();
    if (e == cudaSuccess) e = norm_grad_ring_limits<R, false, true>();
    if (e == cudaSuccess) e = norm_grad_ring_limits<R, true, false>();
    if (e == cudaSuccess) e = norm_grad_ring_limits<R, true, true>();
    return e;
}

// The device, with those limits set once.
moe_status_t norm_device(DeviceInfo& di) {
    moe_status_t st = device_info(di);
    if (st != MOE_OK) return st;
    static bool ready[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    std::lock_guard<std::mutex> lock(g_mu);
    if (e == cudaSuccess && !ready[dev]) {
        e = norm_ring_limits<float>();
        if (e == cudaSuccess) e = norm_ring_limits<__nv_bfloat16>();
        ready[dev] = e == cudaSuccess;
    }
    if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    return MOE_OK;
}

moe_status_t check_norm_sizes(int T, int d, moe_stream_type_t type) {
    if (T < 0) return fail(MOE_ERR_INVALID_ARG, "T=%d < 0", T);
    if (d < 8 || d % 8 || d > BN_MAX_D)
        return fail(MOE_ERR_INVALID_ARG, "d=%d must be a positive multiple of 8, at most %d", d, BN_MAX_D);
    if (type != MOE_STREAM_BF16 && type != MOE_STREAM_FP32)
        return fail(MOE_ERR_INVALID_ARG, "unknown residual type %d", (int)type);
    return MOE_OK;
}

moe_status_t check_norm_eps(float eps) {
    if (!(eps >= 0.f) || eps > 1e30f) return fail(MOE_ERR_INVALID_ARG, "eps=%g must be finite and not negative", (double)eps);
    return MOE_OK;
}

// (without tokens the gate has no rows, and its pointer may be null)
moe_status_t check_norm_gate(const void* gate, int gate_rows, int T) {
    if (gate_rows < 0 || (T > 0 && (gate != nullptr) != (gate_rows > 0)))
        return fail(MOE_ERR_INVALID_ARG, "gate_rows=%d: at least 1 with a gate, 0 without", gate_rows);
    return MOE_OK;
}

// (four CTAs per SM for rows that 128 threads hold, else two)
int norm_grad_ctas(int T, int d) { return std::min(T, d <= 1024 ? BN_GRAD_CTAS : BN_GRAD_CTAS / 2); }

#define MOE_NORM_CASES(s, CALL)                              \
    if (s.stages) {                                          \
        switch (s.vpt) {                                     \
            case 1: CALL(1, true); break;                    \
            case 2: CALL(2, true); break;                    \
            default: CALL(4, true); break;                   \
        }                                                    \
    } else {                                                 \
        switch (s.vpt) {                                     \
            case 1: CALL(1, false); break;                   \
            case 2: CALL(2, false); break;                   \
            default: CALL(4, false); break;                  \
        }                                                    \
    }

template <typename R>
cudaError_t launch_norm_in(const void* x, const float* w, int T, int d, float eps, void* xn, float* rstd, int sms,
                           cudaStream_t stream) {
    const NormShape s = norm_shape(T, d, sms, (size_t)d * sizeof(R), 128, 4, 8);
    cudaError_t e = cudaSuccess;
#define CALL(V, RING)                                                                                                      \
    e = launch_pdl(block_norm_in_kernel<R, V, RING>, dim3(s.grid), dim3(s.threads), s.smem, stream,                        \
                   reinterpret_cast<const R*>(x), w, T, d, eps, reinterpret_cast<__nv_bfloat16*>(xn), rstd, s.stages)
    MOE_NORM_CASES(s, CALL)
#undef CALL
    return e;
}

template <typename R, bool NEXT>
cudaError_t launch_norm_out(const NormOutArgs& a, int sms, cudaStream_t stream) {
    const NormShape s = norm_shape(a.T, a.d, sms, (size_t)a.d * (2 + sizeof(R) + (a.gate ? 2 : 0)), 128, 2, 8);
    cudaError_t e = cudaSuccess;
#define CALL(V, RING)                                                                                                \
    e = launch_pdl(block_norm_out_kernel<R, V, NEXT, RING>, dim3(s.grid), dim3(s.threads), s.smem, stream, a, s.stages)
    MOE_NORM_CASES(s, CALL)
#undef CALL
    return e;
}

// The backward kernels' grids: at most norm_grad_ctas(T, d), the partial rows of the workspace.
NormShape norm_grad_shape(int T, int d, int sms, size_t row_bytes, int per_sm) {
    NormShape s = norm_shape(T, d, sms, row_bytes, BN_MAX_THREADS, per_sm, 4);
    s.grid = std::min(s.grid, norm_grad_ctas(T, d));
    return s;
}

template <typename R>
cudaError_t launch_norm_in_grad(const NormInGradArgs& a, int sms, cudaStream_t stream, int& B) {
    const NormShape s = norm_grad_shape(a.T, a.d, sms, (size_t)a.d * (2 + sizeof(R) * (a.dres ? 2 : 1)), 2);
    B = s.grid;
    cudaError_t e = cudaSuccess;
#define CALL(V, RING)                                                                                                    \
    e = launch_pdl(block_norm_in_grad_kernel<R, V, RING>, dim3(s.grid), dim3(s.threads), s.smem, stream, a, s.stages)
    MOE_NORM_CASES(s, CALL)
#undef CALL
    return e;
}

// n: clusters of `ctas` CTAs of `threads` threads and `smem` bytes that are resident at once (asked once per device and cluster size,
// of whichever kernel comes first: shared memory is what limits them all).
template <typename... KArgs>
cudaError_t resident_clusters(void (*kernel)(KArgs...), int ctas, int threads, size_t smem, int& n) {
    static int known[kMaxDevices][BN_MAX_CLUSTER + 1] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(g_mu);
    if (known[dev][ctas] == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(ctas);
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = ctas, attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
        if (e != cudaSuccess) return e;
        known[dev][ctas] = std::max(n, 1);
    }
    n = known[dev][ctas];
    return cudaSuccess;
}

constexpr int kNormPairThreads = BN_MAX_THREADS / 2;  // CTAs of so many threads run two to an SM (their registers allow no more)
constexpr size_t kNormPairBytes = kNormRingBytes / 2 - 1024;
// a cluster's CTAs have rows in three stages at a time: fp32 stream, next norm and gate are 14 bytes per column
static_assert(kNormPairBytes / (kNormPairThreads * 8 * 14) >= 3, "stages");

// Columns are cut over a cluster so that a thread has one vector of 8.
template <typename R, bool NEXT, bool GATE, bool CLUSTER>
cudaError_t launch_norm_out_grad(const NormOutGradArgs& a, int ctas, int sms, cudaStream_t stream, int& B) {
    const auto ring = block_norm_out_grad_kernel<R, NEXT, GATE, true, CLUSTER>;
    const auto plain = block_norm_out_grad_kernel<R, NEXT, GATE, false, CLUSTER>;
    const int per_cta = (a.d / 8 + ctas - 1) / ctas;
    const size_t row_bytes = (size_t)per_cta * 8 * ((NEXT ? 2 : 1) * (2 + sizeof(R)) + (GATE ? 2 : 0));
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3((per_cta + 31) / 32 * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // as launch_pdl
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas, attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CLUSTER ? 2 : 1;
    // Two CTAs per SM where 256 threads hold a row (8192 rows of 2048 in bf16 50 us, with one 71 us), four where 128 do.
    const int per_sm = std::max(1, std::min(BN_MAX_THREADS / (int)cfg.blockDim.x, 4));
    int stages = 0;
    B = a.T;
    if ((long)a.T * ctas > 2L * sms) {
        stages = (int)std::min<size_t>(BN_MAX_STAGES, (kNormRingBytes / per_sm - 1024) / row_bytes);
        cfg.dynamicSmemBytes = 128 + (size_t)stages * row_bytes;
        int resident = sms * per_sm;
        if (CLUSTER) {
            const cudaError_t e = resident_clusters(ring, ctas, kNormPairThreads, kNormPairBytes, resident);
            if (e != cudaSuccess) return e;
        }
        B = std::min(resident, a.T);
    }
    B = std::min(B, norm_grad_ctas(a.T, a.d));
    cfg.gridDim = dim3(B * ctas);
    return cudaLaunchKernelEx(&cfg, stages ? ring : plain, a, stages);
}

template <typename R, bool NEXT, bool GATE>
cudaError_t launch_norm_out_grad(const NormOutGradArgs& a, int sms, cudaStream_t stream, int& B) {
    // Up to 4096 columns one CTA (8192 rows of 4096 in bf16 89 us; two of 256 threads each, 120 to 150 us), above that CTAs of up to 256
    // threads, two to an SM (6000 rows of 5120 in bf16 139 us, two CTAs of 320 threads 151 us).
    const int ctas = a.d / 8 <= BN_MAX_THREADS ? 1 : (a.d / 8 + kNormPairThreads - 1) / kNormPairThreads;
    return ctas > 1 ? launch_norm_out_grad<R, NEXT, GATE, true>(a, ctas, sms, stream, B)
                    : launch_norm_out_grad<R, NEXT, GATE, false>(a, ctas, sms, stream, B);
}

template <typename R>
cudaError_t launch_norm_out_grad(const NormOutGradArgs& a, int sms, cudaStream_t stream, int& B) {
    if (a.dxn)
        return a.gate ? launch_norm_out_grad<R, true, true>(a, sms, stream, B) : launch_norm_out_grad<R, true, false>(a, sms, stream, B);
    return a.gate ? launch_norm_out_grad<R, false, true>(a, sms, stream, B) : launch_norm_out_grad<R, false, false>(a, sms, stream, B);
}

cudaError_t launch_norm_reduce(NormReduceArgs& a, cudaStream_t stream) {
    a.sums = a.part_next ? 2 : 1;
    int edges = 0;
    if (a.part_gate) {
        // row: norm_first_row(T, B, b + 1), the first row behind CTA b, in steps (its divisions took microseconds of the call)
        const uint32_t step = a.T / a.B, rest = a.T % a.B, rows = a.gate_rows;
        uint32_t row = 0, over = 0, seen = ~0u;  // seen: gate row of the last edge
        for (int b = 0; b + 1 < a.B; ++b) {
            row += step;
            if ((over += rest) >= (uint32_t)a.B) over -= a.B, ++row;
            const uint32_t group = row / rows;
            if (row == group * rows) continue;
            if (group != seen) a.edge[edges++] = (int16_t)b;
            seen = group;
        }
    }
    return launch_pdl(block_norm_reduce_kernel, dim3((a.d + 31) / 32, a.sums + edges), dim3(BNR_WARPS * 32), 0, stream, a);
}

// Workspace of a backward pass: part_w [B][d] | part_next [B][d] | part_gate [B][2][d] (with a gate)
size_t norm_grad_ws(int T, int d, int gate_rows) { return (size_t)norm_grad_ctas(T, d) * d * 4 * (gate_rows > 0 ? 4 : 2); }

}  // namespace

extern "C" {

// ---- the whole layer for few tokens ----

size_t moe_few_tokens_workspace_size(int T, int d, int f, int fs, int E, int k) {
    if (T < 1 || T > MOE_FEW_TOKENS_MAX || d < 8 || f < 8 || fs < 0 || E < 1 || k < 1 || k > 32) return 0;
    return (few_workspace(T, d, f, fs, k).bytes + 255) / 256 * 256;
}

moe_status_t moe_few_tokens(const moe_bf16_t* x, const float* w_router, const float* bias, const moe_bf16_t* w_gateup,
                            const moe_bf16_t* w_down, const moe_bf16_t* w_gateup_shared, const moe_bf16_t* w_down_shared, int T,
                            int d, int f, int fs, int E, int k, moe_route_mode_t mode, float* logits_out, int32_t* topk_idx,
                            float* topk_w, moe_bf16_t* y, void* ws, size_t ws_bytes, cudaStream_t stream) {
    moe_status_t st = check_route_sizes(T, E, k);
    if (st != MOE_OK) return st;
    if (mode < MOE_ROUTE_TOPK_SOFTMAX || mode > MOE_ROUTE_SIGMOID_TOPK_NORM)
        return fail(MOE_ERR_INVALID_ARG, "unknown routing mode %d", (int)mode);
    if (T > MOE_FEW_TOKENS_MAX) return fail(MOE_ERR_INVALID_ARG, "T=%d above %d", T, MOE_FEW_TOKENS_MAX);
    if (d < 8 || f < 8 || d % 8 || f % 8 || fs < 0 || fs % 8)
        return fail(MOE_ERR_INVALID_ARG, "d=%d and f=%d must be positive multiples of 8, fs=%d 0 or one", d, f, fs);
    if ((long)d * f > 0x7fffffffL || (long)d * fs > 0x3fffffffL) return fail(MOE_ERR_INVALID_ARG, "d * f too large");
    if (T == 0) return MOE_OK;
    if (!x || !w_router || !w_gateup || !w_down || !logits_out || !topk_idx || !topk_w || !y ||
        (fs > 0 && (!w_gateup_shared || !w_down_shared)))
        return fail(MOE_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(x) || !aligned16(w_router) || !aligned16(w_gateup) || !aligned16(w_down) || !aligned16(w_gateup_shared) ||
        !aligned16(w_down_shared) || !aligned16(y))
        return fail(MOE_ERR_INVALID_ARG, "x, y and weight pointers must be 16-byte aligned");
    if (!aligned4(bias, logits_out, topk_idx, topk_w))
        return fail(MOE_ERR_INVALID_ARG, "bias, logits_out, topk_idx and topk_w must be 4-byte aligned");
    const FewWorkspace w = few_workspace(T, d, f, fs, k);
    if (!ws || ws_bytes < w.bytes)
        return fail(MOE_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", w.bytes, ws ? ws_bytes : (size_t)0);
    if (reinterpret_cast<uintptr_t>(ws) & 255u) return fail(MOE_ERR_WORKSPACE, "workspace not 256-byte aligned");
    DeviceInfo di;
    if ((st = operator_device(di)) != MOE_OK) return st;
    uint8_t* base = reinterpret_cast<uint8_t*>(ws);
    FewArgs a{};
    a.x = reinterpret_cast<const __nv_bfloat16*>(x);
    a.w_gateup = reinterpret_cast<const __nv_bfloat16*>(w_gateup);
    a.w_down = reinterpret_cast<const __nv_bfloat16*>(w_down);
    a.s_gateup = reinterpret_cast<const __nv_bfloat16*>(w_gateup_shared);
    a.s_down = reinterpret_cast<const __nv_bfloat16*>(w_down_shared);
    a.logits = logits_out, a.topk_idx = topk_idx, a.topk_w = topk_w;
    a.y = reinterpret_cast<__nv_bfloat16*>(y);
    a.counters = reinterpret_cast<int*>(base);
    a.h = reinterpret_cast<__nv_bfloat16*>(base + w.h);
    a.part = reinterpret_cast<float*>(base + w.part);
    a.T = T, a.d = d, a.f = f, a.fs = fs, a.E = E, a.k = k, a.mode = (int)mode, a.ldh = w.ldh;
    cudaError_t e = launch_pdl(few_tokens_logits_kernel, dim3(E), dim3(FT_LOGIT_THREADS), 0, stream, a.x, w_router, bias, T, d, E,
                               logits_out, a.counters, w.n_counters);
    if ((st = check_launch("few_tokens (logits)", e)) != MOE_OK) return st;
    // at least one step of the down projection per CTA (some expert is always active)
    const long steps = (long)((f + FT_KC - 1) / FT_KC) * ((d + 31) / 32);
    const int grid = (int)std::min<long>(steps, std::min(di.sms, FT_MAX_CTAS));
    // the smallest number of 8-token blocks; three of them only where the tables (many choices, many experts) fit beside its ring
    if (T <= 8)
        e = launch_few<1>(a, grid, stream);
    else if (T <= 16)
        e = launch_few<2>(a, grid, stream);
    else if (T <= 24 && few_smem<3>(T * k, E) <= kFewMaxSmem)
        e = launch_few<3>(a, grid, stream);
    else
        e = launch_few<4>(a, grid, stream);
    return check_launch("few_tokens", e);
}

// ---- e4m3 operands with a scale per block of 128 ----

moe_status_t moe_fp8_block_quantize(const moe_bf16_t* w, int G, int N, int K, uint8_t* q, float* s, cudaStream_t stream) {
    if (G < 0 || N < 0) return fail(MOE_ERR_INVALID_ARG, "G=%d or N=%d < 0", G, N);
    if (K < 16 || K % 16) return fail(MOE_ERR_INVALID_ARG, "K=%d must be a positive multiple of 16", K);
    if (G == 0 || N == 0) return MOE_OK;
    if (!w || !q || !s) return fail(MOE_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(w) || !aligned16(q) || !aligned4(s))
        return fail(MOE_ERR_INVALID_ARG, "w and q must be 16-byte, s 4-byte aligned");
    DeviceInfo di;
    moe_status_t st = operator_device(di);
    if (st != MOE_OK) return st;
    const long blocks = (long)G * ((N + F8_BLOCK - 1) / F8_BLOCK) * ((K + F8_BLOCK - 1) / F8_BLOCK);
    // Both encoders are launched plainly: between two expert products they are elementwise kernels behind a GEMM and in front of a
    // CTA-pair GEMM, the place in which one that was launched early stalled the stream (launch_plain).
    return check_launch("fp8_block_quantize",
                        launch_plain(fp8_block_quantize_kernel, dim3(grid_cap(blocks, di.sms, 6)), dim3(256), 0, stream,
                                     reinterpret_cast<const __nv_bfloat16*>(w), N, K, blocks, q, s));
}

moe_status_t moe_fp8_row_quantize(const moe_bf16_t* x, const int32_t* row_src, int T, int K, int R, uint8_t* q, float* s,
                                  cudaStream_t stream) {
    if (T < 0 || R < 0) return fail(MOE_ERR_INVALID_ARG, "T=%d or R=%d < 0", T, R);
    if (K < 16 || K % 16) return fail(MOE_ERR_INVALID_ARG, "K=%d must be a positive multiple of 16", K);
    if (!row_src && R > T) return fail(MOE_ERR_INVALID_ARG, "R=%d rows of T=%d without row_src", R, T);
    if (R == 0) return MOE_OK;
    if (T == 0 || !x || !q || !s) return fail(MOE_ERR_INVALID_ARG, "no source rows, or null pointer");
    if (!aligned16(x) || !aligned16(q) || !aligned4(row_src, s))
        return fail(MOE_ERR_INVALID_ARG, "x and q must be 16-byte, row_src and s 4-byte aligned");
    DeviceInfo di;
    moe_status_t st = operator_device(di);
    if (st != MOE_OK) return st;
    const int chunks = (K / 8 + F8_CHUNK_VEC - 1) / F8_CHUNK_VEC;
    if (chunks > 65535) return fail(MOE_ERR_INVALID_ARG, "K=%d too large", K);
    const int grid = grid_cap(((long)R + 7) / 8, std::max(1, di.sms / chunks), 6);
    // (plainly: see moe_fp8_block_quantize)
    return check_launch("fp8_row_quantize",
                        launch_plain(fp8_row_quantize_kernel, dim3(grid, chunks), dim3(256), 0, stream,
                                     reinterpret_cast<const __nv_bfloat16*>(x), row_src, T, K, R, q, s));
}

moe_status_t moe_grouped_gemm_gateup_fp8(const uint8_t* aq, const float* as, const uint8_t* wq_gateup, const float* ws_gateup,
                                         const int32_t* group_offsets, int G, int M, int d, int f, moe_bf16_t* h,
                                         cudaStream_t stream) {
    return gemm_fp8<true>(aq, as, wq_gateup, ws_gateup, group_offsets, G, M, d, f, h, stream);
}

moe_status_t moe_grouped_gemm_down_fp8(const uint8_t* hq, const float* hs, const uint8_t* wq_down, const float* ws_down,
                                       const int32_t* group_offsets, int G, int M, int d, int f, moe_bf16_t* y,
                                       cudaStream_t stream) {
    return gemm_fp8<false>(hq, hs, wq_down, ws_down, group_offsets, G, M, d, f, y, stream);
}

// ---- block norms ----

moe_status_t moe_block_norm_in(const void* x, moe_stream_type_t type, const float* w, int T, int d, float eps,
                               moe_bf16_t* xn, float* rstd, cudaStream_t stream) {
    moe_status_t st = check_norm_sizes(T, d, type);
    if (st == MOE_OK) st = check_norm_eps(eps);
    if (st != MOE_OK) return st;
    if (!w || (T > 0 && (!x || !xn || !rstd))) return fail(MOE_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(x) || !aligned16(w) || !aligned16(xn)) return fail(MOE_ERR_INVALID_ARG, "x, w and xn must be 16-byte aligned");
    if (!aligned4(rstd)) return fail(MOE_ERR_INVALID_ARG, "rstd must be 4-byte aligned");
    DeviceInfo di;
    if ((st = norm_device(di)) != MOE_OK) return st;
    if (T == 0) return MOE_OK;
    return check_launch("block_norm_in", type == MOE_STREAM_FP32 ? launch_norm_in<float>(x, w, T, d, eps, xn, rstd, di.sms, stream)
                                                                 : launch_norm_in<__nv_bfloat16>(x, w, T, d, eps, xn, rstd, di.sms,
                                                                                                 stream));
}

moe_status_t moe_block_norm_out(const moe_bf16_t* y, const void* r, moe_stream_type_t type, const float* w,
                                const moe_bf16_t* gate, int gate_rows, float alpha, const float* w_next, int T, int d,
                                float eps, void* out, float* rstd, moe_bf16_t* xn, float* rstd_next, cudaStream_t stream) {
    moe_status_t st = check_norm_sizes(T, d, type);
    if (st == MOE_OK) st = check_norm_eps(eps);
    if (st == MOE_OK) st = check_norm_gate(gate, gate_rows, T);
    if (st != MOE_OK) return st;
    if (!w || (T > 0 && (!y || !r || !out || !rstd || (w_next && (!xn || !rstd_next)))))
        return fail(MOE_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(y) || !aligned16(r) || !aligned16(w) || !aligned16(gate) || !aligned16(w_next) || !aligned16(out) ||
        !aligned16(xn))
        return fail(MOE_ERR_INVALID_ARG, "y, r, w, gate, w_next, out and xn must be 16-byte aligned");
    if (!aligned4(rstd, rstd_next)) return fail(MOE_ERR_INVALID_ARG, "rstd and rstd_next must be 4-byte aligned");
    DeviceInfo di;
    if ((st = norm_device(di)) != MOE_OK) return st;
    if (T == 0) return MOE_OK;
    const NormOutArgs a{reinterpret_cast<const __nv_bfloat16*>(y), r, w, reinterpret_cast<const __nv_bfloat16*>(gate), w_next, out,
                        rstd, reinterpret_cast<__nv_bfloat16*>(xn), rstd_next, T, d, gate_rows, alpha, eps};
    const bool f32 = type == MOE_STREAM_FP32;
    cudaError_t e;
    if (w_next)
        e = f32 ? launch_norm_out<float, true>(a, di.sms, stream) : launch_norm_out<__nv_bfloat16, true>(a, di.sms, stream);
    else
        e = f32 ? launch_norm_out<float, false>(a, di.sms, stream) : launch_norm_out<__nv_bfloat16, false>(a, di.sms, stream);
    return check_launch("block_norm_out", e);
}

size_t moe_block_norm_backward_workspace_size(int T, int d, int gate_rows) {
    if (T <= 0 || d <= 0) return 0;
    return round256(norm_grad_ws(T, d, gate_rows));
}

moe_status_t moe_block_norm_in_backward(const moe_bf16_t* dxn, const void* dres, const void* x, moe_stream_type_t type,
                                        const float* w, const float* rstd, int T, int d, void* dx, float* dw, void* ws,
                                        size_t ws_bytes, cudaStream_t stream) {
    moe_status_t st = check_norm_sizes(T, d, type);
    if (st != MOE_OK) return st;
    if (!w || !dw || (T > 0 && (!dxn || !x || !rstd || !dx))) return fail(MOE_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(dxn) || !aligned16(dres) || !aligned16(x) || !aligned16(w) || !aligned16(dx))
        return fail(MOE_ERR_INVALID_ARG, "dxn, dres, x, w and dx must be 16-byte aligned");
    if (!aligned4(rstd, dw)) return fail(MOE_ERR_INVALID_ARG, "rstd and dw must be 4-byte aligned");
    const size_t need = T > 0 ? norm_grad_ws(T, d, 0) : 0;
    if (need && (!ws || ws_bytes < need))
        return fail(MOE_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, ws ? ws_bytes : (size_t)0);
    if (need && !aligned16(ws)) return fail(MOE_ERR_WORKSPACE, "workspace not 16-byte aligned");
    DeviceInfo di;
    if ((st = norm_device(di)) != MOE_OK) return st;
    if (T == 0) {  // no tokens: the gain's gradient is zero
        const cudaError_t e = cudaMemsetAsync(dw, 0, sizeof(float) * (size_t)d, stream);
        return e == cudaSuccess ? MOE_OK : fail(MOE_ERR_CUDA, "cudaMemsetAsync: %s", cudaGetErrorString(e));
    }
    const NormInGradArgs a{reinterpret_cast<const __nv_bfloat16*>(dxn), dres, x, w, rstd, dx, reinterpret_cast<float*>(ws), T, d};
    int B = 0;
    cudaError_t e = type == MOE_STREAM_FP32 ? launch_norm_in_grad<float>(a, di.sms, stream, B)
                                            : launch_norm_in_grad<__nv_bfloat16>(a, di.sms, stream, B);
    if ((st = check_launch("block_norm_in_backward", e)) != MOE_OK) return st;
    NormReduceArgs ra{};
    ra.part_w = a.part_w;
    ra.dw = dw;
    ra.T = T, ra.d = d, ra.B = B;
    return check_launch("block_norm_in_backward (sums)", launch_norm_reduce(ra, stream));
}

moe_status_t moe_block_norm_out_backward(const void* dout, const moe_bf16_t* dxn, const moe_bf16_t* y, const void* out,
                                         moe_stream_type_t type, const float* w, const moe_bf16_t* gate, int gate_rows,
                                         float alpha, const float* w_next, const float* rstd, const float* rstd_next, int T,
                                         int d, void* dr, moe_bf16_t* dy, float* dw, float* dgate, float* dw_next, void* ws,
                                         size_t ws_bytes, cudaStream_t stream) {
    moe_status_t st = check_norm_sizes(T, d, type);
    if (st == MOE_OK) st = check_norm_gate(gate, gate_rows, T);
    if (st != MOE_OK) return st;
    if (!w || !dw || (T > 0 && (!dout || !y || !rstd || !dr || !dy))) return fail(MOE_ERR_INVALID_ARG, "null pointer");
    if ((w_next != nullptr) != (dw_next != nullptr) || (!w_next && dxn) || (T > 0 && w_next && (!dxn || !out || !rstd_next)))
        return fail(MOE_ERR_INVALID_ARG, "the next norm takes w_next, dxn, out, rstd_next and dw_next together");
    if (T > 0 && gate && !dgate) return fail(MOE_ERR_INVALID_ARG, "a gate needs dgate");
    if (!aligned16(dout) || !aligned16(dxn) || !aligned16(y) || !aligned16(out) || !aligned16(w) || !aligned16(gate) ||
        !aligned16(w_next) || !aligned16(dr) || !aligned16(dy) || !aligned16(dgate))
        return fail(MOE_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
    if (!aligned4(rstd, rstd_next, dw, dw_next))
        return fail(MOE_ERR_INVALID_ARG, "rstd, rstd_next, dw and dw_next must be 4-byte aligned");
    const size_t need = T > 0 ? norm_grad_ws(T, d, gate_rows) : 0;
    if (need && (!ws || ws_bytes < need))
        return fail(MOE_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, ws ? ws_bytes : (size_t)0);
    if (need && !aligned16(ws)) return fail(MOE_ERR_WORKSPACE, "workspace not 16-byte aligned");
    DeviceInfo di;
    if ((st = norm_device(di)) != MOE_OK) return st;
    if (T == 0) {  // no tokens: the gains' gradients are zero
        cudaError_t e = cudaMemsetAsync(dw, 0, sizeof(float) * (size_t)d, stream);
        if (e == cudaSuccess && dw_next) e = cudaMemsetAsync(dw_next, 0, sizeof(float) * (size_t)d, stream);
        return e == cudaSuccess ? MOE_OK : fail(MOE_ERR_CUDA, "cudaMemsetAsync: %s", cudaGetErrorString(e));
    }
    int B = norm_grad_ctas(T, d);
    float* part = reinterpret_cast<float*>(ws);
    NormOutGradArgs a{};
    a.dout = dout, a.dxn = reinterpret_cast<const __nv_bfloat16*>(dxn), a.y = reinterpret_cast<const __nv_bfloat16*>(y);
    a.out = out, a.w = w, a.gate = reinterpret_cast<const __nv_bfloat16*>(gate), a.w_next = w_next;
    a.rstd = rstd, a.rstd_next = rstd_next, a.dr = dr, a.dy = reinterpret_cast<__nv_bfloat16*>(dy), a.dgate = dgate;
    a.part_w = part, a.part_next = part + (size_t)B * d, a.part_gate = part + (size_t)2 * B * d;
    a.T = T, a.d = d, a.gate_rows = gate_rows, a.alpha = alpha;
    cudaError_t e = type == MOE_STREAM_FP32 ? launch_norm_out_grad<float>(a, di.sms, stream, B)
                                            : launch_norm_out_grad<__nv_bfloat16>(a, di.sms, stream, B);
    if ((st = check_launch("block_norm_out_backward", e)) != MOE_OK) return st;
    NormReduceArgs ra{};
    ra.part_w = a.part_w, ra.part_next = dxn ? a.part_next : nullptr, ra.part_gate = gate ? a.part_gate : nullptr;
    ra.dw = dw, ra.dw_next = dw_next, ra.dgate = dgate;
    ra.T = T, ra.d = d, ra.gate_rows = gate_rows, ra.B = B;
    return check_launch("block_norm_out_backward (sums)", launch_norm_reduce(ra, stream));
}

}  // extern "C"
