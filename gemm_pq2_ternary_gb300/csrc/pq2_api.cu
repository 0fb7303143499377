// The C ABI (include/pq2.h): host-side argument checks, per-device set-up,
// routing to the kernels, and the device error word.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>
#include <mutex>

#include "../../include/pq2.h"
#include "pq2_internal.h"
#include "pq2_step.cuh"

// Device error word: bit flags of pq2::DEVERR_*, one per device context.
__device__ unsigned g_pq2_error_word = 0;

namespace {

constexpr int kMaxDevices = 64;
std::mutex g_mu;
pq2h::DeviceInfo g_dev[kMaxDevices];
bool g_dev_ok[kMaxDevices] = {};
std::atomic<unsigned long long> g_wait_limit_ns{2000000000ull};
std::atomic<int> g_debug_skip_stage{-1};
std::atomic<int> g_debug_bounds_shrink{0};
// pq2_debug_force_kernel: forced variant per op (GEMV, SMALL, PREFILL)
std::atomic<int> g_force[3] = {{0}, {0}, {0}};

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

pq2_status cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return PQ2_OK;
    if (e == pq2h::kUnsupportedVariant) {
        cudaGetLastError();  // (not sticky; clear it all the same)
        return PQ2_ERR_UNSUPPORTED_SHAPE;
    }
    return PQ2_ERR_CUDA;
}

// Common shape checks: K a positive multiple of 128 within the supported
// range, N >= 1.
pq2_status check_nk(int64_t N, int64_t K) {
    if (N < 1 || K < 1) return PQ2_ERR_INVALID_ARG;
    if (K % 128 != 0 || K > PQ2_MAX_K) return PQ2_ERR_UNSUPPORTED_SHAPE;
    if (N > (int64_t(1) << 31) - 1) return PQ2_ERR_UNSUPPORTED_SHAPE;
    return PQ2_OK;
}

struct Ctx {
    pq2h::DeviceInfo dev;
    pq2::DevCtl ctl;
};

pq2_status get_ctx(Ctx* c) {
    if (!pq2h::device_info(&c->dev)) return PQ2_ERR_CUDA;
    if (!pq2h::make_ctl(&c->ctl)) return PQ2_ERR_CUDA;
    return PQ2_OK;
}

size_t align256(size_t b) { return (b + 255) & ~size_t(255); }

}  // namespace

namespace pq2h {

int forced_variant(int op) {
    return (op >= PQ2_OP_GEMV && op <= PQ2_OP_PREFILL) ? g_force[op].load() : PQ2_VARIANT_DEFAULT;
}

bool device_info(DeviceInfo* out) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
    std::lock_guard<std::mutex> lock(g_mu);
    if (!g_dev_ok[dev]) {
        DeviceInfo d = {};
        d.device = dev;
        if (cudaDeviceGetAttribute(&d.num_sms, cudaDevAttrMultiProcessorCount, dev) !=
            cudaSuccess)
            return false;
        if (cudaDeviceGetAttribute(&d.max_smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin,
                                   dev) != cudaSuccess)
            return false;
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_pq2_error_word) != cudaSuccess) return false;
        d.err = static_cast<unsigned*>(p);
        g_dev[dev] = d;
        g_dev_ok[dev] = true;
    }
    *out = g_dev[dev];
    return true;
}

namespace {
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled_fn() {
    static EncodeTiledFn fn = [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                             cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return static_cast<EncodeTiledFn>(nullptr);
        return reinterpret_cast<EncodeTiledFn>(ptr);
    }();
    return fn;
}
}  // namespace

bool encode_tmap_2d(CUtensorMap* map, CUtensorMapDataType dt, const void* base, uint64_t inner,
                    uint64_t outer, uint64_t pitch_bytes, uint32_t box_inner, uint32_t box_outer,
                    bool swizzle128) {
    EncodeTiledFn fn = encode_tiled_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {inner, outer};
    const cuuint64_t strides[1] = {pitch_bytes};
    const cuuint32_t box[2] = {box_inner, box_outer};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, dt, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE,
              swizzle128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
              CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_ctl(pq2::DevCtl* ctl) {
    DeviceInfo d;
    if (!device_info(&d)) return false;
    ctl->err = d.err;
    ctl->wait_limit_ns = g_wait_limit_ns.load();
    ctl->debug_skip_stage = g_debug_skip_stage.load();
    ctl->debug_bounds_shrink = g_debug_bounds_shrink.load();
    return true;
}

}  // namespace pq2h

extern "C" {

const char* pq2_status_string(int status) {
    switch (status) {
        case PQ2_OK: return "ok";
        case PQ2_ERR_INVALID_ARG: return "invalid argument";
        case PQ2_ERR_UNSUPPORTED_SHAPE: return "unsupported shape";
        case PQ2_ERR_MISALIGNED: return "pointer not 16-byte aligned";
        case PQ2_ERR_CUDA: return "CUDA error";
        case PQ2_ERR_TIMEOUT: return "device wait timed out";
        case PQ2_ERR_WORKSPACE: return "workspace missing or too small";
        case PQ2_ERR_BOUNDS: return "bounds-checked build: a store outside its buffer";
        default: return "unknown status";
    }
}

const char* pq2_version(void) { return "pq2-gb300 0.1 sm_103a"; }

pq2_status pq2_debug_set_wait_limit_ns(uint64_t ns) {
    if (ns == 0) return PQ2_ERR_INVALID_ARG;
    g_wait_limit_ns.store(ns);
    return PQ2_OK;
}

// Not in the public header: makes every later launch's producer withhold
// stage `stage` (-1 = off), so the consumers' bounded wait runs out.  For the
// timeout test only.
pq2_status pq2_debug_skip_stage(int stage) {
    g_debug_skip_stage.store(stage < 0 ? -1 : stage);
    return PQ2_OK;
}

int pq2_bounds_checked(void) { return PQ2_DEBUG; }

pq2_status pq2_debug_shrink_bounds(int elements) {
    if (elements < 0) return PQ2_ERR_INVALID_ARG;
    g_debug_bounds_shrink.store(elements);
    return PQ2_OK;
}

pq2_status pq2_debug_force_kernel(int op, int variant) {
    int max_variant = -1;
    if (op == PQ2_OP_GEMV) max_variant = PQ2_VARIANT_GEMV_STAGED;
    if (op == PQ2_OP_SMALL) max_variant = PQ2_VARIANT_SMALL_WTILE;
    if (op == PQ2_OP_PREFILL) max_variant = PQ2_VARIANT_PREFILL_WTILE;
    if (variant < 0 || variant > max_variant) return PQ2_ERR_INVALID_ARG;
    g_force[op].store(variant);
    return PQ2_OK;
}

pq2_status pq2_debug_gemv_floor(int64_t N, int64_t K, uint32_t flags, void* stream) {
    if (flags & ~static_cast<uint32_t>(PQ2_WEIGHTS_STATIC)) return PQ2_ERR_INVALID_ARG;
    pq2_status s = check_nk(N, K);
    if (s != PQ2_OK) return s;
    if (!pq2h::gemv_fused_supported(K)) return PQ2_ERR_UNSUPPORTED_SHAPE;
    Ctx c;
    s = get_ctx(&c);
    if (s != PQ2_OK) return s;
    return cuda_status(pq2h::launch_gemv_floor(N, K, (flags & PQ2_WEIGHTS_STATIC) != 0,
                                               static_cast<cudaStream_t>(stream), c.ctl, c.dev));
}

pq2_status pq2_debug_mma_rate(int n, int iters, uint64_t* cycles, void* stream) {
    if ((n != 32 && n != 64 && n != 128 && n != 256) || iters < 1 || iters > (1 << 24))
        return PQ2_ERR_INVALID_ARG;
    if (!cycles) return PQ2_ERR_INVALID_ARG;
    Ctx c;
    pq2_status s = get_ctx(&c);
    if (s != PQ2_OK) return s;
    return cuda_status(pq2h::launch_mma_rate(n, iters,
                                             reinterpret_cast<unsigned long long*>(cycles),
                                             static_cast<cudaStream_t>(stream), c.ctl, c.dev));
}

pq2_status pq2_quantize_act(const void* x_f16, int64_t M, int64_t K, int8_t* qp, float* S,
                            int32_t* T, void* stream) {
    if (M < 0 || K < 1) return PQ2_ERR_INVALID_ARG;
    if (K % 128 != 0 || K > PQ2_MAX_K) return PQ2_ERR_UNSUPPORTED_SHAPE;
    if (M == 0) return PQ2_OK;
    if (!x_f16 || !qp || !S || !T) return PQ2_ERR_INVALID_ARG;
    if (!aligned16(x_f16) || !aligned16(qp) || !aligned16(S) || !aligned16(T))
        return PQ2_ERR_MISALIGNED;
    Ctx c;
    pq2_status s = get_ctx(&c);
    if (s != PQ2_OK) return s;
    return cuda_status(pq2h::launch_quantize(static_cast<const __half*>(x_f16), qp, S, T, M, K,
                                             static_cast<cudaStream_t>(stream), c.ctl, c.dev));
}

pq2_status pq2_quantize_swiglu(const float* gu, int64_t M, int64_t I, int8_t* qp, float* S,
                               int32_t* T, void* stream) {
    if (M < 0 || I < 1) return PQ2_ERR_INVALID_ARG;
    if (I % 128 != 0 || I > PQ2_MAX_K) return PQ2_ERR_UNSUPPORTED_SHAPE;
    if (M == 0) return PQ2_OK;
    if (!gu || !qp || !S || !T) return PQ2_ERR_INVALID_ARG;
    if (!aligned16(gu) || !aligned16(qp) || !aligned16(S) || !aligned16(T))
        return PQ2_ERR_MISALIGNED;
    Ctx c;
    pq2_status s = get_ctx(&c);
    if (s != PQ2_OK) return s;
    return cuda_status(pq2h::launch_quantize_swiglu(gu, qp, S, T, M, I,
                                                    static_cast<cudaStream_t>(stream), c.ctl,
                                                    c.dev));
}

pq2_status pq2_pack_weights(const int8_t* tern, const void* ws_f16, int64_t N, int64_t K,
                            uint8_t* codes, void* ws_out, void* stream) {
    pq2_status s = check_nk(N, K);
    if (s != PQ2_OK) return s;
    if (!tern || !codes) return PQ2_ERR_INVALID_ARG;
    if ((ws_f16 == nullptr) != (ws_out == nullptr)) return PQ2_ERR_INVALID_ARG;
    if (!aligned16(tern) || !aligned16(codes) || (ws_f16 && (!aligned16(ws_f16) ||
                                                            !aligned16(ws_out))))
        return PQ2_ERR_MISALIGNED;
    Ctx c;
    s = get_ctx(&c);
    if (s != PQ2_OK) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = pq2h::launch_pack(tern, codes, N, K, st, c.ctl, c.dev);
    if (e != cudaSuccess) return PQ2_ERR_CUDA;
    if (ws_f16 && ws_out != ws_f16) {
        e = cudaMemcpyAsync(ws_out, ws_f16, static_cast<size_t>(N) * (K / 128) * 2,
                            cudaMemcpyDeviceToDevice, st);
        if (e != cudaSuccess) return PQ2_ERR_CUDA;
    }
    return PQ2_OK;
}

static pq2_status check_mm(const int8_t* qp, const float* S, const int32_t* T,
                           const uint8_t* codes, const void* ws, const void* out, int64_t M,
                           int64_t N, int64_t K) {
    pq2_status s = check_nk(N, K);
    if (s != PQ2_OK) return s;
    if (M < 1) return PQ2_ERR_INVALID_ARG;
    if (!qp || !T || !codes || !out) return PQ2_ERR_INVALID_ARG;
    if (!aligned16(qp) || !aligned16(T) || !aligned16(codes) || !aligned16(out))
        return PQ2_ERR_MISALIGNED;
    if (S && !aligned16(S)) return PQ2_ERR_MISALIGNED;
    if (ws && !aligned16(ws)) return PQ2_ERR_MISALIGNED;
    return PQ2_OK;
}

pq2_status pq2_gemv(const int8_t* qp, const float* S, const int32_t* T, const uint8_t* codes,
                    const void* ws_f16, float* y, int64_t N, int64_t K, void* stream) {
    pq2_status s = check_mm(qp, S, T, codes, ws_f16, y, 1, N, K);
    if (s != PQ2_OK) return s;
    if (!S || !ws_f16) return PQ2_ERR_INVALID_ARG;
    Ctx c;
    s = get_ctx(&c);
    if (s != PQ2_OK) return s;
    return cuda_status(pq2h::launch_gemv(nullptr, qp, S, T, codes,
                                         static_cast<const __half*>(ws_f16), y, nullptr, N, K,
                                         static_cast<cudaStream_t>(stream), c.ctl, c.dev));
}

size_t pq2_workspace_bytes(int op, int64_t M, int64_t N, int64_t K) {
    if (check_nk(N, K) != PQ2_OK || M < 1) return SIZE_MAX;
    switch (op) {
        case PQ2_OP_GEMV: return M == 1 ? 0 : SIZE_MAX;
        case PQ2_OP_SMALL:
            return (M >= 2 && M <= 16) ? pq2h::small_tc_workspace_bytes(M, N, K) : SIZE_MAX;
        case PQ2_OP_PREFILL: return pq2h::prefill_workspace_bytes(M, N, K);
        case PQ2_OP_SWIGLU_DOWN:  // K is the intermediate size I
        case PQ2_OP_MATMUL: {
            if (op == PQ2_OP_MATMUL && M == 1 && pq2h::gemv_fused_supported(K))
                return 0;  // fused, no scratch
            const size_t G = static_cast<size_t>(K / 128);
            const size_t act = align256(static_cast<size_t>(M) * K) +
                               2 * align256(static_cast<size_t>(M) * G * 4);
            const int inner = M == 1 ? PQ2_OP_GEMV : (M <= 16 ? PQ2_OP_SMALL : PQ2_OP_PREFILL);
            const size_t k = pq2_workspace_bytes(inner, M, N, K);
            return k == SIZE_MAX ? SIZE_MAX : act + k;
        }
        default: return SIZE_MAX;
    }
}

// pq2_gemm_small; weights_static: PQ2_WEIGHTS_STATIC of pq2_matmul_ex
static pq2_status gemm_small(const int8_t* qp, const float* S, const int32_t* T, const uint8_t* codes,
                      const void* ws_f16, float* y, int64_t M, int64_t N, int64_t K,
                      void* workspace, size_t workspace_bytes, void* stream, bool weights_static) {
    pq2_status s = check_mm(qp, S, T, codes, ws_f16, y, M, N, K);
    if (s != PQ2_OK) return s;
    if (!S || !ws_f16) return PQ2_ERR_INVALID_ARG;
    if (M < 2 || M > 16) return PQ2_ERR_UNSUPPORTED_SHAPE;
    const size_t need = pq2_workspace_bytes(PQ2_OP_SMALL, M, N, K);
    if (need > 0 && (!workspace || workspace_bytes < need)) return PQ2_ERR_WORKSPACE;
    Ctx c;
    s = get_ctx(&c);
    if (s != PQ2_OK) return s;
    if (pq2h::gemv_multi_supported(M, N, K, c.dev.num_sms))
        return cuda_status(pq2h::launch_gemv_multi(qp, S, T, codes,
                                                   static_cast<const __half*>(ws_f16), y, nullptr,
                                                   M, N, K, static_cast<cudaStream_t>(stream),
                                                   c.dev, weights_static, c.ctl));
    return cuda_status(pq2h::launch_small_tc(qp, S, T, codes, static_cast<const __half*>(ws_f16), y,
                                          nullptr, M, N, K, workspace,
                                          static_cast<cudaStream_t>(stream), c.ctl, c.dev));
}

pq2_status pq2_gemm_small(const int8_t* qp, const float* S, const int32_t* T,
                          const uint8_t* codes, const void* ws_f16, float* y, int64_t M,
                          int64_t N, int64_t K, void* workspace, size_t workspace_bytes,
                          void* stream) {
    return gemm_small(qp, S, T, codes, ws_f16, y, M, N, K, workspace, workspace_bytes, stream,
                      false);
}

pq2_status pq2_gemm_small_ex(const int8_t* qp, const float* S, const int32_t* T,
                             const uint8_t* codes, const void* ws_f16, float* y, int64_t M,
                             int64_t N, int64_t K, uint32_t flags, void* workspace,
                             size_t workspace_bytes, void* stream) {
    if (flags & ~PQ2_WEIGHTS_STATIC) return PQ2_ERR_INVALID_ARG;
    return gemm_small(qp, S, T, codes, ws_f16, y, M, N, K, workspace, workspace_bytes, stream,
                      (flags & PQ2_WEIGHTS_STATIC) != 0);
}

pq2_status pq2_gemm_prefill(const int8_t* qp, const float* S, const int32_t* T,
                            const uint8_t* codes, const void* ws_f16, float* y, int64_t M,
                            int64_t N, int64_t K, void* workspace, size_t workspace_bytes,
                            void* stream) {
    pq2_status s = check_mm(qp, S, T, codes, ws_f16, y, M, N, K);
    if (s != PQ2_OK) return s;
    if (!S || !ws_f16) return PQ2_ERR_INVALID_ARG;
    if (M > (int64_t(1) << 31) - 1) return PQ2_ERR_UNSUPPORTED_SHAPE;
    const size_t need = pq2_workspace_bytes(PQ2_OP_PREFILL, M, N, K);
    if (need > 0 && (!workspace || workspace_bytes < need)) return PQ2_ERR_WORKSPACE;
    if (!aligned16(workspace)) return PQ2_ERR_MISALIGNED;
    Ctx c;
    s = get_ctx(&c);
    if (s != PQ2_OK) return s;
    return cuda_status(pq2h::launch_prefill(qp, S, T, codes, static_cast<const __half*>(ws_f16), y,
                                            nullptr, M, N, K, workspace,
                                            static_cast<cudaStream_t>(stream), c.ctl, c.dev));
}

pq2_status pq2_matmul(const void* x_f16, const uint8_t* codes, const void* ws_f16, float* y,
                      int64_t M, int64_t N, int64_t K, void* workspace, size_t workspace_bytes,
                      void* stream) {
    return pq2_matmul_ex(x_f16, codes, ws_f16, y, M, N, K, 0u, workspace, workspace_bytes, stream);
}

pq2_status pq2_matmul_ex(const void* x_f16, const uint8_t* codes, const void* ws_f16, float* y,
                         int64_t M, int64_t N, int64_t K, uint32_t flags, void* workspace,
                         size_t workspace_bytes, void* stream) {
    if (flags & ~PQ2_WEIGHTS_STATIC) return PQ2_ERR_INVALID_ARG;
    pq2_status s = check_nk(N, K);
    if (s != PQ2_OK) return s;
    if (M < 1 || !x_f16 || !codes || !ws_f16 || !y) return PQ2_ERR_INVALID_ARG;
    const size_t need = pq2_workspace_bytes(PQ2_OP_MATMUL, M, N, K);
    if (need == SIZE_MAX) return PQ2_ERR_UNSUPPORTED_SHAPE;
    if (M == 1 && pq2h::gemv_fused_supported(K)) {
        // fused: the GEMV kernel quantises x itself
        if (!aligned16(x_f16) || !aligned16(codes) || !aligned16(ws_f16) || !aligned16(y))
            return PQ2_ERR_MISALIGNED;
        Ctx c;
        s = get_ctx(&c);
        if (s != PQ2_OK) return s;
        return cuda_status(pq2h::launch_gemv(static_cast<const __half*>(x_f16), nullptr, nullptr,
                                             nullptr, codes, static_cast<const __half*>(ws_f16),
                                             y, nullptr, N, K, static_cast<cudaStream_t>(stream),
                                             c.ctl, c.dev, (flags & PQ2_WEIGHTS_STATIC) != 0));
    }
    if (!workspace || workspace_bytes < need) return PQ2_ERR_WORKSPACE;
    if (!aligned16(workspace)) return PQ2_ERR_MISALIGNED;
    const size_t G = static_cast<size_t>(K / 128);
    uint8_t* w = static_cast<uint8_t*>(workspace);
    int8_t* qp = reinterpret_cast<int8_t*>(w);
    w += align256(static_cast<size_t>(M) * K);
    float* S = reinterpret_cast<float*>(w);
    w += align256(static_cast<size_t>(M) * G * 4);
    int32_t* T = reinterpret_cast<int32_t*>(w);
    w += align256(static_cast<size_t>(M) * G * 4);
    const size_t rest = need - static_cast<size_t>(w - static_cast<uint8_t*>(workspace));
    if (M > 1 && M <= pq2h::kTileMaxM) {
        // the token-tile tensor-core kernels: their token tiles straight from
        // x (one launch fewer; y bit-identical to quantise + the matmul)
        Ctx c;
        s = get_ctx(&c);
        if (s != PQ2_OK) return s;
        using pq2h::TokenTile;
        const TokenTile tt =
            M <= 16 ? (pq2h::small_x_supported(M, N, K, c.dev.num_sms) ? TokenTile::kSmall
                                                                       : TokenTile::kNone)
                    : pq2h::prefill_token_tile_kernel(M, N, K, c.dev.num_sms);
        if (tt != TokenTile::kNone) {
            if (!aligned16(x_f16) || !aligned16(codes) || !aligned16(ws_f16) || !aligned16(y))
                return PQ2_ERR_MISALIGNED;
            const int op = M <= 16 ? PQ2_OP_SMALL : PQ2_OP_PREFILL;
            if (rest < pq2_workspace_bytes(op, M, N, K)) return PQ2_ERR_WORKSPACE;
            const __half* xh = static_cast<const __half*>(x_f16);
            const __half* wsh = static_cast<const __half*>(ws_f16);
            const cudaStream_t st = static_cast<cudaStream_t>(stream);
            if (tt == TokenTile::kSmall)
                return cuda_status(pq2h::launch_small_x(xh, codes, wsh, y, M, N, K, w, st, c.ctl,
                                                        c.dev));
            if (tt == TokenTile::kWide)
                return cuda_status(pq2h::launch_wtile_x(xh, codes, wsh, y, M, N, K, w, st, c.ctl,
                                                        c.dev));
            return cuda_status(pq2h::launch_tile_x(xh, codes, wsh, y, M, N, K, w, st, c.ctl, c.dev));
        }
    }
    s = pq2_quantize_act(x_f16, M, K, qp, S, T, stream);
    if (s != PQ2_OK) return s;
    if (M == 1) return pq2_gemv(qp, S, T, codes, ws_f16, y, N, K, stream);
    if (M <= 16)
        return gemm_small(qp, S, T, codes, ws_f16, y, M, N, K, rest ? w : nullptr, rest, stream,
                          (flags & PQ2_WEIGHTS_STATIC) != 0);
    return pq2_gemm_prefill(qp, S, T, codes, ws_f16, y, M, N, K, rest ? w : nullptr, rest,
                            stream);
}

pq2_status pq2_mlp_down_swiglu(const float* gu, const uint8_t* codes, const void* ws_f16, float* y,
                               int64_t M, int64_t N, int64_t I, void* workspace,
                               size_t workspace_bytes, void* stream) {
    pq2_status s = check_nk(N, I);
    if (s != PQ2_OK) return s;
    if (M < 1 || !gu || !codes || !ws_f16 || !y) return PQ2_ERR_INVALID_ARG;
    const size_t need = pq2_workspace_bytes(PQ2_OP_SWIGLU_DOWN, M, N, I);
    if (need == SIZE_MAX) return PQ2_ERR_UNSUPPORTED_SHAPE;
    if (!workspace || workspace_bytes < need) return PQ2_ERR_WORKSPACE;
    if (!aligned16(workspace)) return PQ2_ERR_MISALIGNED;
    const size_t G = static_cast<size_t>(I / 128);
    uint8_t* w = static_cast<uint8_t*>(workspace);
    int8_t* qp = reinterpret_cast<int8_t*>(w);
    w += align256(static_cast<size_t>(M) * I);
    float* S = reinterpret_cast<float*>(w);
    w += align256(static_cast<size_t>(M) * G * 4);
    int32_t* T = reinterpret_cast<int32_t*>(w);
    w += align256(static_cast<size_t>(M) * G * 4);
    const size_t rest = need - static_cast<size_t>(w - static_cast<uint8_t*>(workspace));
    s = pq2_quantize_swiglu(gu, M, I, qp, S, T, stream);
    if (s != PQ2_OK) return s;
    if (M == 1) return pq2_gemv(qp, S, T, codes, ws_f16, y, N, I, stream);
    if (M <= 16)
        return pq2_gemm_small(qp, S, T, codes, ws_f16, y, M, N, I, rest ? w : nullptr, rest,
                              stream);
    return pq2_gemm_prefill(qp, S, T, codes, ws_f16, y, M, N, I, rest ? w : nullptr, rest,
                            stream);
}

pq2_status pq2_gemm_bf16_splitk(const uint16_t* x, const uint16_t* w, uint16_t* y, int64_t M,
                                int64_t N, int64_t K, uint32_t flags, void* stream) {
    if (M < 0 || N < 0 || K < 0) return PQ2_ERR_INVALID_ARG;
    if (flags & ~static_cast<uint32_t>(PQ2_WEIGHTS_STATIC)) return PQ2_ERR_INVALID_ARG;
    if (K % 8 != 0 || K > PQ2_MAX_K || M > PQ2_MAX_M_BF16 || N > PQ2_MAX_N_BF16)
        return PQ2_ERR_UNSUPPORTED_SHAPE;
    if (M == 0 || N == 0) return PQ2_OK;
    if (!y || (K > 0 && (!x || !w))) return PQ2_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(w) || (reinterpret_cast<uintptr_t>(y) & 1u))
        return PQ2_ERR_MISALIGNED;
    Ctx c;
    pq2_status s = get_ctx(&c);
    if (s != PQ2_OK) return s;
    return cuda_status(pq2h::launch_bf16_splitk(x, w, y, M, N, K,
                                                (flags & PQ2_WEIGHTS_STATIC) != 0,
                                                static_cast<cudaStream_t>(stream), c.ctl));
}

static size_t type_bytes(int type) { return type == PQ2_F32 ? 4 : 2; }
static bool type_ok(int type) { return type == PQ2_F32 || type == PQ2_F16 || type == PQ2_BF16; }
static bool aligned_to(const void* p, size_t unit) {
    return reinterpret_cast<uintptr_t>(p) % unit == 0;
}

// The checks and the launch shared by the two norms (a.y null: the norm
// before a block alone).
static pq2_status norm(const pq2_norm_residual_args& a, int64_t M, int64_t H, void* stream) {
    const uint32_t flags = PQ2_WEIGHTS_STATIC | PQ2_NORM_UNIT_OFFSET | PQ2_NORM_NO_POST |
                           PQ2_GATE_SIGMOID | PQ2_GATE_SILU;
    const uint32_t both = PQ2_GATE_SIGMOID | PQ2_GATE_SILU;
    if (M < 0 || H < 1 || (a.flags & ~flags) || (a.flags & both) == both) return PQ2_ERR_INVALID_ARG;
    if (!(a.eps >= 0.0f)) return PQ2_ERR_INVALID_ARG;
    if (H > PQ2_NORM_MAX_H || M > (int64_t(1) << 31) - 1) return PQ2_ERR_UNSUPPORTED_SHAPE;
    if (!type_ok(a.r_type) || (a.x && !type_ok(a.x_type)) || (a.y && !type_ok(a.y_type)) ||
        (a.gate && !type_ok(a.gate_type)) || ((a.w_post || a.w_next) && !type_ok(a.w_type)))
        return PQ2_ERR_INVALID_ARG;
    if ((a.y && a.ld_y < H) || a.ld_r < H || (a.r_out && a.ld_r_out < H) || (a.x && a.ld_x < H) ||
        (a.gate && a.ld_gate != 0 && a.ld_gate < H))
        return PQ2_ERR_INVALID_ARG;
    if (M == 0) return PQ2_OK;
    if (!a.r) return PQ2_ERR_INVALID_ARG;
    if (!aligned_to(a.r, type_bytes(a.r_type)) || !aligned_to(a.r_out, type_bytes(a.r_type)) ||
        !aligned_to(a.y, type_bytes(a.y_type)) || !aligned_to(a.gate, type_bytes(a.gate_type)) ||
        !aligned_to(a.w_post, type_bytes(a.w_type)) || !aligned_to(a.w_next, type_bytes(a.w_type)) ||
        !aligned_to(a.x, type_bytes(a.x_type)))
        return PQ2_ERR_MISALIGNED;
    // in place only row on row: rows are taken in any order, and read ahead
    if (a.r_out == a.r && M > 1 && a.ld_r_out != a.ld_r) return PQ2_ERR_INVALID_ARG;
    if (!a.y && a.x == a.r && (a.x_type != a.r_type || (M > 1 && a.ld_x != a.ld_r)))
        return PQ2_ERR_INVALID_ARG;
    Ctx c;
    const pq2_status s = get_ctx(&c);
    if (s != PQ2_OK) return s;
    pq2h::NormParams p = {};
    p.y = a.y, p.r = a.r, p.r_out = a.r_out, p.w_post = a.w_post, p.gate = a.gate;
    p.w_next = a.w_next, p.x = a.x;
    p.ld_y = a.ld_y, p.ld_r = a.ld_r, p.ld_ro = a.ld_r_out, p.ld_gate = a.ld_gate, p.ld_x = a.ld_x;
    p.M = M;
    p.H = static_cast<int>(H);
    p.ro_elems = (M - 1) * a.ld_r_out + H;
    p.x_elems = (M - 1) * a.ld_x + H;
    p.y_type = a.y_type, p.r_type = a.r_type, p.w_type = a.w_type, p.gate_type = a.gate_type;
    p.x_type = a.x_type;
    p.eps = a.eps, p.alpha = a.alpha;
    p.w_offset = (a.flags & PQ2_NORM_UNIT_OFFSET) ? 1.0f : 0.0f;
    p.flags = a.flags;
    p.weights_static = (a.flags & PQ2_WEIGHTS_STATIC) ? 1 : 0;
    p.ctl = c.ctl;
    return cuda_status(pq2h::launch_norm(p, static_cast<cudaStream_t>(stream), c.dev));
}

pq2_status pq2_rmsnorm(const void* r, int r_type, int64_t ld_r, const void* w, int w_type, void* x,
                       int x_type, int64_t ld_x, int64_t M, int64_t H, float eps, uint32_t flags,
                       void* stream) {
    if (flags & ~(PQ2_WEIGHTS_STATIC | PQ2_NORM_UNIT_OFFSET)) return PQ2_ERR_INVALID_ARG;
    if (M > 0 && !x) return PQ2_ERR_INVALID_ARG;
    pq2_norm_residual_args a = {};
    a.r = r, a.w_next = w, a.x = x;
    a.ld_r = ld_r, a.ld_x = ld_x;
    a.r_type = r_type, a.w_type = w_type, a.x_type = x_type;
    a.eps = eps, a.flags = flags;
    return norm(a, M, H, stream);
}

pq2_status pq2_norm_residual(const pq2_norm_residual_args* args, int64_t M, int64_t H,
                             void* stream) {
    if (!args) return PQ2_ERR_INVALID_ARG;
    if (M > 0 && (!args->y || !args->r || !args->r_out)) return PQ2_ERR_INVALID_ARG;
    return norm(*args, M, H, stream);
}

static pq2_status check_lora(int64_t M, int64_t N, int64_t K, int64_t L, int64_t R) {
    if (M < 0 || N < 0 || K < 1 || L < 1 || R < 1) return PQ2_ERR_INVALID_ARG;
    if (K % 8 != 0 || K > PQ2_MAX_K || R % 8 != 0 || R > PQ2_LORA_MAX_R || L > PQ2_LORA_MAX_L ||
        M > PQ2_LORA_MAX_M || N > (int64_t(1) << 30))
        return PQ2_ERR_UNSUPPORTED_SHAPE;
    return PQ2_OK;
}

size_t pq2_lora_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t L, int64_t R) {
    if (check_lora(M, N, K, L, R) != PQ2_OK) return SIZE_MAX;
    return M == 0 ? 0 : pq2h::lora_workspace_bytes(M, N, K, L, R);
}

pq2_status pq2_lora_add(const void* x, int64_t ld_x, const void* A, const void* B, int type,
                        const int32_t* ids, const int32_t* ranks, const float* scales,
                        const void* y_in, int64_t ld_in, void* y_out, int64_t ld_out, int y_type,
                        int64_t M, int64_t N, int64_t K, int64_t L, int64_t R, void* workspace,
                        size_t workspace_bytes, void* stream) {
    pq2_status s = check_lora(M, N, K, L, R);
    if (s != PQ2_OK) return s;
    if ((type != PQ2_F16 && type != PQ2_BF16) || (y_type != PQ2_F32 && y_type != PQ2_BF16))
        return PQ2_ERR_INVALID_ARG;
    if (ld_x < K || ld_in < N || ld_out < N) return PQ2_ERR_INVALID_ARG;
    if (ld_x % 8 != 0) return PQ2_ERR_UNSUPPORTED_SHAPE;
    if (M == 0 || N == 0) return PQ2_OK;
    if (!x || !A || !B || !ids || !y_in || !y_out) return PQ2_ERR_INVALID_ARG;
    if (y_in == y_out && ld_in != ld_out) return PQ2_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(A) || !aligned16(B) || !aligned16(workspace) ||
        !aligned_to(ids, 4) || !aligned_to(ranks, 4) || !aligned_to(scales, 4) ||
        !aligned_to(y_in, type_bytes(y_type)) || !aligned_to(y_out, type_bytes(y_type)))
        return PQ2_ERR_MISALIGNED;
    pq2h::LoraParams p = {};
    p.x = static_cast<const uint16_t*>(x);
    p.A = static_cast<const uint16_t*>(A);
    p.B = static_cast<const uint16_t*>(B);
    p.ids = ids, p.ranks = ranks, p.scales = scales;
    p.y_in = y_in, p.y_out = y_out;
    p.ld_x = ld_x, p.ld_in = ld_in, p.ld_out = ld_out;
    p.M = static_cast<int>(M), p.N = static_cast<int>(N), p.K = static_cast<int>(K);
    p.L = static_cast<int>(L), p.R = static_cast<int>(R);
    p.bf16 = type == PQ2_BF16;
    p.y_type = y_type;
    if (!workspace || workspace_bytes < pq2h::lora_workspace_needed(p)) return PQ2_ERR_WORKSPACE;
    Ctx c;
    s = get_ctx(&c);
    if (s != PQ2_OK) return s;
    p.ctl = c.ctl;
    return cuda_status(pq2h::launch_lora(p, workspace, static_cast<cudaStream_t>(stream), c.dev));
}

// (bindings build these structs byte by byte)
static_assert(sizeof(pq2_lora_add_args) == 152 && sizeof(pq2_verify_drafts_args) == 136, "no padding");

pq2_status pq2_lora_add_packed(const pq2_lora_add_args* a, void* stream) {
    if (!a) return PQ2_ERR_INVALID_ARG;
    return pq2_lora_add(a->x, a->ld_x, a->A, a->B, a->type, a->ids, a->ranks, a->scales, a->y_in,
                        a->ld_in, a->y_out, a->ld_out, a->y_type, a->M, a->N, a->K, a->L, a->R,
                        a->workspace, a->workspace_bytes, stream);
}

static pq2_status check_verify(int64_t B, int64_t rows, int64_t V) {
    if (B < 0 || rows < 0 || V < 1) return PQ2_ERR_INVALID_ARG;
    // pieces of rows, and of sequences, are counted in 31 bits
    const int64_t pieces = V / 4096 + 2;
    if (V > (int64_t(1) << 30) || rows > (int64_t(1) << 24) || B > (int64_t(1) << 24) ||
        std::max(B, rows) * pieces > (int64_t(1) << 31) - 1)
        return PQ2_ERR_UNSUPPORTED_SHAPE;
    return PQ2_OK;
}

size_t pq2_verify_workspace_bytes(int64_t B, int64_t rows, int64_t V) {
    if (check_verify(B, rows, V) != PQ2_OK) return SIZE_MAX;
    return pq2h::verify_workspace_bytes(B, rows, V);
}

pq2_status pq2_verify_drafts(const float* logits, int64_t ld_logits, const int32_t* row_start,
                             const int32_t* drafts, const float* q, int64_t ld_q, const float* u,
                             const float* e, int64_t ld_e, const float* temperature,
                             int32_t* accepted, int32_t* tokens, int64_t B, int64_t rows, int64_t V,
                             void* workspace, size_t workspace_bytes, void* stream) {
    pq2_status s = check_verify(B, rows, V);
    if (s != PQ2_OK) return s;
    if (ld_logits < V || (q && ld_q < V) || ld_e < V) return PQ2_ERR_INVALID_ARG;
    if (B == 0) return PQ2_OK;
    if (!row_start || !e || !temperature || !accepted) return PQ2_ERR_INVALID_ARG;
    if (rows > 0 && (!logits || !drafts || !u || !tokens)) return PQ2_ERR_INVALID_ARG;
    if (!aligned_to(logits, 4) || !aligned_to(q, 4) || !aligned_to(u, 4) || !aligned_to(e, 4) ||
        !aligned_to(row_start, 4) || !aligned_to(drafts, 4) || !aligned_to(temperature, 4) ||
        !aligned_to(accepted, 4) || !aligned_to(tokens, 4) || !aligned16(workspace))
        return PQ2_ERR_MISALIGNED;
    if (!workspace || workspace_bytes < pq2h::verify_workspace_bytes(B, rows, V))
        return PQ2_ERR_WORKSPACE;
    Ctx c;
    s = get_ctx(&c);
    if (s != PQ2_OK) return s;
    pq2h::VerifyParams p = {};
    p.logits = logits, p.row_start = row_start, p.drafts = drafts, p.q = q, p.u = u, p.e = e;
    p.temperature = temperature, p.accepted = accepted, p.tokens = tokens;
    p.ld_logits = ld_logits, p.ld_q = ld_q, p.ld_e = ld_e;
    p.B = B, p.rows = rows, p.V = static_cast<int>(V);
    p.ctl = c.ctl;
    return cuda_status(pq2h::launch_verify(p, workspace, static_cast<cudaStream_t>(stream)));
}

pq2_status pq2_verify_drafts_packed(const pq2_verify_drafts_args* a, void* stream) {
    if (!a) return PQ2_ERR_INVALID_ARG;
    return pq2_verify_drafts(a->logits, a->ld_logits, a->row_start, a->drafts, a->q, a->ld_q, a->u,
                             a->e, a->ld_e, a->temperature, a->accepted, a->tokens, a->B, a->rows,
                             a->V, a->workspace, a->workspace_bytes, stream);
}

// --- rotary positions, the cache in 4 bits, its pages -----------------------

static_assert(sizeof(pq2_cache4) == 88 && sizeof(pq2_rope_args) == 160 &&
                  sizeof(pq2_cache4_append_args) == 240 && sizeof(pq2_cache4_read_args) == 152 &&
                  sizeof(pq2_cache4_attend_args) == 192 && sizeof(pq2_pages_update_args) == 144 &&
                  sizeof(pq2_pages_compact_args) == 120,
              "no padding");

// The last element (and one more) of an array [M, heads, dim].
static int64_t extent(int64_t M, int64_t ld, int64_t heads, int64_t hs, int64_t dim) {
    return M > 0 && heads > 0 ? (M - 1) * ld + (heads - 1) * hs + dim : 0;
}

// One array of heads: present, strides that keep heads and tokens apart.
static pq2_status check_heads(const void* x, int type, int64_t ld, int64_t hs, int64_t heads, int64_t dim) {
    if (heads == 0) return PQ2_OK;
    if (!x || (heads > 1 && hs < dim) || ld < dim || hs < 0) return PQ2_ERR_INVALID_ARG;
    return aligned_to(x, type_bytes(type)) ? PQ2_OK : PQ2_ERR_MISALIGNED;
}

pq2_status pq2_rope_table(float* table, int64_t first, int64_t count, int64_t rot, double base,
                          const pq2_rope_scaling* scaling, void* stream) {
    if (first < 0 || count < 0 || rot < 2 || rot % 2 != 0 || !(base > 1.0) || !std::isfinite(base))
        return PQ2_ERR_INVALID_ARG;
    pq2_rope_scaling s = {};
    if (scaling) s = *scaling;
    if (s.kind < PQ2_ROPE_PLAIN || s.kind > PQ2_ROPE_BANDS || !std::isfinite(s.magnitude)) return PQ2_ERR_INVALID_ARG;
    if (s.kind != PQ2_ROPE_PLAIN && (!(s.factor >= 1.0) || !std::isfinite(s.factor))) return PQ2_ERR_INVALID_ARG;
    if (s.kind == PQ2_ROPE_BASE && rot == 2) return PQ2_ERR_INVALID_ARG;
    if ((s.kind == PQ2_ROPE_RAMP || s.kind == PQ2_ROPE_BANDS) &&
        (!(s.old_len > 0.0) || !(s.low > 0.0) || !(s.high > s.low) || !std::isfinite(s.old_len) ||
         !std::isfinite(s.high)))
        return PQ2_ERR_INVALID_ARG;
    if (rot > PQ2_ROPE_MAX_DIM || first > (int64_t(1) << 31) || count > (int64_t(1) << 31) - first) return PQ2_ERR_UNSUPPORTED_SHAPE;
    if (count == 0) return PQ2_OK;
    if (!table) return PQ2_ERR_INVALID_ARG;
    if (!aligned16(table)) return PQ2_ERR_MISALIGNED;
    pq2h::RopeTableParams p = {};
    p.table = table;
    p.first = first, p.count = count;
    p.rot = static_cast<int>(rot);
    p.kind = s.kind;
    p.factor = s.kind == PQ2_ROPE_PLAIN ? 1.0 : s.factor;
    p.magnitude = s.magnitude == 0.0f ? 1.0 : s.magnitude;
    p.old_len = s.old_len, p.low = s.low, p.high = s.high;
    p.log_base = std::log(base);
    const double r = static_cast<double>(rot);
    if (s.kind == PQ2_ROPE_BASE) p.log_base += std::log(s.factor) * r / (r - 2.0);
    if (s.kind == PQ2_ROPE_RAMP) {
        // the index whose pair turns n times over old_len positions
        const auto index = [&](double n) { return r / 2.0 * std::log(s.old_len / (6.283185307179586476925 * n)) / p.log_base; };
        p.low = std::max(std::floor(index(s.high)), 0.0);
        p.high = std::min(std::ceil(index(s.low)), r - 1.0);
        if (p.high - p.low < 0.001) p.high = p.low + 0.001;
    }
    Ctx c;
    const pq2_status st = get_ctx(&c);
    if (st != PQ2_OK) return st;
    p.ctl = c.ctl;
    return cuda_status(pq2h::launch_rope_table(p, static_cast<cudaStream_t>(stream)));
}

pq2_status pq2_rope(const pq2_rope_args* args, void* stream) {
    if (!args) return PQ2_ERR_INVALID_ARG;
    const pq2_rope_args& a = *args;
    if (a.M < 0 || a.heads < 0 || a.heads2 < 0 || a.dim < 1 || a.rot < 0 || a.rot > a.dim || a.rot % 2 != 0 ||
        a.table_rows < 0 || a.reserved != 0 || (a.flags & ~(PQ2_ROPE_NEIGHBOURS | PQ2_ROPE_INVERSE)) ||
        !type_ok(a.x_type) || !type_ok(a.out_type))
        return PQ2_ERR_INVALID_ARG;
    if (a.dim > PQ2_ROPE_MAX_DIM || int64_t(a.heads) + a.heads2 > 65536 || a.M > (int64_t(1) << 24))
        return PQ2_ERR_UNSUPPORTED_SHAPE;
    if (a.M == 0 || a.heads + a.heads2 == 0) return PQ2_OK;
    pq2_status s = check_heads(a.x, a.x_type, a.ld_x, a.hs_x, a.heads, a.dim);
    if (s == PQ2_OK) s = check_heads(a.x2, a.x_type, a.ld_x2, a.hs_x2, a.heads2, a.dim);
    if (s == PQ2_OK) s = check_heads(a.out, a.out_type, a.ld_out, a.hs_out, a.heads, a.dim);
    if (s == PQ2_OK) s = check_heads(a.out2, a.out_type, a.ld_out2, a.hs_out2, a.heads2, a.dim);
    if (s != PQ2_OK) return s;
    if (a.rot > 0 && (!a.table || !a.positions)) return PQ2_ERR_INVALID_ARG;
    if (!aligned16(a.table) || !aligned_to(a.positions, 4)) return PQ2_ERR_MISALIGNED;
    if ((a.heads > 0 && a.out == a.x && (a.out_type != a.x_type || a.ld_out != a.ld_x || a.hs_out != a.hs_x)) ||
        (a.heads2 > 0 && a.out2 == a.x2 && (a.out_type != a.x_type || a.ld_out2 != a.ld_x2 || a.hs_out2 != a.hs_x2)))
        return PQ2_ERR_INVALID_ARG;
    Ctx c;
    s = get_ctx(&c);
    if (s != PQ2_OK) return s;
    pq2h::RopeParams p = {};
    p.x[0] = a.x, p.x[1] = a.x2, p.out[0] = a.out, p.out[1] = a.out2;
    p.ld[0] = a.ld_x, p.hs[0] = a.hs_x, p.ld[1] = a.ld_x2, p.hs[1] = a.hs_x2;
    p.ldo[0] = a.ld_out, p.hso[0] = a.hs_out, p.ldo[1] = a.ld_out2, p.hso[1] = a.hs_out2;
    p.out_elems[0] = extent(a.M, a.ld_out, a.heads, a.hs_out, a.dim);
    p.out_elems[1] = extent(a.M, a.ld_out2, a.heads2, a.hs_out2, a.dim);
    p.table = a.table, p.positions = a.positions;
    p.M = a.M, p.table_rows = a.table_rows;
    p.heads[0] = a.heads, p.heads[1] = a.heads2;
    p.dim = a.dim, p.rot = a.rot, p.x_type = a.x_type, p.out_type = a.out_type;
    p.flags = a.flags;
    p.ctl = c.ctl;
    return cuda_status(pq2h::launch_rope(p, static_cast<cudaStream_t>(stream)));
}

size_t pq2_cache4_page_bytes(int64_t heads, int64_t dim, int64_t page_tokens) {
    if (heads < 1 || heads > PQ2_CACHE4_MAX_HEADS || (dim != 64 && dim != 128 && dim != 256) || page_tokens < 16 ||
        page_tokens % 16 != 0 || page_tokens > 1024)
        return 0;
    return static_cast<size_t>(heads * page_tokens * (dim + 8));
}

// Sizes first (they decide what is supported), then, where there is work to
// do, pointers.
static pq2_status check_cache(const pq2_cache4& a) {
    if (a.B < 0 || a.W < 0 || a.num_pages < 0 || a.heads < 1 || a.reserved != 0) return PQ2_ERR_INVALID_ARG;
    const size_t page = pq2_cache4_page_bytes(a.heads, a.dim, a.page_tokens);
    if (page == 0 || a.B > (int64_t(1) << 20) || a.num_pages > (int64_t(1) << 30) || a.page_stride % 16 != 0 ||
        a.W > (int64_t(1) << 30) || a.W * a.page_tokens > (int64_t(1) << 30))
        return PQ2_ERR_UNSUPPORTED_SHAPE;
    if (a.page_stride < static_cast<int64_t>(page) || a.ld_pages < a.W) return PQ2_ERR_INVALID_ARG;
    return PQ2_OK;
}
static pq2_status check_cache_pointers(const pq2_cache4& a) {
    if (!a.row_start || !a.lens || (a.W > 0 && !a.pages) || (a.num_pages > 0 && !a.pool)) return PQ2_ERR_INVALID_ARG;
    if (!aligned16(a.pool) || !aligned_to(a.pages, 4) || !aligned_to(a.row_start, 4) || !aligned_to(a.lens, 4))
        return PQ2_ERR_MISALIGNED;
    return PQ2_OK;
}
static pq2h::CacheParams cache_params(const pq2_cache4& a) {
    pq2h::CacheParams p = {};
    p.pool = static_cast<uint8_t*>(a.pool);
    p.pages = a.pages, p.row_start = a.row_start, p.lens = a.lens;
    p.page_stride = a.page_stride, p.num_pages = a.num_pages, p.ld_pages = a.ld_pages;
    p.pool_bytes = a.num_pages > 0 ? (a.num_pages - 1) * a.page_stride +
                                         static_cast<int64_t>(pq2_cache4_page_bytes(a.heads, a.dim, a.page_tokens))
                                   : 0;
    p.B = static_cast<int>(a.B), p.W = static_cast<int>(a.W), p.heads = a.heads, p.T = a.page_tokens;
    return p;
}

pq2_status pq2_cache4_append(const pq2_cache4_append_args* args, void* stream) {
    if (!args) return PQ2_ERR_INVALID_ARG;
    const pq2_cache4_append_args& a = *args;
    pq2_status s = check_cache(a.cache);
    if (s != PQ2_OK) return s;
    const int dim = a.cache.dim;
    if (a.M < 0 || a.q_heads < 0 || a.rot < 0 || a.rot > dim || a.rot % 2 != 0 || a.table_rows < 0 || a.reserved != 0 ||
        (a.flags & ~PQ2_ROPE_NEIGHBOURS) || !type_ok(a.x_type) || (a.q_heads > 0 && !type_ok(a.out_type)))
        return PQ2_ERR_INVALID_ARG;
    if (a.M > (int64_t(1) << 24) || a.q_heads > 65536) return PQ2_ERR_UNSUPPORTED_SHAPE;
    if (a.M == 0 || a.cache.B == 0) return PQ2_OK;
    s = check_cache_pointers(a.cache);
    if (s == PQ2_OK) s = check_heads(a.k, a.x_type, a.ld_k, a.hs_k, a.cache.heads, dim);
    if (s == PQ2_OK) s = check_heads(a.v, a.x_type, a.ld_v, a.hs_v, a.cache.heads, dim);
    if (s == PQ2_OK) s = check_heads(a.q, a.x_type, a.ld_q, a.hs_q, a.q_heads, dim);
    if (s == PQ2_OK && a.q_heads > 0) s = check_heads(a.q_out, a.out_type, a.ld_q_out, a.hs_q_out, a.q_heads, dim);
    if (s != PQ2_OK) return s;
    if (a.rot > 0 && !a.table) return PQ2_ERR_INVALID_ARG;
    if (!aligned16(a.table) || !aligned_to(a.positions, 4)) return PQ2_ERR_MISALIGNED;
    if (a.q_heads > 0 && a.q_out == a.q && (a.out_type != a.x_type || a.ld_q_out != a.ld_q || a.hs_q_out != a.hs_q))
        return PQ2_ERR_INVALID_ARG;
    Ctx c;
    s = get_ctx(&c);
    if (s != PQ2_OK) return s;
    pq2h::RopeParams p = {};
    p.x[0] = a.q, p.x[1] = a.k, p.x[2] = a.v, p.out[0] = a.q_out;
    p.ld[0] = a.ld_q, p.hs[0] = a.hs_q, p.ld[1] = a.ld_k, p.hs[1] = a.hs_k, p.ld[2] = a.ld_v, p.hs[2] = a.hs_v;
    p.ldo[0] = a.ld_q_out, p.hso[0] = a.hs_q_out;
    p.out_elems[0] = extent(a.M, a.ld_q_out, a.q_heads, a.hs_q_out, dim);
    p.table = a.table, p.positions = a.positions;
    p.M = a.M, p.table_rows = a.table_rows;
    p.heads[0] = a.q_heads, p.heads[1] = p.heads[2] = a.cache.heads;
    p.dim = dim, p.rot = a.rot, p.x_type = a.x_type, p.out_type = a.out_type;
    p.flags = a.flags;
    p.cache = cache_params(a.cache);
    p.ctl = c.ctl;
    return cuda_status(pq2h::launch_cache_append(p, static_cast<cudaStream_t>(stream)));
}

pq2_status pq2_cache4_read(const pq2_cache4_read_args* args, void* stream) {
    if (!args) return PQ2_ERR_INVALID_ARG;
    const pq2_cache4_read_args& a = *args;
    pq2_status s = check_cache(a.cache);
    if (s != PQ2_OK) return s;
    const int dim = a.cache.dim, heads = a.cache.heads;
    if (a.M < 0 || a.reserved != 0 || !type_ok(a.out_type)) return PQ2_ERR_INVALID_ARG;
    if (a.M > (int64_t(1) << 24)) return PQ2_ERR_UNSUPPORTED_SHAPE;
    if (a.M == 0 || a.cache.B == 0 || (!a.k_out && !a.v_out)) return PQ2_OK;
    s = check_cache_pointers(a.cache);
    if (s == PQ2_OK && a.k_out) s = check_heads(a.k_out, a.out_type, a.ld_k, a.hs_k, heads, dim);
    if (s == PQ2_OK && a.v_out) s = check_heads(a.v_out, a.out_type, a.ld_v, a.hs_v, heads, dim);
    if (s != PQ2_OK) return s;
    Ctx c;
    s = get_ctx(&c);
    if (s != PQ2_OK) return s;
    pq2h::RopeParams p = {};
    int n = 0;
    for (int value = 0; value < 2; ++value) {
        if (!(value ? a.v_out : a.k_out)) continue;
        p.out[n] = value ? a.v_out : a.k_out;
        p.ldo[n] = value ? a.ld_v : a.ld_k;
        p.hso[n] = value ? a.hs_v : a.hs_k;
        p.out_elems[n] = extent(a.M, p.ldo[n], heads, p.hso[n], dim);
        p.heads[n] = heads;
        p.read_kind[n++] = value;
    }
    p.M = a.M;
    p.dim = dim, p.out_type = a.out_type;
    p.cache = cache_params(a.cache);
    p.ctl = c.ctl;
    return cuda_status(pq2h::launch_cache_read(p, static_cast<cudaStream_t>(stream)));
}

static pq2_status check_attend(int64_t M, int64_t q_heads, int64_t heads, int64_t dim) {
    if (M < 0 || q_heads < 1 || heads < 1 || q_heads % heads != 0) return PQ2_ERR_INVALID_ARG;
    if (M > (int64_t(1) << 20) || heads > PQ2_CACHE4_MAX_HEADS || q_heads / heads > 64 ||
        M * q_heads > (int64_t(1) << 30) || (dim != 64 && dim != 128 && dim != 256))
        return PQ2_ERR_UNSUPPORTED_SHAPE;
    return PQ2_OK;
}

size_t pq2_cache4_attend_workspace_bytes(int64_t M, int64_t q_heads, int64_t heads, int64_t dim) {
    if (check_attend(M, q_heads, heads, dim) != PQ2_OK) return SIZE_MAX;
    return M == 0 ? 0 : pq2h::attend_workspace_bytes(M, q_heads, heads, dim);
}

pq2_status pq2_cache4_attend(const pq2_cache4_attend_args* args, void* stream) {
    if (!args) return PQ2_ERR_INVALID_ARG;
    const pq2_cache4_attend_args& a = *args;
    pq2_status s = check_cache(a.cache);
    if (s == PQ2_OK) s = check_attend(a.M, a.q_heads, a.cache.heads, a.cache.dim);
    if (s != PQ2_OK) return s;
    const int dim = a.cache.dim;
    if ((a.type != PQ2_F16 && a.type != PQ2_BF16) || a.max_rows < 0 || a.window < 0 || !std::isfinite(a.scale) ||
        a.reserved != 0)
        return PQ2_ERR_INVALID_ARG;
    if (a.M == 0 || a.cache.B == 0) return PQ2_OK;
    s = check_cache_pointers(a.cache);
    if (s == PQ2_OK) s = check_heads(a.q, a.type, a.ld_q, a.hs_q, a.q_heads, dim);
    if (s == PQ2_OK) s = check_heads(a.out, a.type, a.ld_out, a.hs_out, a.q_heads, dim);
    if (s != PQ2_OK) return s;
    if (!aligned16(a.q) || !aligned16(a.out) || !aligned16(a.workspace) || a.ld_q % 8 != 0 || a.hs_q % 8 != 0 ||
        a.ld_out % 8 != 0 || a.hs_out % 8 != 0)
        return PQ2_ERR_MISALIGNED;
    if (!a.workspace || a.workspace_bytes < pq2h::attend_workspace_bytes(a.M, a.q_heads, a.cache.heads, dim))
        return PQ2_ERR_WORKSPACE;
    Ctx c;
    s = get_ctx(&c);
    if (s != PQ2_OK) return s;
    pq2h::AttendParams p = {};
    p.cache = cache_params(a.cache);
    p.q = static_cast<const uint16_t*>(a.q);
    p.out = static_cast<uint16_t*>(a.out);
    p.ld_q = a.ld_q, p.hs_q = a.hs_q, p.ld_out = a.ld_out, p.hs_out = a.hs_out;
    p.out_elems = extent(a.M, a.ld_out, a.q_heads, a.hs_out, dim);
    p.M = static_cast<int>(a.M);
    p.max_rows = static_cast<int>(a.max_rows > 0 ? std::min(a.max_rows, a.M) : a.M);
    p.window = static_cast<int>(std::min<int64_t>(a.window, (int64_t(1) << 30) + 1));
    p.q_heads = a.q_heads, p.dim = dim, p.bf16 = a.type == PQ2_BF16;
    p.scale = a.scale;
    p.ctl = c.ctl;
    return cuda_status(pq2h::launch_attend(p, a.workspace, static_cast<cudaStream_t>(stream), c.dev));
}

static pq2_status check_pages(int64_t B, int64_t W, int64_t P, int64_t T, int64_t ld_pages, int64_t ld_out) {
    if (B < 0 || W < 1 || P < 0 || T < 1) return PQ2_ERR_INVALID_ARG;
    if (B > (int64_t(1) << 20) || W > (int64_t(1) << 20) || B * W > (int64_t(1) << 30) || P > (int64_t(1) << 28) ||
        T > (int64_t(1) << 20) || W * T > (int64_t(1) << 30))
        return PQ2_ERR_UNSUPPORTED_SHAPE;
    return ld_pages >= W && ld_out >= W ? PQ2_OK : PQ2_ERR_INVALID_ARG;
}

size_t pq2_pages_workspace_bytes(int64_t B, int64_t P) {
    if (check_pages(B, 1, P, 1, 1, 1) != PQ2_OK) return SIZE_MAX;
    return pq2h::pages_workspace_bytes(B, P);
}

pq2_status pq2_pages_update(const pq2_pages_update_args* args, void* stream) {
    if (!args) return PQ2_ERR_INVALID_ARG;
    const pq2_pages_update_args& a = *args;
    pq2_status s = check_pages(a.B, a.W, a.P, a.T, a.ld_pages, a.ld_out);
    if (s != PQ2_OK) return s;
    if (!a.info || (a.P > 0 && (!a.refs || !a.refs_out)) ||
        (a.B > 0 && (!a.pages || !a.lens || !a.source || !a.keep || !a.new_lens || !a.pages_out || !a.copies)))
        return PQ2_ERR_INVALID_ARG;
    for (const void* x : {static_cast<const void*>(a.pages), static_cast<const void*>(a.lens),
                          static_cast<const void*>(a.refs), static_cast<const void*>(a.source),
                          static_cast<const void*>(a.keep), static_cast<const void*>(a.new_lens),
                          static_cast<const void*>(a.pages_out), static_cast<const void*>(a.refs_out),
                          static_cast<const void*>(a.copies), static_cast<const void*>(a.info)})
        if (!aligned_to(x, 4)) return PQ2_ERR_MISALIGNED;
    if (a.B > 0 && a.pages_out == a.pages) return PQ2_ERR_INVALID_ARG;
    if (!aligned16(a.workspace)) return PQ2_ERR_MISALIGNED;
    if (!a.workspace || a.workspace_bytes < pq2h::pages_workspace_bytes(a.B, a.P)) return PQ2_ERR_WORKSPACE;
    Ctx c;
    s = get_ctx(&c);
    if (s != PQ2_OK) return s;
    pq2h::PagesParams p = {};
    p.pages = a.pages, p.lens = a.lens, p.refs = a.refs, p.source = a.source, p.keep = a.keep;
    p.new_lens = a.new_lens, p.pages_out = a.pages_out, p.refs_out = a.refs_out, p.copies = a.copies;
    p.info = a.info;
    p.ld_pages = a.ld_pages, p.ld_out = a.ld_out;
    p.B = static_cast<int>(a.B), p.W = static_cast<int>(a.W), p.P = static_cast<int>(a.P);
    p.T = static_cast<int>(a.T);
    p.ctl = c.ctl;
    return cuda_status(pq2h::launch_pages_update(p, a.workspace, static_cast<cudaStream_t>(stream)));
}

pq2_status pq2_pages_compact(const pq2_pages_compact_args* args, void* stream) {
    if (!args) return PQ2_ERR_INVALID_ARG;
    const pq2_pages_compact_args& a = *args;
    pq2_status s = check_pages(a.B, a.W, a.P, a.T, a.ld_pages, a.ld_out);
    if (s != PQ2_OK) return s;
    if (!a.info || (a.P > 0 && (!a.refs || !a.refs_out)) || (a.P > 1 && !a.copies) ||
        (a.B > 0 && (!a.pages || !a.lens || !a.pages_out)))
        return PQ2_ERR_INVALID_ARG;
    for (const void* x : {static_cast<const void*>(a.pages), static_cast<const void*>(a.lens),
                          static_cast<const void*>(a.refs), static_cast<const void*>(a.pages_out),
                          static_cast<const void*>(a.refs_out), static_cast<const void*>(a.copies),
                          static_cast<const void*>(a.info)})
        if (!aligned_to(x, 4)) return PQ2_ERR_MISALIGNED;
    if (a.B > 0 && a.pages_out == a.pages && a.ld_out != a.ld_pages) return PQ2_ERR_INVALID_ARG;
    if (!aligned16(a.workspace)) return PQ2_ERR_MISALIGNED;
    if (!a.workspace || a.workspace_bytes < pq2h::pages_workspace_bytes(a.B, a.P)) return PQ2_ERR_WORKSPACE;
    Ctx c;
    s = get_ctx(&c);
    if (s != PQ2_OK) return s;
    pq2h::PagesParams p = {};
    p.pages = a.pages, p.lens = a.lens, p.refs = a.refs;
    p.pages_out = a.pages_out, p.refs_out = a.refs_out, p.copies = a.copies, p.info = a.info;
    p.ld_pages = a.ld_pages, p.ld_out = a.ld_out;
    p.B = static_cast<int>(a.B), p.W = static_cast<int>(a.W), p.P = static_cast<int>(a.P);
    p.T = static_cast<int>(a.T);
    p.ctl = c.ctl;
    return cuda_status(pq2h::launch_pages_compact(p, a.workspace, static_cast<cudaStream_t>(stream)));
}

pq2_status pq2_pages_copy(void* pool, int64_t page_bytes, int64_t page_stride, int64_t P, int64_t layers,
                          int64_t layer_stride, const int32_t* pairs, int64_t n, void* stream) {
    if (page_bytes < 0 || page_stride < page_bytes || P < 0 || layers < 0 || layer_stride < 0 || n < 0)
        return PQ2_ERR_INVALID_ARG;
    if (page_bytes % 16 != 0 || page_stride % 16 != 0 || layer_stride % 16 != 0 || layers > 65536 ||
        n > (int64_t(1) << 28) || P > (int64_t(1) << 31) || page_bytes > (int64_t(1) << 32))
        return PQ2_ERR_UNSUPPORTED_SHAPE;
    if (n == 0 || layers == 0 || P == 0 || page_bytes == 0) return PQ2_OK;
    if (!pool || !pairs) return PQ2_ERR_INVALID_ARG;
    if (!aligned16(pool) || !aligned_to(pairs, 8)) return PQ2_ERR_MISALIGNED;
    Ctx c;
    const pq2_status s = get_ctx(&c);
    if (s != PQ2_OK) return s;
    pq2h::PagesCopyParams p = {};
    p.pool = static_cast<uint8_t*>(pool);
    p.pairs = pairs;
    p.page_bytes = page_bytes, p.page_stride = page_stride, p.P = P, p.layer_stride = layer_stride, p.n = n;
    p.layers = static_cast<int>(layers);
    p.ctl = c.ctl;
    return cuda_status(pq2h::launch_pages_copy(p, static_cast<cudaStream_t>(stream), c.dev));
}

pq2_status pq2_group_dots(int op, const int8_t* qp, const int32_t* T, const uint8_t* codes,
                          int64_t M, int64_t N, int64_t K, int32_t* dots, void* workspace,
                          size_t workspace_bytes, void* stream) {
    pq2_status s = check_mm(qp, nullptr, T, codes, nullptr, dots, M, N, K);
    if (s != PQ2_OK) return s;
    if (op != PQ2_OP_GEMV && op != PQ2_OP_SMALL && op != PQ2_OP_PREFILL)
        return PQ2_ERR_INVALID_ARG;
    const size_t need = pq2_workspace_bytes(op, M, N, K);
    if (need == SIZE_MAX) return PQ2_ERR_UNSUPPORTED_SHAPE;
    if (need > 0 && (!workspace || workspace_bytes < need)) return PQ2_ERR_WORKSPACE;
    Ctx c;
    s = get_ctx(&c);
    if (s != PQ2_OK) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (op == PQ2_OP_GEMV)
        return cuda_status(
            pq2h::launch_gemv(nullptr, qp, nullptr, T, codes, nullptr, nullptr, dots, N, K, st,
                              c.ctl, c.dev));
    if (op == PQ2_OP_SMALL) {
        if (pq2h::gemv_multi_supported(M, N, K, c.dev.num_sms))
            return cuda_status(pq2h::launch_gemv_multi(qp, nullptr, T, codes, nullptr, nullptr,
                                                       dots, M, N, K, st, c.dev, false, c.ctl));
        return cuda_status(pq2h::launch_small_tc(qp, nullptr, T, codes, nullptr, nullptr, dots, M, N,
                                              K, workspace, st, c.ctl, c.dev));
    }
    // the prefill path needs S only to prepare its token planes
    return cuda_status(pq2h::launch_prefill(qp, nullptr, T, codes, nullptr, nullptr, dots, M, N,
                                            K, workspace, st, c.ctl, c.dev));
}

pq2_status pq2_last_device_error(void* stream) {
    Ctx c;
    pq2_status s = get_ctx(&c);
    if (s != PQ2_OK) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (cudaStreamSynchronize(st) != cudaSuccess) return PQ2_ERR_CUDA;
    unsigned word = 0;
    if (cudaMemcpy(&word, c.dev.err, sizeof(word), cudaMemcpyDeviceToHost) != cudaSuccess)
        return PQ2_ERR_CUDA;
    const unsigned zero = 0;
    if (cudaMemcpy(c.dev.err, &zero, sizeof(zero), cudaMemcpyHostToDevice) != cudaSuccess)
        return PQ2_ERR_CUDA;
    if (word & pq2::DEVERR_TIMEOUT) return PQ2_ERR_TIMEOUT;
    if (word & pq2::DEVERR_BOUNDS) return PQ2_ERR_BOUNDS;
    if (word & (pq2::DEVERR_BAD_TERNARY | pq2::DEVERR_BAD_INDEX)) return PQ2_ERR_INVALID_ARG;
    return PQ2_OK;
}

}  // extern "C"
