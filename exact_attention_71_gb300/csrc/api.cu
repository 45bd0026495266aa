// C ABI of the fused exact-attention forward: argument checks, TMA tensor
// maps, dispatch to the kernel instantiations, status and error reporting.
// The declarations and the contract are in include/attn.h.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <mutex>

#include "../../include/attn.h"
#include "attn_bwd.cuh"
#include "attn_bwd_kernel.cuh"
#include "attn_launch.cuh"
#include "fp8_prep.cuh"
#include "paged.cuh"

#include <algorithm>
#include <vector>

namespace attn {

bool causal_item_order(int nmb, int BH, int G, ItemOrder* order) {
    order->n = 0;
    const long long n = static_cast<long long>(nmb) * BH;
    if (n <= 0 || n > kOrderMax || G <= 0 || BH > 0xffff || nmb > 0xffff) return false;
    const int full = static_cast<int>((n / G) * G), rest = static_cast<int>(n) - full;
    struct It {
        int mb, bh;
    };
    // The `rest` lightest items, (query block ascending, head ascending)
    // positions below `rest`, form the last round; the rest, head by head
    // with the query block descending, make up the full rounds.
    std::vector<It> body, tail;
    body.reserve(static_cast<size_t>(full));
    for (int bh = 0; bh < BH; ++bh)
        for (int mb = nmb - 1; mb >= 0; --mb)
            if (static_cast<long long>(mb) * BH + bh >= rest) body.push_back({mb, bh});
    for (int mb = nmb - 1; mb >= 0; --mb)
        for (int bh = 0; bh < BH; ++bh)
            if (static_cast<long long>(mb) * BH + bh < rest) tail.push_back({mb, bh});
    auto heavier = [](const It& a, const It& b) { return a.mb > b.mb; };
    int k = 0;
    for (size_t r = 0; r < body.size(); r += static_cast<size_t>(G)) {
        auto first = body.begin() + static_cast<long>(r);
        auto last = body.begin() + static_cast<long>(std::min(body.size(), r + static_cast<size_t>(G)));
        std::stable_sort(first, last, heavier);     // heaviest first; heads ascending among equals
        for (auto x = first; x != last; ++x) order->e[k++] = static_cast<uint32_t>(x->mb) | (static_cast<uint32_t>(x->bh) << 16);
    }
    for (const It& x : tail) order->e[k++] = static_cast<uint32_t>(x.mb) | (static_cast<uint32_t>(x.bh) << 16);
    order->n = k;
    return k == n;
}

}  // namespace attn

namespace {

thread_local char g_err[512] = "";

int fail(int code, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    return code;
}

int cuda_fail(cudaError_t e, const char* what) {
    return fail(ATTN_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

// Device status word: first failing wait site of any kernel launched by the
// library (0 = none).  Its address is looked up once per device.
__device__ int g_attn_status;

constexpr int kMaxDevices = 64;
int* g_status_ptr[kMaxDevices] = {};
std::mutex g_status_mutex;

constexpr unsigned long long kDefaultWaitLimit = 4000000000ull;   // ~2 s of SM clock
std::atomic<unsigned long long> g_wait_limit{kDefaultWaitLimit};

int status_ptr(int** out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (dev < 0 || dev >= kMaxDevices) return fail(ATTN_ERR_UNSUPPORTED, "device ordinal %d out of range", dev);
    std::lock_guard<std::mutex> lock(g_status_mutex);
    if (!g_status_ptr[dev]) {
        void* ptr = nullptr;
        e = cudaGetSymbolAddress(&ptr, g_attn_status);
        if (e != cudaSuccess) return cuda_fail(e, "cudaGetSymbolAddress(status)");
        g_status_ptr[dev] = static_cast<int*>(ptr);
    }
    *out = g_status_ptr[dev];
    return ATTN_OK;
}

int g_sm_count[kMaxDevices] = {};

// Streaming multiprocessors of the current device (cached per device).
int sm_count(int* out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (dev < 0 || dev >= kMaxDevices) return fail(ATTN_ERR_UNSUPPORTED, "device ordinal %d out of range", dev);
    std::lock_guard<std::mutex> lock(g_status_mutex);
    if (g_sm_count[dev] == 0) {
        int n = 0;
        e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute(multiProcessorCount)");
        g_sm_count[dev] = n > 0 ? n : 1;
    }
    *out = g_sm_count[dev];
    return ATTN_OK;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// (B, N, H, d) tensor viewed as 4-D {d, H, N, B}; box = one `swizzle`-byte
// column block (128, or 64 for 64-byte rows) of `rows` tokens of one head,
// with that swizzle (the layout the MMA shared-memory descriptors expect).
// Rows past N read as zero.
int make_map(CUtensorMap* map, const void* base, int B, int H, int N, int d, int elem_bytes, int rows,
             int swizzle = 128) {
    auto enc = encode_fn();
    if (!enc) return fail(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    const CUtensorMapDataType dt =
        elem_bytes == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8;
    cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(N),
                          static_cast<cuuint64_t>(B)};
    cuuint64_t strides[3] = {static_cast<cuuint64_t>(d) * elem_bytes, static_cast<cuuint64_t>(H) * d * elem_bytes,
                             static_cast<cuuint64_t>(N) * H * d * elem_bytes};
    cuuint32_t box[4] = {static_cast<cuuint32_t>(swizzle / elem_bytes), 1, static_cast<cuuint32_t>(rows), 1};
    cuuint32_t estride[4] = {1, 1, 1, 1};
    CUresult r = enc(map, dt, 4, const_cast<void*>(base), dims, strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     swizzle == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled failed (CUresult %d)", static_cast<int>(r));
    return ATTN_OK;
}

// bf16 (B, N, H, d) tensor as 4-D {d, H, N, B}; box = whole rows (d
// elements) of 128 tokens of one head, no swizzle: the FP8 prep's tile.
int make_row_map(CUtensorMap* map, const void* base, int B, int H, int N, int d) {
    auto enc = encode_fn();
    if (!enc) return fail(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(N),
                          static_cast<cuuint64_t>(B)};
    cuuint64_t strides[3] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(H) * d * 2,
                             static_cast<cuuint64_t>(N) * H * d * 2};
    cuuint32_t box[4] = {static_cast<cuuint32_t>(d), 1, 128, 1};
    cuuint32_t estride[4] = {1, 1, 1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estride,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled (rows) failed (CUresult %d)", static_cast<int>(r));
    return ATTN_OK;
}

// Everything the prep launch needs besides its arguments.
int prep_launch(const void* x, int B, int H, int N, int d, CUtensorMap* map, attn::PrepLaunch* L) {
    int rc = make_row_map(map, x, B, H, N, d);
    if (rc != ATTN_OK) return rc;
    if ((rc = sm_count(&L->num_sms)) != ATTN_OK) return rc;
    if ((rc = status_ptr(&L->status)) != ATTN_OK) return rc;
    L->wait_limit = g_wait_limit.load();
    return ATTN_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The tensor-core prep (modes 0 and 1 at d = 64 and 128) of up to three bf16
// (B, N, H_i, d) tensors in one launch: x[i] -> codes x8[i], block scales
// scales[i]; rotate[i] = 1 multiplies tensor i by diag(+-1) x Hadamard.
int prep_tc(int n, const void* const* x, void* const* x8, float* const* scales, const int* Hs, const int* rotate,
            int B, int N, int d, unsigned long long sign_seed, cudaStream_t stream) {
    CUtensorMap maps[3];
    attn::PrepTcParams p{};
    p.N = N;
    p.nblk = (N + 127) / 128;
    long long total = 0;
    for (int i = 0; i < 3; ++i) {
        const int src = i < n ? i : 0;     // unused slots repeat tensor 0's map, with no blocks
        int rc = make_map(&maps[i], x[src], B, Hs[src], N, d, 2, 128, 128);
        if (rc != ATTN_OK) return rc;
        p.t[i].x8 = static_cast<uint8_t*>(x8[src]);
        p.t[i].scales = scales[src];
        p.t[i].H = Hs[src];
        p.t[i].rotate = rotate[src];
        const long long blocks = i < n ? static_cast<long long>(B) * Hs[i] * p.nblk : 0;
        p.t[i].blocks = static_cast<int>(blocks);
        total += blocks;
    }
    if (total >= (1ll << 31)) return fail(ATTN_ERR_INVALID_ARG, "problem too large for one launch");
    p.total_blocks = static_cast<int>(total);
    p.seed = sign_seed;
    attn::PrepLaunch L;
    int rc = sm_count(&L.num_sms);
    if (rc != ATTN_OK) return rc;
    if ((rc = status_ptr(&L.status)) != ATTN_OK) return rc;
    L.wait_limit = g_wait_limit.load();
    p.wait_limit = L.wait_limit;
    p.status = L.status;
    cudaError_t e = attn::run_fp8_prep_tc(maps, p, d, L, stream);
    if (e != cudaSuccess) return cuda_fail(e, "FP8 prep launch");
    return ATTN_OK;
}

int check_common(const void* q, const void* k, const void* v, const void* o, const float* lse, int B, int H, int N,
                 int d, int window) {
    if (B < 0 || H < 0 || N < 0) return fail(ATTN_ERR_INVALID_ARG, "negative size (B=%d H=%d N=%d)", B, H, N);
    if (d != 64 && d != 128 && d != 256) return fail(ATTN_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128, 256)", d);
    if (window < 0) return fail(ATTN_ERR_INVALID_ARG, "window %d < 0", window);
    if (static_cast<long long>(B) * H * N == 0) return ATTN_OK;
    if (!q || !k || !v || !o || !lse) return fail(ATTN_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
        return fail(ATTN_ERR_INVALID_ARG, "pointers must be 16-byte aligned");
    const long long items = static_cast<long long>(B) * H * ((N + 127) / 128);
    if (items >= (1ll << 31)) return fail(ATTN_ERR_INVALID_ARG, "problem too large for one launch");
    return ATTN_OK;
}

float resolve_scale(float scale, int d) {
    if (!(scale > 0.0f) || !std::isfinite(scale)) scale = 1.0f / std::sqrt(static_cast<float>(d));
    return scale;
}

int launch_forward(bool fp8, const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int Hkv,
                   int N, int d, int causal, float scale, int window, const float* qs, const float* ks, const float* vs,
                   void* stream, const uint8_t* block_mask = nullptr) {
    attn::FwdGeometry g;
    cudaError_t (*run)(const attn::FwdMaps&, const attn::FwdParams&, int, cudaStream_t) = nullptr;
    if (block_mask) {
        if (d == 64) {
            g = attn::geom_sparse_d64();
            run = attn::run_fwd_sparse_d64;
        } else if (d == 128) {
            g = attn::geom_sparse_d128();
            run = attn::run_fwd_sparse_d128;
        } else {
            g = attn::geom_sparse_d256();
            run = attn::run_fwd_sparse_d256;
        }
    } else if (fp8) {
        if (d == 128) {
            g = attn::geom_fp8_d128();
            run = attn::run_fwd_fp8_d128;
        } else if (d == 64) {
            g = attn::geom_fp8_d64();
            run = attn::run_fwd_fp8_d64;
        } else if (d == 256) {
            g = attn::geom_fp8_d256();
            run = attn::run_fwd_fp8_d256;
        } else {
            return fail(ATTN_ERR_UNSUPPORTED, "attn_fwd_fp8 supports head_dim 64, 128 and 256 (got %d)", d);
        }
    } else if (d == 64) {
        g = attn::geom_bf16_d64();
        run = attn::run_fwd_bf16_d64;
    } else if (d == 128) {
        g = attn::geom_bf16_d128();
        run = attn::run_fwd_bf16_d128;
    } else {
        g = attn::geom_bf16_d256();
        run = attn::run_fwd_bf16_d256;
    }
    attn::FwdMaps maps;
    int rc;
    if ((rc = make_map(&maps.q, q, B, H, N, d, g.elem_bytes, 128, g.swizzle)) != ATTN_OK) return rc;
    if ((rc = make_map(&maps.k, k, B, Hkv, N, d, g.elem_bytes, g.bn, g.swizzle)) != ATTN_OK) return rc;
    if ((rc = make_map(&maps.v, v, B, Hkv, N, d, g.elem_bytes, g.bn, g.swizzle)) != ATTN_OK) return rc;
    if ((rc = make_map(&maps.o, o, B, H, N, d, 2, 32, 128)) != ATTN_OK) return rc;
    attn::FwdParams p{};
    p.o = o;
    p.lse = lse;
    p.q_scale = qs;
    p.k_scale = ks;
    p.v_scale = vs;
    p.B = B;
    p.H = H;
    p.N = N;
    p.group = H / Hkv;
    p.causal = causal ? 1 : 0;
    p.window = window;
    p.scale_log2 = resolve_scale(scale, d) * 1.4426950408889634f;
    p.n_mblocks = (N + g.nq * 128 - 1) / (g.nq * 128);
    p.block_mask = block_mask;
    p.n_tb = (N + 127) / 128;
    p.wait_limit = g_wait_limit.load();
    if ((rc = status_ptr(&p.status)) != ATTN_OK) return rc;
    int sms = 0;
    if ((rc = sm_count(&sms)) != ATTN_OK) return rc;
    // Causal launches of the d = 128 kernels without grouped heads take their
    // work order from the launch parameters (copied at the launch, so the
    // buffer is free again when run() returns).  With grouped heads several
    // query heads already share each K/V head; the order then only crowds
    // more CTAs onto the same tiles.
    static thread_local attn::ItemOrder order;
    if (causal && !block_mask && d == 128 && Hkv == H) {
        const long long units = static_cast<long long>(p.n_mblocks) * B * H;
        const int G = static_cast<int>(units < sms ? units : sms);
        if (attn::causal_item_order(p.n_mblocks, B * H, G, &order)) maps.order = &order;
    }
    cudaError_t e = run(maps, p, sms, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess)
        return cuda_fail(e, block_mask ? "attn_fwd_sparse launch" : (fp8 ? "attn_fwd_fp8 launch" : "attn_fwd launch"));
    return ATTN_OK;
}

}  // namespace

extern "C" {

int attn_fwd_work_order(int n_mblocks, int BH, int grid, unsigned int* out, int capacity) {
    if (out == nullptr || n_mblocks <= 0 || BH <= 0 || grid <= 0) return 0;
    static thread_local attn::ItemOrder order;
    if (!attn::causal_item_order(n_mblocks, BH, grid, &order) || order.n > capacity) return 0;
    for (int i = 0; i < order.n; ++i) out[i] = order.e[i];
    return order.n;
}

int attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int N, int d,
             int causal, float scale, int window, void* stream) {
    return attn_fwd_gqa(q, k, v, o, lse, B, H, H, N, d, causal, scale, window, stream);
}

int attn_fwd_gqa(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int H_kv, int N,
                 int d, int causal, float scale, int window, void* stream) {
    g_err[0] = '\0';
    int rc = check_common(q, k, v, o, lse, B, H, N, d, window);
    if (rc != ATTN_OK) return rc;
    if (H_kv <= 0 || H % H_kv != 0)
        return fail(ATTN_ERR_INVALID_ARG, "key/value heads (%d) must divide query heads (%d)", H_kv, H);
    if (static_cast<long long>(B) * H * N == 0) return ATTN_OK;
    return launch_forward(false, q, k, v, o, lse, B, H, H_kv, N, d, causal, scale, window, nullptr, nullptr,
                          nullptr, stream);
}

int attn_fwd_fp8(const void* q8, const void* k8, const void* v8, void* o, float* lse, int B, int H, int N, int d,
                 int causal, float scale, int window, const float* q_scale, const float* k_scale,
                 const float* v_scale, void* stream) {
    return attn_fwd_fp8_gqa(q8, k8, v8, o, lse, B, H, H, N, d, causal, scale, window, q_scale, k_scale, v_scale,
                            stream);
}

int attn_fwd_fp8_gqa(const void* q8, const void* k8, const void* v8, void* o, float* lse, int B, int H, int H_kv,
                     int N, int d, int causal, float scale, int window, const float* q_scale, const float* k_scale,
                     const float* v_scale, void* stream) {
    g_err[0] = '\0';
    int rc = check_common(q8, k8, v8, o, lse, B, H, N, d, window);
    if (rc != ATTN_OK) return rc;
    if (H_kv <= 0 || H % H_kv != 0)
        return fail(ATTN_ERR_INVALID_ARG, "key/value heads (%d) must divide query heads (%d)", H_kv, H);
    if (static_cast<long long>(B) * H * N == 0) return ATTN_OK;
    if (d != 64 && d != 128 && d != 256)
        return fail(ATTN_ERR_UNSUPPORTED, "attn_fwd_fp8 supports head_dim 64, 128 and 256 (got %d)", d);
    if (!q_scale || !k_scale || !v_scale) return fail(ATTN_ERR_INVALID_ARG, "null scale pointer");
    return launch_forward(true, q8, k8, v8, o, lse, B, H, H_kv, N, d, causal, scale, window, q_scale, k_scale,
                          v_scale, stream);
}

int attn_fp8_prep(const void* x, void* x8, float* scales, int B, int H, int N, int d, int block_rows, int mode,
                  unsigned long long sign_seed, int is_v, void* stream) {
    g_err[0] = '\0';
    if (B < 0 || H < 0 || N < 0) return fail(ATTN_ERR_INVALID_ARG, "negative size (B=%d H=%d N=%d)", B, H, N);
    if (d != 64 && d != 128 && d != 256) return fail(ATTN_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128, 256)", d);
    if (block_rows != 128) return fail(ATTN_ERR_UNSUPPORTED, "block_rows must be 128 (got %d)", block_rows);
    if (mode < 0 || mode > 2) return fail(ATTN_ERR_INVALID_ARG, "mode %d (0, 1 or 2)", mode);
    if (static_cast<long long>(B) * H * N == 0) return ATTN_OK;
    if (!x || !x8 || !scales) return fail(ATTN_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(x) || !aligned16(x8) || !aligned16(scales))
        return fail(ATTN_ERR_INVALID_ARG, "pointers must be 16-byte aligned");
    if ((mode == 0 || mode == 1) && d <= 128) {
        // The rotation as a tensor-core product.
        const int rot = (mode == 1 && !is_v) ? 1 : 0;
        return prep_tc(1, &x, &x8, &scales, &H, &rot, B, N, d, sign_seed, static_cast<cudaStream_t>(stream));
    }
    CUtensorMap map;
    attn::PrepLaunch L;
    int rc = prep_launch(x, B, H, N, d, &map, &L);
    if (rc != ATTN_OK) return rc;
    cudaError_t e = attn::run_fp8_prep(map, x8, scales, B, H, N, d, mode, sign_seed, is_v != 0, nullptr, nullptr, 0, L,
                                       static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "attn_fp8_prep launch");
    return ATTN_OK;
}

int attn_fp8_prep_qkv(const void* q, const void* k, const void* v, void* q8, void* k8, void* v8, float* q_scale,
                      float* k_scale, float* v_scale, int B, int H, int H_kv, int N, int d, int mode,
                      unsigned long long sign_seed, void* stream) {
    g_err[0] = '\0';
    if (B < 0 || H < 0 || N < 0) return fail(ATTN_ERR_INVALID_ARG, "negative size (B=%d H=%d N=%d)", B, H, N);
    if (d != 64 && d != 128 && d != 256) return fail(ATTN_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128, 256)", d);
    if (mode < 0 || mode > 2) return fail(ATTN_ERR_INVALID_ARG, "mode %d (0, 1 or 2)", mode);
    if (H_kv <= 0 || H % H_kv != 0)
        return fail(ATTN_ERR_INVALID_ARG, "key/value heads (%d) must divide query heads (%d)", H_kv, H);
    if (static_cast<long long>(B) * H * N == 0) return ATTN_OK;
    const void* x[3] = {q, k, v};
    void* x8[3] = {q8, k8, v8};
    float* sc[3] = {q_scale, k_scale, v_scale};
    for (int i = 0; i < 3; ++i) {
        if (!x[i] || !x8[i] || !sc[i]) return fail(ATTN_ERR_INVALID_ARG, "null pointer");
        if (!aligned16(x[i]) || !aligned16(x8[i]) || !aligned16(sc[i]))
            return fail(ATTN_ERR_INVALID_ARG, "pointers must be 16-byte aligned");
    }
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if ((mode == 0 || mode == 1) && d <= 128) {
        const int Hs[3] = {H, H_kv, H_kv};
        const int rot[3] = {mode == 1 ? 1 : 0, mode == 1 ? 1 : 0, 0};
        return prep_tc(3, x, x8, sc, Hs, rot, B, N, d, sign_seed, s);
    }
    // Head dim 256 and the per-tensor mode: one launch per tensor.
    int rc = attn_fp8_prep(q, q8, q_scale, B, H, N, d, 128, mode, sign_seed, 0, stream);
    if (rc == ATTN_OK) rc = attn_fp8_prep(k, k8, k_scale, B, H_kv, N, d, 128, mode, sign_seed, 0, stream);
    if (rc == ATTN_OK) rc = attn_fp8_prep(v, v8, v_scale, B, H_kv, N, d, 128, mode, sign_seed, 1, stream);
    return rc;
}

int attn_fp8_prep_rope(const void* x, void* x8, float* scales, const float* rope_cos, const float* rope_sin,
                       int B, int H, int N, int d, int block_rows, int mode, unsigned long long sign_seed,
                       int interleaved, void* stream) {
    g_err[0] = '\0';
    if (B < 0 || H < 0 || N < 0) return fail(ATTN_ERR_INVALID_ARG, "negative size (B=%d H=%d N=%d)", B, H, N);
    if (d != 64 && d != 128 && d != 256) return fail(ATTN_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128, 256)", d);
    if (block_rows != 128) return fail(ATTN_ERR_UNSUPPORTED, "block_rows must be 128 (got %d)", block_rows);
    if (mode < 0 || mode > 2) return fail(ATTN_ERR_INVALID_ARG, "mode %d (0, 1 or 2)", mode);
    if (static_cast<long long>(B) * H * N == 0) return ATTN_OK;
    if (!x || !x8 || !scales || !rope_cos || !rope_sin) return fail(ATTN_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(x) || !aligned16(x8) || !aligned16(scales) || !aligned16(rope_cos) || !aligned16(rope_sin))
        return fail(ATTN_ERR_INVALID_ARG, "pointers must be 16-byte aligned");
    CUtensorMap map;
    attn::PrepLaunch L;
    int rc = prep_launch(x, B, H, N, d, &map, &L);
    if (rc != ATTN_OK) return rc;
    cudaError_t e = attn::run_fp8_prep(map, x8, scales, B, H, N, d, mode, sign_seed, false, rope_cos, rope_sin,
                                       interleaved ? 2 : 1, L, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "attn_fp8_prep_rope launch");
    return ATTN_OK;
}

int attn_fwd_sparse(const void* q, const void* k, const void* v, void* o, float* lse, const unsigned char* block_mask,
                    int B, int H, int H_kv, int N, int d, int causal, float scale, int window, void* stream) {
    g_err[0] = '\0';
    int rc = check_common(q, k, v, o, lse, B, H, N, d, window);
    if (rc != ATTN_OK) return rc;
    if (H_kv <= 0 || H % H_kv != 0)
        return fail(ATTN_ERR_INVALID_ARG, "key/value heads (%d) must divide query heads (%d)", H_kv, H);
    if (static_cast<long long>(B) * H * N == 0) return ATTN_OK;
    if (!block_mask) return fail(ATTN_ERR_INVALID_ARG, "null block mask");
    return launch_forward(false, q, k, v, o, lse, B, H, H_kv, N, d, causal, scale, window, nullptr, nullptr, nullptr,
                          stream, block_mask);
}

size_t attn_bwd_workspace_size(int B, int H, int N, int d) {
    if (B < 0 || H < 0 || N < 0 || d <= 0) return 0;
    return static_cast<size_t>(attn::bwd_workspace(B, H, N, d).bytes);
}

int attn_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dout,
             void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes, int B, int H, int H_kv, int N,
             int d, int causal, float scale, int window, void* stream) {
    g_err[0] = '\0';
    int rc = check_common(q, k, v, o, lse, B, H, N, d, window);
    if (rc != ATTN_OK) return rc;
    if (d != 128 && d != 64) return fail(ATTN_ERR_UNSUPPORTED, "attn_bwd supports head_dim 64 and 128 (got %d)", d);
    if (H_kv <= 0 || H % H_kv != 0)
        return fail(ATTN_ERR_INVALID_ARG, "key/value heads (%d) must divide query heads (%d)", H_kv, H);
    if (static_cast<long long>(B) * H * N == 0) return ATTN_OK;
    if (!dout || !dq || !dk || !dv || !workspace) return fail(ATTN_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(dout) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv))
        return fail(ATTN_ERR_INVALID_ARG, "pointers must be 16-byte aligned");
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return fail(ATTN_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    const attn::BwdWorkspace ws = attn::bwd_workspace(B, H, N, d);
    if (workspace_bytes < static_cast<size_t>(ws.bytes))
        return fail(ATTN_ERR_INVALID_ARG, "workspace of %zu bytes is smaller than the %lld bytes needed",
                    workspace_bytes, ws.bytes);
    attn::BwdMaps maps;
    const int qrows = attn::bwd_query_rows(d);
    if ((rc = make_map(&maps.q, q, B, H, N, d, 2, qrows)) != ATTN_OK) return rc;
    if ((rc = make_map(&maps.dout, dout, B, H, N, d, 2, qrows)) != ATTN_OK) return rc;
    if ((rc = make_map(&maps.k, k, B, H_kv, N, d, 2, 128)) != ATTN_OK) return rc;
    if ((rc = make_map(&maps.v, v, B, H_kv, N, d, 2, 128)) != ATTN_OK) return rc;
    uint8_t* wsb = static_cast<uint8_t*>(workspace);
    attn::BwdParams p{};
    p.lse2 = reinterpret_cast<const float*>(wsb + ws.off_lse2);
    p.dvec = reinterpret_cast<const float*>(wsb + ws.off_dvec);
    p.dq_acc = reinterpret_cast<float*>(wsb + ws.off_dq);
    p.dk = dk;
    p.dv = dv;
    p.B = B;
    p.H = H;
    p.H_kv = H_kv;
    p.N = N;
    p.N_pad = ws.n_pad;
    p.group = H / H_kv;
    p.causal = causal ? 1 : 0;
    p.window = window;
    p.scale = resolve_scale(scale, d);
    p.scale_log2 = p.scale * 1.4426950408889634f;
    p.n_kblocks = (N + 127) / 128;
    p.wait_limit = g_wait_limit.load();
    if ((rc = status_ptr(&p.status)) != ATTN_OK) return rc;
    cudaError_t e = attn::run_bwd(d, maps, p, o, dout, lse, dq, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "attn_bwd launch");
    return ATTN_OK;
}

int attn_device_status(void* stream, int* site) {
    g_err[0] = '\0';
    if (site) *site = 0;
    cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "cudaStreamSynchronize");
    int* ptr = nullptr;
    int rc = status_ptr(&ptr);
    if (rc != ATTN_OK) return rc;
    int value = 0;
    e = cudaMemcpy(&value, ptr, sizeof value, cudaMemcpyDeviceToHost);
    if (e != cudaSuccess) return cuda_fail(e, "reading the status word");
    if (value != 0) {
        const int zero = 0;
        e = cudaMemcpy(ptr, &zero, sizeof zero, cudaMemcpyHostToDevice);
        if (e != cudaSuccess) return cuda_fail(e, "clearing the status word");
        if (site) *site = value;
        if (value >= attn::SITE_BAD_INDEX)
            return fail(ATTN_ERR_BAD_INDEX, "a kernel refused %s (site 0x%x)",
                        value == attn::SITE_PAGED_SLOT   ? "a cache slot beyond the cache"
                        : value == attn::SITE_PAGED_PAGE ? "a page index outside the cache"
                                                         : "a sequence length beyond its page table",
                        value);
        return fail(ATTN_ERR_DEVICE_TIMEOUT, "a kernel gave up waiting at site 0x%x", value);
    }
    return ATTN_OK;
}

int attn_set_wait_limit(unsigned long long cycles) {
    g_err[0] = '\0';
    g_wait_limit.store(cycles ? cycles : kDefaultWaitLimit);
    return ATTN_OK;
}

const char* attn_last_error_string(void) { return g_err; }

}  // extern "C"

// ---------------------------------------------------------------------------
// attn_bwd_noalloc: the backward for callers that cannot allocate device
// memory (see include/attn.h).  Its scratch -- the LSE / D rows and the
// float32 dQ accumulator that attn_bwd keeps in the caller's workspace -- is
// this file-scope array, created once per device when the library's device
// code is loaded there and held until the process exits.
namespace {

constexpr size_t kNoAllocScratchBytes = size_t(256) << 20;   // 256 MiB
static __device__ __align__(256) unsigned char g_bwd_scratch[kNoAllocScratchBytes];

void* g_scratch_ptr[kMaxDevices] = {};
std::mutex g_scratch_mutex;

// Device address of g_bwd_scratch on the current device (host code may not
// use the array's name as a device address).  Looked up once per device.
int scratch_ptr(void** out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (dev < 0 || dev >= kMaxDevices) return fail(ATTN_ERR_UNSUPPORTED, "device ordinal %d out of range", dev);
    std::lock_guard<std::mutex> lock(g_scratch_mutex);
    if (!g_scratch_ptr[dev]) {
        void* ptr = nullptr;
        e = cudaGetSymbolAddress(&ptr, g_bwd_scratch);
        if (e != cudaSuccess) return cuda_fail(e, "cudaGetSymbolAddress(backward scratch)");
        g_scratch_ptr[dev] = ptr;
    }
    *out = g_scratch_ptr[dev];
    return ATTN_OK;
}

}  // namespace

extern "C" {

size_t attn_bwd_noalloc_max_scratch(void) { return kNoAllocScratchBytes; }

int attn_bwd_noalloc(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dout,
                     void* dq, void* dk, void* dv, int B, int H, int H_kv, int N, int d, int causal, float scale,
                     int window, void* stream) {
    g_err[0] = '\0';
    if (B < 0 || H < 0 || N < 0) return fail(ATTN_ERR_INVALID_ARG, "negative size (B=%d H=%d N=%d)", B, H, N);
    if ((d == 128 || d == 64) && static_cast<long long>(B) * H * N > 0) {
        const size_t need = attn_bwd_workspace_size(B, H, N, d);
        if (need > kNoAllocScratchBytes)
            return fail(ATTN_ERR_INVALID_ARG,
                        "attn_bwd_noalloc: this problem needs %zu bytes of scratch, more than the built-in %zu "
                        "(4 * B * H * ceil(N / 128) * 128 * (d + 2) bytes must fit); use attn_bwd with a workspace",
                        need, kNoAllocScratchBytes);
    }
    void* scratch = nullptr;
    if (static_cast<long long>(B) * H * N > 0) {
        const int rc = scratch_ptr(&scratch);
        if (rc != ATTN_OK) return rc;
    }
    // The prep launch of attn_bwd rewrites every scratch entry the call reads
    // (it zeroes the dQ accumulator), so nothing left by an earlier call leaks in.
    return attn_bwd(q, k, v, o, lse, dout, dq, dk, dv, scratch, kNoAllocScratchBytes, B, H, H_kv, N, d, causal, scale,
                    window, stream);
}

}  // extern "C"

// ---------------------------------------------------------------------------
// attn_fwd_host: the forward on host buffers (see include/attn.h).  Chunks of
// whole sequences go through two device staging slots; per chunk c (slot
// c % 2, counted per device across calls):
//   h2d stream : wait freed[slot] (the D2H of the chunk that used the slot
//                before), copy Q, K, V in, record loaded[slot]
//   comp stream: wait loaded[slot], forward, record computed[slot]
//   d2h stream : wait computed[slot], copy O, LSE out, record freed[slot]
// so the copies in one direction overlap the forward and the copies in the
// other direction of the neighbouring chunks.

namespace {

constexpr int kHostChunks = 4;   // chunks per call (at most B)

struct HostPipe {
    cudaStream_t h2d = nullptr, comp = nullptr, d2h = nullptr;
    cudaEvent_t entry = nullptr, done = nullptr;
    cudaEvent_t loaded[2] = {}, computed[2] = {}, freed[2] = {};
    unsigned long long chunks = 0;
    const void* last_ws = nullptr;   // staging layout of the previous call
    size_t last_slot = 0;
    bool ready = false;
};

HostPipe g_pipe[kMaxDevices];
std::mutex g_pipe_mutex;   // guards g_pipe and the order of the enqueued work

// Called with g_pipe_mutex held.
int host_pipe(HostPipe** out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (dev < 0 || dev >= kMaxDevices) return fail(ATTN_ERR_UNSUPPORTED, "device ordinal %d out of range", dev);
    HostPipe& P = g_pipe[dev];
    if (!P.ready) {
        cudaStream_t* streams[3] = {&P.h2d, &P.comp, &P.d2h};
        for (cudaStream_t* s : streams) {
            if (*s) continue;
            e = cudaStreamCreateWithFlags(s, cudaStreamNonBlocking);
            if (e != cudaSuccess) return cuda_fail(e, "cudaStreamCreateWithFlags");
        }
        cudaEvent_t* events[8] = {&P.entry, &P.done, &P.loaded[0], &P.loaded[1],
                                  &P.computed[0], &P.computed[1], &P.freed[0], &P.freed[1]};
        for (cudaEvent_t* ev : events) {
            if (*ev) continue;
            e = cudaEventCreateWithFlags(ev, cudaEventDisableTiming);
            if (e != cudaSuccess) return cuda_fail(e, "cudaEventCreateWithFlags");
        }
        P.ready = true;
    }
    *out = &P;
    return ATTN_OK;
}

// Staging layout of one slot: the chunk's inputs, outputs and the scratch
// its compute step uses, each part 256-byte aligned.  Part sizes are given
// per sequence; the batch dimension is outermost in every host tensor.
struct Staging {
    long long cb = 0;                  // sequences per chunk
    int n_in = 0, n_out = 0;
    size_t in_seq[6] = {}, out_seq[3] = {};
    size_t in_off[6] = {}, out_off[3] = {}, scratch_off = 0, slot = 0;
};

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

bool staging(int B, const size_t* in_seq, int n_in, const size_t* out_seq, int n_out, const size_t* scratch_seq,
             int n_scratch, Staging* L) {
    if (B <= 0) return false;
    const long long nch = B < kHostChunks ? B : kHostChunks;
    L->cb = (B + nch - 1) / nch;
    const size_t cb = static_cast<size_t>(L->cb);
    L->n_in = n_in;
    L->n_out = n_out;
    size_t off = 0;
    for (int x = 0; x < n_in; ++x) { L->in_seq[x] = in_seq[x]; L->in_off[x] = off; off += up256(cb * in_seq[x]); }
    for (int x = 0; x < n_out; ++x) { L->out_seq[x] = out_seq[x]; L->out_off[x] = off; off += up256(cb * out_seq[x]); }
    L->scratch_off = off;
    for (int x = 0; x < n_scratch; ++x) off += up256(cb * scratch_seq[x]);
    L->slot = off;
    return true;
}

// The forward's parts: Q, K, V in; O, LSE out.
bool fwd_staging(int B, int H, int H_kv, int N, int d, const size_t* scratch_seq, int n_scratch, Staging* L) {
    if (H <= 0 || H_kv <= 0 || N <= 0 || d <= 0) return false;
    const size_t q_seq = static_cast<size_t>(N) * H * d * 2, kv_seq = static_cast<size_t>(N) * H_kv * d * 2;
    const size_t in[3] = {q_seq, kv_seq, kv_seq}, out[2] = {q_seq, static_cast<size_t>(H) * N * 4};
    return staging(B, in, 3, out, 2, scratch_seq, n_scratch, L);
}

// Runs the chunks of one call through the staging slots (see above).
// compute(nb, slot_base, stream) queues the chunk's work on `stream`.
template <class Compute>
int host_pipeline(const void* const* in, void* const* out, int B, const Staging& L, void* workspace,
                  size_t workspace_bytes, void* stream, const char* who, Compute&& compute) {
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || workspace_bytes < 2 * L.slot)
        return fail(ATTN_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned and at least %zu bytes (got %zu)",
                    who, 2 * L.slot, workspace_bytes);
    std::lock_guard<std::mutex> lock(g_pipe_mutex);
    HostPipe* P = nullptr;
    int rc = host_pipe(&P);
    if (rc != ATTN_OK) return rc;
    const cudaStream_t user = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaEventRecord(P->entry, user);
    if (e == cudaSuccess) e = cudaStreamWaitEvent(P->h2d, P->entry, 0);
    if (e != cudaSuccess) return cuda_fail(e, "host pipeline: ordering after the caller's stream");
    // A call with another staging layout (workspace or slot size) than the
    // previous one waits until both slots of the previous one are free: its
    // slots need not coincide with the old ones.
    if (P->last_ws != workspace || P->last_slot != L.slot) {
        for (int s = 0; s < 2 && e == cudaSuccess; ++s) e = cudaStreamWaitEvent(P->h2d, P->freed[s], 0);
        if (e != cudaSuccess) return cuda_fail(e, "host pipeline: ordering after the previous staging");
        P->last_ws = workspace;
        P->last_slot = L.slot;
    }
    for (long long b0 = 0; b0 < B && rc == ATTN_OK; b0 += L.cb) {
        const long long nb = B - b0 < L.cb ? B - b0 : L.cb;
        const int slot = static_cast<int>(P->chunks & 1);
        ++P->chunks;
        char* base = static_cast<char*>(workspace) + slot * L.slot;
        e = cudaStreamWaitEvent(P->h2d, P->freed[slot], 0);
        for (int x = 0; x < L.n_in && e == cudaSuccess; ++x)
            e = cudaMemcpyAsync(base + L.in_off[x], static_cast<const char*>(in[x]) + b0 * L.in_seq[x],
                                nb * L.in_seq[x], cudaMemcpyHostToDevice, P->h2d);
        if (e == cudaSuccess) e = cudaEventRecord(P->loaded[slot], P->h2d);
        if (e == cudaSuccess) e = cudaStreamWaitEvent(P->comp, P->loaded[slot], 0);
        if (e != cudaSuccess) {
            rc = cuda_fail(e, "host pipeline: host-to-device copy");
            break;
        }
        rc = compute(static_cast<int>(nb), base, P->comp);
        if (rc != ATTN_OK) break;
        e = cudaEventRecord(P->computed[slot], P->comp);
        if (e == cudaSuccess) e = cudaStreamWaitEvent(P->d2h, P->computed[slot], 0);
        for (int x = 0; x < L.n_out && e == cudaSuccess; ++x)
            e = cudaMemcpyAsync(static_cast<char*>(out[x]) + b0 * L.out_seq[x], base + L.out_off[x],
                                nb * L.out_seq[x], cudaMemcpyDeviceToHost, P->d2h);
        if (e == cudaSuccess) e = cudaEventRecord(P->freed[slot], P->d2h);
        if (e != cudaSuccess) rc = cuda_fail(e, "host pipeline: device-to-host copy");
    }
    // The caller's stream resumes after everything queued above.
    e = cudaEventRecord(P->done, P->d2h);
    if (e == cudaSuccess) e = cudaStreamWaitEvent(user, P->done, 0);
    if (e != cudaSuccess && rc == ATTN_OK) rc = cuda_fail(e, "host pipeline: ordering the caller's stream");
    return rc;
}

// Scratch of the FP8 host forward per sequence: Q8, K8, V8 codes and the
// three block-scale arrays.
void fp8_scratch(int H, int H_kv, int N, int d, size_t s[6]) {
    const size_t nblk = (static_cast<size_t>(N) + 127) / 128;
    s[0] = static_cast<size_t>(N) * H * d;
    s[1] = s[2] = static_cast<size_t>(N) * H_kv * d;
    s[3] = static_cast<size_t>(H) * nblk * 4;
    s[4] = s[5] = static_cast<size_t>(H_kv) * nblk * 4;
}

}  // namespace

extern "C" {

size_t attn_fwd_host_workspace_size(int B, int H, int H_kv, int N, int d) {
    Staging L;
    if (!fwd_staging(B, H, H_kv, N, d, nullptr, 0, &L)) return 0;
    return 2 * L.slot;
}

int attn_fwd_host(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int H_kv, int N,
                  int d, int causal, float scale, int window, void* workspace, size_t workspace_bytes,
                  void* stream) {
    g_err[0] = '\0';
    int rc = check_common(q, k, v, o, lse, B, H, N, d, window);
    if (rc != ATTN_OK) return rc;
    if (H_kv <= 0 || H % H_kv != 0)
        return fail(ATTN_ERR_INVALID_ARG, "key/value heads (%d) must divide query heads (%d)", H_kv, H);
    if (static_cast<long long>(B) * H * N == 0) return ATTN_OK;
    Staging L;
    fwd_staging(B, H, H_kv, N, d, nullptr, 0, &L);
    const void* in[3] = {q, k, v};
    void* out[2] = {o, lse};
    return host_pipeline(in, out, B, L, workspace, workspace_bytes, stream, "attn_fwd_host",
                         [&](int nb, char* base, cudaStream_t s) {
                             return launch_forward(false, base + L.in_off[0], base + L.in_off[1], base + L.in_off[2],
                                                   base + L.out_off[0], reinterpret_cast<float*>(base + L.out_off[1]),
                                                   nb, H, H_kv, N, d, causal, scale, window, nullptr, nullptr,
                                                   nullptr, s);
                         });
}

size_t attn_fwd_fp8_host_workspace_size(int B, int H, int H_kv, int N, int d) {
    Staging L;
    size_t sc[6];
    if (H <= 0 || H_kv <= 0 || N <= 0 || d <= 0) return 0;
    fp8_scratch(H, H_kv, N, d, sc);
    if (!fwd_staging(B, H, H_kv, N, d, sc, 6, &L)) return 0;
    return 2 * L.slot;
}

int attn_fwd_fp8_host(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int H_kv,
                      int N, int d, int causal, float scale, int window, int mode, unsigned long long sign_seed,
                      void* workspace, size_t workspace_bytes, void* stream) {
    g_err[0] = '\0';
    int rc = check_common(q, k, v, o, lse, B, H, N, d, window);
    if (rc != ATTN_OK) return rc;
    if (H_kv <= 0 || H % H_kv != 0)
        return fail(ATTN_ERR_INVALID_ARG, "key/value heads (%d) must divide query heads (%d)", H_kv, H);
    if (mode != 0 && mode != 1)
        return fail(ATTN_ERR_INVALID_ARG, "attn_fwd_fp8_host: mode %d (0 or 1; the per-tensor mode spans chunks)",
                    mode);
    if (static_cast<long long>(B) * H * N == 0) return ATTN_OK;
    Staging L;
    size_t sc[6];
    fp8_scratch(H, H_kv, N, d, sc);
    fwd_staging(B, H, H_kv, N, d, sc, 6, &L);
    size_t soff[6];
    for (int x = 0; x < 6; ++x)
        soff[x] = x == 0 ? L.scratch_off : soff[x - 1] + up256(static_cast<size_t>(L.cb) * sc[x - 1]);
    const void* in[3] = {q, k, v};
    void* out[2] = {o, lse};
    return host_pipeline(in, out, B, L, workspace, workspace_bytes, stream, "attn_fwd_fp8_host",
                         [&](int nb, char* base, cudaStream_t s) {
                             float* qs = reinterpret_cast<float*>(base + soff[3]);
                             float* ks = reinterpret_cast<float*>(base + soff[4]);
                             float* vs = reinterpret_cast<float*>(base + soff[5]);
                             int r = attn_fp8_prep_qkv(base + L.in_off[0], base + L.in_off[1], base + L.in_off[2],
                                                       base + soff[0], base + soff[1], base + soff[2], qs, ks, vs, nb,
                                                       H, H_kv, N, d, mode, sign_seed, s);
                             if (r != ATTN_OK) return r;
                             return launch_forward(true, base + soff[0], base + soff[1], base + soff[2],
                                                   base + L.out_off[0], reinterpret_cast<float*>(base + L.out_off[1]),
                                                   nb, H, H_kv, N, d, causal, scale, window, qs, ks, vs, s);
                         });
}

}  // extern "C"

namespace {

// The backward's parts: Q, K, V, O, LSE, dO in; dQ, dK, dV out; the
// backward's own workspace for one chunk as scratch.
bool bwd_staging(int B, int H, int H_kv, int N, int d, Staging* L) {
    if (B <= 0 || H <= 0 || H_kv <= 0 || N <= 0 || d <= 0) return false;
    const size_t q_seq = static_cast<size_t>(N) * H * d * 2, kv_seq = static_cast<size_t>(N) * H_kv * d * 2;
    const size_t l_seq = static_cast<size_t>(H) * N * 4;
    const size_t in[6] = {q_seq, kv_seq, kv_seq, q_seq, l_seq, q_seq}, out[3] = {q_seq, kv_seq, kv_seq};
    if (!staging(B, in, 6, out, 3, nullptr, 0, L)) return false;
    // one chunk's backward workspace (not a per-sequence size: added whole)
    L->slot += up256(static_cast<size_t>(attn::bwd_workspace(static_cast<int>(L->cb), H, N, d).bytes));
    return true;
}

}  // namespace

extern "C" {

size_t attn_bwd_host_workspace_size(int B, int H, int H_kv, int N, int d) {
    Staging L;
    if (!bwd_staging(B, H, H_kv, N, d, &L)) return 0;
    return 2 * L.slot;
}

int attn_bwd_host(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dout,
                  void* dq, void* dk, void* dv, int B, int H, int H_kv, int N, int d, int causal, float scale,
                  int window, void* workspace, size_t workspace_bytes, void* stream) {
    g_err[0] = '\0';
    int rc = check_common(q, k, v, o, lse, B, H, N, d, window);
    if (rc != ATTN_OK) return rc;
    if (d != 128 && d != 64) return fail(ATTN_ERR_UNSUPPORTED, "attn_bwd_host supports head_dim 64 and 128 (got %d)", d);
    if (H_kv <= 0 || H % H_kv != 0)
        return fail(ATTN_ERR_INVALID_ARG, "key/value heads (%d) must divide query heads (%d)", H_kv, H);
    if (static_cast<long long>(B) * H * N == 0) return ATTN_OK;
    if (!dout || !dq || !dk || !dv) return fail(ATTN_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(dout) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv))
        return fail(ATTN_ERR_INVALID_ARG, "pointers must be 16-byte aligned");
    Staging L;
    bwd_staging(B, H, H_kv, N, d, &L);
    const size_t bwd_ws = up256(static_cast<size_t>(attn::bwd_workspace(static_cast<int>(L.cb), H, N, d).bytes));
    const void* in[6] = {q, k, v, o, lse, dout};
    void* out[3] = {dq, dk, dv};
    return host_pipeline(in, out, B, L, workspace, workspace_bytes, stream, "attn_bwd_host",
                         [&](int nb, char* base, cudaStream_t s) {
                             return attn_bwd(base + L.in_off[0], base + L.in_off[1], base + L.in_off[2],
                                             base + L.in_off[3], reinterpret_cast<const float*>(base + L.in_off[4]),
                                             base + L.in_off[5], base + L.out_off[0], base + L.out_off[1],
                                             base + L.out_off[2], base + L.scratch_off, bwd_ws, nb, H, H_kv, N, d,
                                             causal, scale, window, s);
                         });
}

}  // extern "C"

// ---------------------------------------------------------------------------
// The paged key/value cache (see include/attn.h).

namespace {

// Sizes and pointers of the cache that every entry shares.
int check_cache(const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale, int H_kv, int d,
                int num_pages, int page_size, int cache_dtype) {
    if (d != 64 && d != 128 && d != 256) return fail(ATTN_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128, 256)", d);
    if (cache_dtype != ATTN_CACHE_BF16 && cache_dtype != ATTN_CACHE_E4M3)
        return fail(ATTN_ERR_INVALID_ARG, "cache_dtype %d (ATTN_CACHE_BF16 or ATTN_CACHE_E4M3)", cache_dtype);
    if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)) != 0)
        return fail(ATTN_ERR_UNSUPPORTED, "page_size %d (supported: 16, 32, 64, 128, 256)", page_size);
    if (H_kv <= 0) return fail(ATTN_ERR_INVALID_ARG, "key/value heads %d", H_kv);
    if (num_pages < 0) return fail(ATTN_ERR_INVALID_ARG, "negative size (num_pages=%d)", num_pages);
    if (num_pages > 0) {
        if (!k_cache || !v_cache) return fail(ATTN_ERR_INVALID_ARG, "null pointer");
        if (cache_dtype == ATTN_CACHE_E4M3 && (!k_scale || !v_scale))
            return fail(ATTN_ERR_INVALID_ARG, "null scale pointer (an e4m3 cache has a scale per row)");
    }
    if (!aligned16(k_cache) || !aligned16(v_cache) ||
        (cache_dtype == ATTN_CACHE_E4M3 && (!aligned16(k_scale) || !aligned16(v_scale))))
        return fail(ATTN_ERR_INVALID_ARG, "pointers must be 16-byte aligned");
    return ATTN_OK;
}

// K and V of the cache as {d, page_size, H_kv, num_pages}: a box of `rows` rows of
// up to 128 bytes of one head of one page, swizzled.
int make_cache_maps(attn::PagedMaps* maps, const void* k, const void* v, int num_pages, int H_kv, int page_size, int d,
                    int elem_bytes, int rows) {
    if (num_pages == 0) return ATTN_OK;      // every page is refused: no copy is made
    auto enc = encode_fn();
    if (!enc) return fail(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    const int span = d * elem_bytes < 128 ? 64 : 128;
    const cuuint64_t row = static_cast<cuuint64_t>(d) * elem_bytes, head = row * page_size;
    cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(page_size),
                          static_cast<cuuint64_t>(H_kv), static_cast<cuuint64_t>(num_pages)};
    cuuint64_t strides[3] = {row, head, head * static_cast<cuuint64_t>(H_kv)};
    cuuint32_t box[4] = {static_cast<cuuint32_t>(span / elem_bytes), static_cast<cuuint32_t>(rows), 1, 1};
    cuuint32_t estride[4] = {1, 1, 1, 1};
    for (int x = 0; x < 2; ++x) {
        CUresult r = enc(x ? &maps->v : &maps->k,
                         elem_bytes == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 4,
                         const_cast<void*>(x ? v : k), dims, strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         span == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        if (r != CUDA_SUCCESS)
            return fail(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled (cache) failed (CUresult %d)", static_cast<int>(r));
    }
    return ATTN_OK;
}

int log2_of(int page_size) {
    int s = 0;
    while ((1 << s) < page_size) ++s;
    return s;
}

// A sequence's keys are counted in int with headroom for rounding up.
constexpr long long kMaxKeys = 1ll << 30;

int check_table(const int* table, long long table_stride, int max_pages, int page_size, const int* seq_lens) {
    if (max_pages < 0) return fail(ATTN_ERR_INVALID_ARG, "negative size (max_pages=%d)", max_pages);
    if (!seq_lens || (max_pages > 0 && !table)) return fail(ATTN_ERR_INVALID_ARG, "null pointer");
    if (table_stride < max_pages)
        return fail(ATTN_ERR_INVALID_ARG, "table_stride %lld < max_pages %d", table_stride, max_pages);
    if (static_cast<long long>(max_pages) * page_size > kMaxKeys)
        return fail(ATTN_ERR_INVALID_ARG, "a page table of more than 2^30 tokens");
    if ((reinterpret_cast<uintptr_t>(table) & 3u) != 0 || (reinterpret_cast<uintptr_t>(seq_lens) & 3u) != 0)
        return fail(ATTN_ERR_INVALID_ARG, "page tables and lengths must be 4-byte aligned");
    return ATTN_OK;
}

// Sizes of an attention call, and its plan (empty problems: as it is).
int check_paged_sizes(int B, int Nq, int H, int H_kv, int d, int prefix_len, int max_pages, int page_size,
                      attn::PagedPlan* plan, bool tree = false) {
    if (B < 0 || Nq < 0 || H < 0 || prefix_len < 0 || max_pages < 0)
        return fail(ATTN_ERR_INVALID_ARG, "negative size (B=%d Nq=%d H=%d prefix_len=%d max_pages=%d)", B, Nq, H,
                    prefix_len, max_pages);
    if (H_kv <= 0 || H % H_kv != 0)
        return fail(ATTN_ERR_INVALID_ARG, "key/value heads (%d) must divide query heads (%d)", H_kv, H);
    if (d != 64 && d != 128 && d != 256) return fail(ATTN_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128, 256)", d);
    if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)) != 0)
        return fail(ATTN_ERR_UNSUPPORTED, "page_size %d (supported: 16, 32, 64, 128, 256)", page_size);
    if (prefix_len > kMaxKeys || static_cast<long long>(max_pages) * page_size > kMaxKeys)
        return fail(ATTN_ERR_INVALID_ARG, "more than 2^30 tokens in a prefix or a page table");
    // Row indices are ints with headroom for the last tile.  CTAs are counted in
    // long long by the plan: their indices are ints too.
    if (static_cast<long long>(B) * Nq > (1ll << 30) || static_cast<long long>(B) * Nq * std::max(H, 1) > (1ll << 30))
        return fail(ATTN_ERR_INVALID_ARG, "problem too large for one launch");
    if (static_cast<long long>(B) * Nq * H > 0) *plan = attn::paged_plan(B, Nq, H, H_kv, d, prefix_len, max_pages, page_size, tree);
    if (plan->blocks > 0x7fffffffll) return fail(ATTN_ERR_INVALID_ARG, "problem too large for one launch");
    return ATTN_OK;
}

// The size that a tree's call adds.
int check_tree(int Nq) {
    if (Nq > attn::kMaxTree) return fail(ATTN_ERR_UNSUPPORTED, "a tree of %d nodes (at most %d)", Nq, attn::kMaxTree);
    return ATTN_OK;
}

// attn_fwd_paged, and attn_fwd_paged_tree where `name` is that (parents: its trees).
int paged_call(const char* name, bool tree, const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
               const float* v_scale, const int* prefix_table, int prefix_len, const int* block_table,
               long long table_stride, int max_pages, const int* seq_lens, const int* parents, long long parents_stride,
               void* o, float* lse, int B, int Nq, int H, int H_kv, int d, int num_pages, int page_size,
               int cache_dtype, int causal, float scale, void* workspace, size_t workspace_bytes, void* stream) {
    g_err[0] = '\0';
    int rc = check_cache(k_cache, v_cache, k_scale, v_scale, H_kv, d, num_pages, page_size, cache_dtype);
    if (rc != ATTN_OK) return rc;
    attn::PagedPlan plan;
    if ((rc = check_paged_sizes(B, Nq, H, H_kv, d, prefix_len, max_pages, page_size, &plan, tree)) != ATTN_OK) return rc;
    if (tree && (rc = check_tree(Nq)) != ATTN_OK) return rc;
    if (static_cast<long long>(B) * Nq * H == 0) return ATTN_OK;
    if ((rc = check_table(block_table, table_stride, max_pages, page_size, seq_lens)) != ATTN_OK) return rc;
    if (!q || !o || !lse || (prefix_len > 0 && !prefix_table)) return fail(ATTN_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(q) || !aligned16(o) || !aligned16(lse))
        return fail(ATTN_ERR_INVALID_ARG, "pointers must be 16-byte aligned");
    if ((reinterpret_cast<uintptr_t>(prefix_table) & 3u) != 0)
        return fail(ATTN_ERR_INVALID_ARG, "page tables and lengths must be 4-byte aligned");
    if (tree) {
        if (!parents) return fail(ATTN_ERR_INVALID_ARG, "null pointer");
        if ((reinterpret_cast<uintptr_t>(parents) & 3u) != 0)
            return fail(ATTN_ERR_INVALID_ARG, "parents must be 4-byte aligned");
        if (parents_stride != 0 && parents_stride < Nq)
            return fail(ATTN_ERR_INVALID_ARG, "parents_stride %lld (0, or at least Nq = %d)", parents_stride, Nq);
    }
    if (plan.bytes > 0) {
        if (!workspace) return fail(ATTN_ERR_INVALID_ARG, "null pointer");
        if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
            return fail(ATTN_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
        if (workspace_bytes < plan.bytes)
            return fail(ATTN_ERR_INVALID_ARG, "workspace of %zu bytes is smaller than the %zu bytes needed",
                        workspace_bytes, plan.bytes);
    }
    attn::PagedParams p{};
    p.q = q;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.prefix_table = prefix_table;
    p.table = block_table;
    p.table_stride = table_stride;
    p.seq_lens = seq_lens;
    p.o = o;
    p.lse = lse;
    p.part_o = static_cast<float*>(workspace);
    p.part_lse = reinterpret_cast<float*>(static_cast<char*>(workspace) + plan.part_o_bytes);
    p.B = B;
    p.Nq = Nq;
    p.H = H;
    p.H_kv = H_kv;
    p.G = H / H_kv;
    p.d = d;
    p.num_pages = num_pages;
    p.page_shift = log2_of(page_size);
    p.max_pages = max_pages;
    p.prefix_len = prefix_len;
    p.causal = causal ? 1 : 0;
    p.prefix_parts = plan.prefix_parts;
    p.own_parts = plan.own_parts;
    p.prefix_items = plan.prefix_items;
    p.prefix_ctas = plan.prefix_ctas;
    p.own_items = plan.own_items;
    p.own_ctas = plan.own_ctas;
    p.stream_tile = plan.stream_tile;
    p.parents = parents;
    p.parents_stride = parents_stride;
    // (CTAs replace one another as they finish.  It takes a CTA 0.4 us to find its sequence: 33
    // drafts x 24 sequences of up to 256, 512 and 1024 tokens, d = 128, bf16, in their order |
    // the longest first, lengths from all to half 24.4 | 26.1, 30.0 | 30.4, 41.3 | 36.3; from all
    // to 33 25.3 | 23.2, 28.4 | 26.0, 36.5 | 32.0.  More than 64 stay in their order: with four
    // keys a lane 128 sequences of up to 1024 took 146 | 147 and 123 | 125.)
    p.longest_first = tree && B > 1 && B <= 64 && (static_cast<long long>(max_pages) << p.page_shift) >= 512 &&
                      plan.prefix_items + plan.own_items > attn::kPlanSms;
    attn::paged_divisors(p);
    p.scale_log2 = resolve_scale(scale, d) * 1.4426950408889634f;
    p.fp8 = cache_dtype == ATTN_CACHE_E4M3;
    p.wait_limit = g_wait_limit.load();
    if ((rc = status_ptr(&p.status)) != ATTN_OK) return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const auto pick = [&](auto d64, auto d128, auto d256) { return d == 64 ? d64 : d == 128 ? d128 : d256; };
    const auto rows = tree ? pick(attn::run_paged_stream_tree_d64, attn::run_paged_stream_tree_d128, attn::run_paged_stream_tree_d256)
                           : pick(attn::run_paged_stream_d64, attn::run_paged_stream_d128, attn::run_paged_stream_d256);
    const auto tiles = tree ? pick(attn::run_paged_tile_tree_d64, attn::run_paged_tile_tree_d128, attn::run_paged_tile_tree_d256)
                            : pick(attn::run_paged_tile_d64, attn::run_paged_tile_d128, attn::run_paged_tile_d256);
    cudaError_t e = cudaSuccess;
    attn::PagedMaps maps{};
    const int es = p.fp8 ? 1 : 2;
    if (plan.prefix_items + plan.own_items > 0) {
        const int bn = d == 256 ? 64 : 128;
        if ((rc = make_cache_maps(&maps, k_cache, v_cache, num_pages, H_kv, page_size, d, es,
                                  page_size < bn ? page_size : bn)) != ATTN_OK)
            return rc;
        e = tiles(maps, p, plan.direct, s);
    }
    if (e == cudaSuccess && (plan.prefix_stream || plan.own_items == 0)) {
        if ((rc = make_cache_maps(&maps, k_cache, v_cache, num_pages, H_kv, page_size, d, es, 16)) != ATTN_OK) return rc;
        e = rows(maps, p, plan.prefix_stream, plan.own_items == 0, plan.direct, plan.prefix_items + plan.own_items > 0, s);
    }
    if (e == cudaSuccess && !plan.direct) e = attn::run_paged_merge(p, s);
    if (e != cudaSuccess) return cuda_fail(e, name);
    return ATTN_OK;
}

// The plan of a call, as attn_fwd_paged_plan gives it (0: refused or empty).
int paged_plan_out(int B, int Nq, int H, int H_kv, int d, int prefix_len, int max_pages, int page_size, bool tree, int* out,
                   int capacity) {
    if (!out || capacity < 8) return 0;
    attn::PagedPlan plan;
    if (check_paged_sizes(B, Nq, H, H_kv, d, prefix_len, max_pages, page_size, &plan, tree) != ATTN_OK) return 0;
    if (tree && check_tree(Nq) != ATTN_OK) return 0;
    if (static_cast<long long>(B) * Nq * H == 0) return 0;
    const long long rows = static_cast<long long>(Nq) * (H / H_kv);
    out[0] = plan.prefix_items > 0 ? 2 : plan.prefix_stream ? 1 : 0;
    out[1] = plan.own_items > 0 ? 2 : 1;
    out[2] = plan.prefix_parts;
    out[3] = plan.own_parts;
    out[4] = out[0] == 1 || out[1] == 1 ? plan.stream_tile : 0;
    out[5] = out[0] == 2 ? static_cast<int>((B * rows + 127) / 128) : 0;
    out[6] = out[1] == 2 ? static_cast<int>((rows + 127) / 128) : 0;
    out[7] = plan.direct ? 1 : 0;
    return 8;
}

// What attn_rope and attn_kv_append share: sizes, tables, positions.
int check_rope(attn::RopeParams* p, int T, int H, int H_kv, int d, const long long* positions, long long axis_stride,
               int n_axes, const unsigned char* pair_axis, const float* rope_cos, const float* rope_sin,
               long long table_rows, int rot, int interleaved) {
    if (T < 0 || H < 0 || H_kv < 0) return fail(ATTN_ERR_INVALID_ARG, "negative size (T=%d H=%d H_kv=%d)", T, H, H_kv);
    if (d != 64 && d != 128 && d != 256) return fail(ATTN_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128, 256)", d);
    if (rot < 16 || rot > d || rot % 16 != 0)
        return fail(ATTN_ERR_UNSUPPORTED, "%d rotary elements of %d (supported: multiples of 16 from 16 on)", rot, d);
    if (n_axes < 1 || n_axes > 4) return fail(ATTN_ERR_UNSUPPORTED, "%d axes (supported: 1 to 4)", n_axes);
    if (table_rows < 0) return fail(ATTN_ERR_INVALID_ARG, "negative size (table_rows=%lld)", table_rows);
    if (n_axes > 1 && !pair_axis) return fail(ATTN_ERR_INVALID_ARG, "null pair_axis (%d axes)", n_axes);
    for (int i = 0; pair_axis && i < rot / 2; ++i) {
        const int a = pair_axis[i];
        if (a >= n_axes) return fail(ATTN_ERR_INVALID_ARG, "pair %d turns by axis %d of %d", i, a, n_axes);
        p->axes[i >> 4] |= static_cast<uint32_t>(a) << (2 * (i & 15));
    }
    if (static_cast<long long>(T) * (static_cast<long long>(H) + H_kv) > (1ll << 30))
        return fail(ATTN_ERR_INVALID_ARG, "problem too large for one launch");
    if (T == 0) return ATTN_OK;
    if (!rope_cos || !rope_sin) return fail(ATTN_ERR_INVALID_ARG, "null rope table");
    if (!aligned16(rope_cos) || !aligned16(rope_sin)) return fail(ATTN_ERR_INVALID_ARG, "rope tables must be 16-byte aligned");
    if ((reinterpret_cast<uintptr_t>(positions) & 7u) != 0)
        return fail(ATTN_ERR_INVALID_ARG, "positions must be 8-byte aligned");
    p->positions = positions;
    p->axis_stride = axis_stride;
    p->cos = rope_cos;
    p->sin = rope_sin;
    p->rows = table_rows;
    p->T = T;
    p->d = d;
    p->rot = rot;
    p->n_axes = n_axes;
    p->interleaved = interleaved != 0;
    p->by_period = attn::FastDiv(1);
    return ATTN_OK;
}

// Rows of T tokens: `row` elements each, `stride` elements apart.
struct Rows {
    const void* at;
    long long stride, row;
};

// Whether written rows `out` meet rows `other` (columns of one buffer do not).
bool rows_meet(const Rows& out, const Rows& other, int T) {
    if (out.row == 0 || other.row == 0) return false;
    const long long a = static_cast<long long>(reinterpret_cast<uintptr_t>(out.at)), b = static_cast<long long>(reinterpret_cast<uintptr_t>(other.at));
    const long long a1 = a + 2 * ((T - 1) * out.stride + out.row), b1 = b + 2 * ((T - 1) * other.stride + other.row);
    if (a >= b1 || b >= a1) return false;
    if (T == 1 || out.stride != other.stride) return true;
    const long long s = 2 * out.stride, off = ((b - a) % s + s) % s;
    return off < 2 * out.row || s - off < 2 * other.row;
}

// q or k and its output: pointers, strides, and that they are the same rows or apart.
int check_rows(const char* what, const Rows& in, const Rows& out, int T) {
    if (in.row == 0) return ATTN_OK;
    if (!in.at || !out.at) return fail(ATTN_ERR_INVALID_ARG, "null pointer (%s)", what);
    if (!aligned16(in.at) || !aligned16(out.at)) return fail(ATTN_ERR_INVALID_ARG, "pointers must be 16-byte aligned");
    if (in.stride % 8 != 0 || out.stride % 8 != 0)
        return fail(ATTN_ERR_INVALID_ARG, "token strides (%lld, %lld elements) must be multiples of 8", in.stride, out.stride);
    if (in.stride < 0) return fail(ATTN_ERR_INVALID_ARG, "negative token stride (%lld)", in.stride);
    if (T > 1 && out.stride < out.row)
        return fail(ATTN_ERR_INVALID_ARG, "output rows of %s overlap (stride %lld < %lld)", what, out.stride, out.row);
    if (in.at == out.at && (T == 1 || in.stride == out.stride)) return ATTN_OK;
    if (rows_meet(out, in, T)) return fail(ATTN_ERR_INVALID_ARG, "%s's output overlaps its input and is not the same rows", what);
    return ATTN_OK;
}

}  // namespace

extern "C" {

int attn_kv_write(const void* k, const void* v, long long k_stride, long long v_stride, const long long* slots,
                  void* k_cache, void* v_cache, float* k_scale, float* v_scale, int T, int H_kv, int d, int num_pages,
                  int page_size, int cache_dtype, void* stream) {
    g_err[0] = '\0';
    if (T < 0) return fail(ATTN_ERR_INVALID_ARG, "negative size (T=%d)", T);
    int rc = check_cache(k_cache, v_cache, k_scale, v_scale, H_kv, d, num_pages, page_size, cache_dtype);
    if (rc != ATTN_OK) return rc;
    if (T == 0) return ATTN_OK;
    if (!k || !v || !slots) return fail(ATTN_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(k) || !aligned16(v)) return fail(ATTN_ERR_INVALID_ARG, "pointers must be 16-byte aligned");
    if ((reinterpret_cast<uintptr_t>(slots) & 7u) != 0)
        return fail(ATTN_ERR_INVALID_ARG, "slots must be 8-byte aligned");
    if (k_stride % 8 != 0 || v_stride % 8 != 0)
        return fail(ATTN_ERR_INVALID_ARG, "token strides (%lld, %lld elements) must be multiples of 8", k_stride,
                    v_stride);
    if (static_cast<long long>(T) * H_kv > (1ll << 30))
        return fail(ATTN_ERR_INVALID_ARG, "problem too large for one launch");
    attn::KvWriteParams p{};
    p.k = k;
    p.v = v;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.slots = slots;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.T = T;
    p.H_kv = H_kv;
    p.by_heads = attn::FastDiv(H_kv);
    p.d = d;
    p.page_shift = log2_of(page_size);
    p.num_slots = static_cast<long long>(num_pages) * page_size;
    p.fp8 = cache_dtype == ATTN_CACHE_E4M3;
    if ((rc = status_ptr(&p.status)) != ATTN_OK) return rc;
    cudaError_t e = attn::run_kv_write(p, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "attn_kv_write launch");
    return ATTN_OK;
}

int attn_kv_read(const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                 const int* block_table, long long table_stride, int max_pages, const int* seq_lens, void* k, void* v,
                 int B, int N, int H_kv, int d, int num_pages, int page_size, int cache_dtype, void* stream) {
    g_err[0] = '\0';
    if (B < 0 || N < 0) return fail(ATTN_ERR_INVALID_ARG, "negative size (B=%d N=%d)", B, N);
    int rc = check_cache(k_cache, v_cache, k_scale, v_scale, H_kv, d, num_pages, page_size, cache_dtype);
    if (rc != ATTN_OK) return rc;
    if (B == 0 || N == 0) return ATTN_OK;
    if ((rc = check_table(block_table, table_stride, max_pages, page_size, seq_lens)) != ATTN_OK) return rc;
    if (!k || !v) return fail(ATTN_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(k) || !aligned16(v)) return fail(ATTN_ERR_INVALID_ARG, "pointers must be 16-byte aligned");
    if (B > 65535 || static_cast<long long>(N) * H_kv > (1ll << 30))
        return fail(ATTN_ERR_INVALID_ARG, "problem too large for one launch");
    attn::KvReadParams p{};
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.table = block_table;
    p.table_stride = table_stride;
    p.seq_lens = seq_lens;
    p.k = k;
    p.v = v;
    p.B = B;
    p.N = N;
    p.H_kv = H_kv;
    p.by_heads = attn::FastDiv(H_kv);
    p.d = d;
    p.num_pages = num_pages;
    p.page_shift = log2_of(page_size);
    p.max_pages = max_pages;
    p.fp8 = cache_dtype == ATTN_CACHE_E4M3;
    if ((rc = status_ptr(&p.status)) != ATTN_OK) return rc;
    cudaError_t e = attn::run_kv_read(p, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "attn_kv_read launch");
    return ATTN_OK;
}

size_t attn_fwd_paged_workspace_size(int B, int Nq, int H, int H_kv, int d, int prefix_len, int max_pages,
                                     int page_size) {
    attn::PagedPlan plan;
    return check_paged_sizes(B, Nq, H, H_kv, d, prefix_len, max_pages, page_size, &plan) == ATTN_OK ? plan.bytes : 0;
}

int attn_fwd_paged_plan(int B, int Nq, int H, int H_kv, int d, int prefix_len, int max_pages, int page_size, int* out,
                        int capacity) {
    return paged_plan_out(B, Nq, H, H_kv, d, prefix_len, max_pages, page_size, false, out, capacity);
}

int attn_fwd_paged_tree_plan(int B, int Nq, int H, int H_kv, int d, int prefix_len, int max_pages, int page_size, int* out,
                             int capacity) {
    return paged_plan_out(B, Nq, H, H_kv, d, prefix_len, max_pages, page_size, true, out, capacity);
}

int attn_fwd_paged(const void* q, const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                   const int* prefix_table, int prefix_len, const int* block_table, long long table_stride,
                   int max_pages, const int* seq_lens, void* o, float* lse, int B, int Nq, int H, int H_kv, int d,
                   int num_pages, int page_size, int cache_dtype, int causal, float scale, void* workspace,
                   size_t workspace_bytes, void* stream) {
    return paged_call("attn_fwd_paged launch", false, q, k_cache, v_cache, k_scale, v_scale, prefix_table, prefix_len,
                      block_table, table_stride, max_pages, seq_lens, nullptr, 0, o, lse, B, Nq, H, H_kv, d, num_pages,
                      page_size, cache_dtype, causal, scale, workspace, workspace_bytes, stream);
}

size_t attn_fwd_paged_tree_workspace_size(int B, int Nq, int H, int H_kv, int d, int prefix_len, int max_pages,
                                          int page_size) {
    attn::PagedPlan plan;
    if (check_paged_sizes(B, Nq, H, H_kv, d, prefix_len, max_pages, page_size, &plan, true) != ATTN_OK) return 0;
    return check_tree(Nq) == ATTN_OK ? plan.bytes : 0;
}

int attn_fwd_paged_tree(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                        const float* v_scale, const int* prefix_table, int prefix_len, const int* block_table,
                        long long table_stride, int max_pages, const int* seq_lens, const int* parents,
                        long long parents_stride, void* o, float* lse, int B, int Nq, int H, int H_kv, int d,
                        int num_pages, int page_size, int cache_dtype, float scale, void* workspace,
                        size_t workspace_bytes, void* stream) {
    return paged_call("attn_fwd_paged_tree launch", true, q, k_cache, v_cache, k_scale, v_scale, prefix_table, prefix_len,
                      block_table, table_stride, max_pages, seq_lens, parents, parents_stride, o, lse, B, Nq, H, H_kv, d,
                      num_pages, page_size, cache_dtype, 0, scale, workspace, workspace_bytes, stream);
}

int attn_kv_accept(void* k_cache, void* v_cache, float* k_scale, float* v_scale, const int* block_table,
                   long long table_stride, int max_pages, const int* seq_lens, const int* accepted, int B, int Nq, int M,
                   int H_kv, int d, int num_pages, int page_size, int cache_dtype, void* stream) {
    g_err[0] = '\0';
    if (B < 0 || Nq < 0 || M < 0) return fail(ATTN_ERR_INVALID_ARG, "negative size (B=%d Nq=%d M=%d)", B, Nq, M);
    int rc = check_cache(k_cache, v_cache, k_scale, v_scale, H_kv, d, num_pages, page_size, cache_dtype);
    if (rc != ATTN_OK) return rc;
    if (M > Nq) return fail(ATTN_ERR_INVALID_ARG, "%d accepted of %d drafts", M, Nq);
    if (M > attn::kMaxAccepted) return fail(ATTN_ERR_UNSUPPORTED, "%d accepted drafts (at most %d)", M, attn::kMaxAccepted);
    if (B == 0 || M == 0) return ATTN_OK;
    if ((rc = check_table(block_table, table_stride, max_pages, page_size, seq_lens)) != ATTN_OK) return rc;
    if (!accepted) return fail(ATTN_ERR_INVALID_ARG, "null pointer");
    if ((reinterpret_cast<uintptr_t>(accepted) & 3u) != 0)
        return fail(ATTN_ERR_INVALID_ARG, "accepted must be 4-byte aligned");
    if (static_cast<long long>(B) * H_kv > (1ll << 28)) return fail(ATTN_ERR_INVALID_ARG, "problem too large for one launch");
    attn::KvAcceptParams p{};
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.table = block_table;
    p.table_stride = table_stride;
    p.seq_lens = seq_lens;
    p.accepted = accepted;
    p.B = B;
    p.Nq = Nq;
    p.M = M;
    p.H_kv = H_kv;
    p.d = d;
    p.num_pages = num_pages;
    p.page_shift = log2_of(page_size);
    p.max_pages = max_pages;
    p.fp8 = cache_dtype == ATTN_CACHE_E4M3;
    if ((rc = status_ptr(&p.status)) != ATTN_OK) return rc;
    cudaError_t e = attn::run_kv_accept(p, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "attn_kv_accept launch");
    return ATTN_OK;
}

int attn_rope(const void* q, long long q_stride, void* q_out, long long q_out_stride, const void* k, long long k_stride,
              void* k_out, long long k_out_stride, const long long* positions, long long axis_stride, int n_axes,
              const unsigned char* pair_axis, const float* rope_cos, const float* rope_sin, long long table_rows, int rot,
              int interleaved, int inverse, int T, int period, int H, int H_kv, int d, void* stream) {
    g_err[0] = '\0';
    attn::RopeParams p{};
    int rc = check_rope(&p, T, H, H_kv, d, positions, axis_stride, n_axes, pair_axis, rope_cos, rope_sin, table_rows, rot,
                        interleaved);
    if (rc != ATTN_OK) return rc;
    if (period < 0) return fail(ATTN_ERR_INVALID_ARG, "negative size (period=%d)", period);
    if (T == 0 || H + H_kv == 0) return ATTN_OK;
    if (!positions) {
        if (n_axes > 1) return fail(ATTN_ERR_INVALID_ARG, "null positions (%d axes)", n_axes);
        if (table_rows < (period > 0 && period < T ? period : T))
            return fail(ATTN_ERR_INVALID_ARG, "rope tables of %lld rows are shorter than the tokens", table_rows);
    }
    const long long qw = static_cast<long long>(H) * d, kw = static_cast<long long>(H_kv) * d;
    const Rows qi{q, q_stride, qw}, qo{q_out, q_out_stride, qw}, ki{k, k_stride, kw}, ko{k_out, k_out_stride, kw};
    if ((rc = check_rows("q", qi, qo, T)) != ATTN_OK || (rc = check_rows("k", ki, ko, T)) != ATTN_OK) return rc;
    if (rows_meet(qo, ki, T) || rows_meet(ko, qi, T) || rows_meet(qo, ko, T))
        return fail(ATTN_ERR_INVALID_ARG, "q's rows overlap k's, and are written");
    p.q = q;
    p.k = k;
    p.q_out = q_out;
    p.k_out = k_out;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.q_out_stride = q_out_stride;
    p.k_out_stride = k_out_stride;
    p.H = H;
    p.H_kv = H_kv;
    p.period = static_cast<unsigned>(period);
    if (period > 0) p.by_period = attn::FastDiv(period);
    p.inverse = inverse != 0;
    if ((rc = status_ptr(&p.status)) != ATTN_OK) return rc;
    cudaError_t e = attn::run_rope(p, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "attn_rope launch");
    return ATTN_OK;
}

int attn_kv_append(const void* q, long long q_stride, void* q_out, long long q_out_stride, const void* k, const void* v,
                   long long k_stride, long long v_stride, const long long* positions, long long axis_stride, int n_axes,
                   const unsigned char* pair_axis, const float* rope_cos, const float* rope_sin, long long table_rows,
                   int rot, int interleaved, const long long* slots, void* k_cache, void* v_cache, float* k_scale,
                   float* v_scale, int T, int H, int H_kv, int d, int num_pages, int page_size, int cache_dtype,
                   void* stream) {
    g_err[0] = '\0';
    int rc = check_cache(k_cache, v_cache, k_scale, v_scale, H_kv, d, num_pages, page_size, cache_dtype);
    if (rc != ATTN_OK) return rc;
    attn::RopeParams p{};
    rc = check_rope(&p, T, H, H_kv, d, positions, axis_stride, n_axes, pair_axis, rope_cos, rope_sin, table_rows, rot,
                    interleaved);
    if (rc != ATTN_OK) return rc;
    if (T == 0) return ATTN_OK;
    if (!k || !v || !slots || !positions) return fail(ATTN_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(k) || !aligned16(v)) return fail(ATTN_ERR_INVALID_ARG, "pointers must be 16-byte aligned");
    if ((reinterpret_cast<uintptr_t>(slots) & 7u) != 0)
        return fail(ATTN_ERR_INVALID_ARG, "slots must be 8-byte aligned");
    if (k_stride % 8 != 0 || v_stride % 8 != 0)
        return fail(ATTN_ERR_INVALID_ARG, "token strides (%lld, %lld elements) must be multiples of 8", k_stride,
                    v_stride);
    const long long qw = static_cast<long long>(H) * d, kw = static_cast<long long>(H_kv) * d;
    const Rows qo{q_out, q_out_stride, qw};
    if ((rc = check_rows("q", {q, q_stride, qw}, qo, T)) != ATTN_OK) return rc;
    if (k_stride < 0 || v_stride < 0) return fail(ATTN_ERR_INVALID_ARG, "negative token stride (%lld, %lld)", k_stride, v_stride);
    if (rows_meet(qo, {k, k_stride, kw}, T) || rows_meet(qo, {v, v_stride, kw}, T))
        return fail(ATTN_ERR_INVALID_ARG, "q's output overlaps the new keys or values");
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_out = q_out;
    p.q_stride = q_stride;
    p.q_out_stride = q_out_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.H = H;
    p.H_kv = H_kv;
    p.slots = slots;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.num_slots = static_cast<long long>(num_pages) * page_size;
    p.page_shift = log2_of(page_size);
    p.append = true;
    p.fp8 = cache_dtype == ATTN_CACHE_E4M3;
    if ((rc = status_ptr(&p.status)) != ATTN_OK) return rc;
    cudaError_t e = attn::run_rope(p, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "attn_kv_append launch");
    return ATTN_OK;
}

}  // extern "C"
