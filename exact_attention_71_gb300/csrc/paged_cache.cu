// Writing new tokens into the paged cache (quantised on the way for an e4m3
// cache) and reading sequences back out of it.
//
// Both are streams: a row of a token is read once and written once, so the
// bound is memory bandwidth, and the instructions have to stay below it.  A row is
// d / 16 lanes, each with eight elements of either half of the row (so that the
// lanes of a load or a store instruction are next to one another); K and V of a row
// go through the same thread, which keeps four independent loads in flight.
// Measured, e4m3, 8 heads of 128: writing 32768 tokens 31.4 us, 6.5 TB/s (97 % of
// the copy rate), reading 16 sequences of up to 8192 back 91.7 us, 6.7 TB/s (the
// copy rate; with 16 elements in a row a lane, 107 us).  A call of a few tokens is
// one launch, 2.1 us on the GPU.
#include "kv_rows.cuh"
#include "paged.cuh"

namespace attn {
namespace {

constexpr int kThreads = 256;

template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const KvWriteParams p) {
    constexpr int LANES = D / 16;
    const unsigned row = blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
    const int lane = threadIdx.x % LANES;
    const bool in = row < static_cast<unsigned>(p.T) * p.H_kv;
    const unsigned t = in ? p.by_heads.div(row) : 0, h = in ? row - t * p.H_kv : 0;
    Row16 k{}, v{};
    long long slot = -1;
    if (in) {
        slot = __ldg(p.slots + t);
        k = load_row<D>(p.k, t * p.k_stride + h * D, lane);
        v = load_row<D>(p.v, t * p.v_stride + h * D, lane);
    }
    const bool store = slot >= 0 && slot < p.num_slots;
    if (slot >= p.num_slots) report(p.status, SITE_PAGED_SLOT);
    const long long page = slot >> p.page_shift;
    const long long at = ((page * p.H_kv + h) << p.page_shift) + (slot & ((1ll << p.page_shift) - 1));
    if constexpr (FP8) {
        // The shuffles inside need every lane; rows that are not stored take part.
        float ks, vs;
        const uint4 kc = quantise_row<LANES>(k, ks), vc = quantise_row<LANES>(v, vs);
        if (store) {
            store_codes<D>(p.k_cache, at * D, lane, kc);
            store_codes<D>(p.v_cache, at * D, lane, vc);
            if (lane == 0) {
                p.k_scale[at] = ks;
                p.v_scale[at] = vs;
            }
        }
    } else if (store) {
        store_row<D>(p.k_cache, at * D, lane, k);
        store_row<D>(p.v_cache, at * D, lane, v);
    }
}

// Four codes and their row's scale -> four bf16 (code * scale in binary32,
// rounded once).
__device__ __forceinline__ uint2 dequantise4(uint32_t c, float2 scale) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(c));
    const float2 a = __fmul2_rn(f16x2_to_float2(lo), scale), b = __fmul2_rn(f16x2_to_float2(hi), scale);
    return make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(b.x, b.y));
}

__device__ __forceinline__ Row16 dequantise(const uint4& c, float scale) {
    const float2 s = make_float2(scale, scale);
    const uint2 a = dequantise4(c.x, s), b = dequantise4(c.y, s), d = dequantise4(c.z, s), e = dequantise4(c.w, s);
    return {make_uint4(a.x, a.y, b.x, b.y), make_uint4(d.x, d.y, e.x, e.y)};
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const KvReadParams p) {
    constexpr int LANES = D / 16;
    const int b = blockIdx.y;
    const unsigned row = blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
    const int lane = threadIdx.x % LANES;
    const int n = static_cast<int>(p.by_heads.div(row)), h = static_cast<int>(row - n * p.H_kv);
    int len = __ldg(p.seq_lens + b);
    const long long room = static_cast<long long>(p.max_pages) << p.page_shift;
    if (len > room) {
        report(p.status, SITE_PAGED_LENGTH);
        len = static_cast<int>(room);
    }
    if (n >= min(p.N, len)) return;
    const int page = __ldg(p.table + b * p.table_stride + (n >> p.page_shift));
    if (page < 0 || page >= p.num_pages) {
        report(p.status, SITE_PAGED_PAGE);
        return;
    }
    const long long at = ((static_cast<long long>(page) * p.H_kv + h) << p.page_shift) +
                         (n & ((1 << p.page_shift) - 1));
    const long long to = ((static_cast<long long>(b) * p.N + n) * p.H_kv + h) * D;
    Row16 k, v;
    if constexpr (FP8) {
        const uint4 kc = load_codes<D>(p.k_cache, at * D, lane), vc = load_codes<D>(p.v_cache, at * D, lane);
        k = dequantise(kc, __ldg(p.k_scale + at));
        v = dequantise(vc, __ldg(p.v_scale + at));
    } else {
        k = load_row<D>(p.k_cache, at * D, lane);
        v = load_row<D>(p.v_cache, at * D, lane);
    }
    store_row<D>(p.k, to, lane, k);
    store_row<D>(p.v, to, lane, v);
}

// The accepted drafts' rows move up behind the context.  All of a sequence's are read
// before one is written, since a row may be another's place; rows of different columns
// do not meet, so a thread takes 16 bytes (a column) of one head's K or V rows, all of
// them in registers, and nothing waits for another thread but for the indices.  More
// than kAcceptRows rows go through shared memory, one head's K or V a CTA.  ROW: bytes of
// a row.
// 32 sequences of up to 8 rows, 8 heads of 128, e4m3: 2.8 us, through shared memory 3.1; 512 of up to 5,
// 8 heads of 256, bf16: 4.7 us, through shared memory 7.9.
constexpr int kAcceptThreads = 128, kAcceptRows = 16;

// Cache rows of head 0 that accepted draft j of sequence b moves from and to (-1: it does
// not move): the first M threads; then a barrier.  A length beyond the table is not cut
// to it, as where rows are only read: the drafts would then be other tokens, rows of the
// context, and those would be overwritten.
__device__ __forceinline__ void accept_rows(const KvAcceptParams& p, int b, long long* from, long long* to) {
    const int len = max(0, __ldg(p.seq_lens + b));
    const bool beyond = len > (static_cast<long long>(p.max_pages) << p.page_shift);
    if (beyond) report(p.status, SITE_PAGED_LENGTH);
    const int start = len - p.Nq;
    for (int j = threadIdx.x; j < p.M; j += kAcceptThreads) {
        from[j] = -1;
        if (beyond) continue;
        const int node = __ldg(p.accepted + static_cast<long long>(b) * p.M + j);
        if (node < 0 || (node == j && start >= 0)) continue;       // (padding, or it stays)
        if (node >= p.Nq || start < 0) {
            report(p.status, SITE_TREE_NODE);
            continue;
        }
        const int* table = p.table + b * p.table_stride;
        const int at[2] = {start + node, start + j};
        const int page[2] = {__ldg(table + (at[0] >> p.page_shift)), __ldg(table + (at[1] >> p.page_shift))};
        if (page[0] < 0 || page[0] >= p.num_pages || page[1] < 0 || page[1] >= p.num_pages) {
            report(p.status, SITE_PAGED_PAGE);
            continue;
        }
        const int in_page = (1 << p.page_shift) - 1;
        from[j] = ((static_cast<long long>(page[0]) * p.H_kv) << p.page_shift) + (at[0] & in_page);
        to[j] = ((static_cast<long long>(page[1]) * p.H_kv) << p.page_shift) + (at[1] & in_page);
    }
    __syncthreads();
}

// R: rows of a sequence at most.
template <int ROW, int R>
__global__ void __launch_bounds__(kAcceptThreads) kv_accept_kernel(const KvAcceptParams p) {
    constexpr int CH = ROW / 16;
    __shared__ long long from[R], to[R];
    const unsigned b = p.by_blocks.div(blockIdx.x);
    accept_rows(p, b, from, to);
    const int x = (blockIdx.x - b * p.by_blocks.d) * kAcceptThreads + threadIdx.x;         // (head, K or V, column)
    const int c = x % CH, is_v = x / CH & 1, h = x / (2 * CH);
    if (h >= p.H_kv) return;
    uint8_t* cache = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache);
    float* scale = is_v ? p.v_scale : p.k_scale;
    const long long head = static_cast<long long>(h) << p.page_shift;
    uint4 rows[R];
    float scales[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
        if (j >= p.M || from[j] < 0) continue;
        rows[j] = reinterpret_cast<const uint4*>(cache + (from[j] + head) * ROW)[c];
        if (p.fp8 && c == 0) scales[j] = scale[from[j] + head];
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
        if (j >= p.M || from[j] < 0) continue;
        reinterpret_cast<uint4*>(cache + (to[j] + head) * ROW)[c] = rows[j];
        if (p.fp8 && c == 0) scale[to[j] + head] = scales[j];
    }
}

template <int ROW>
__global__ void __launch_bounds__(kAcceptThreads) kv_accept_long_kernel(const KvAcceptParams p) {
    constexpr int CH = ROW / 16;
    extern __shared__ uint4 rows[];                        // (M, CH)
    __shared__ long long from[kMaxAccepted], to[kMaxAccepted];
    __shared__ float scales[kMaxAccepted];
    const unsigned b = p.by_blocks.div(blockIdx.x);
    accept_rows(p, b, from, to);
    const int x = blockIdx.x - b * p.by_blocks.d, is_v = x & 1;            // (head, K or V)
    uint8_t* cache = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache);
    float* scale = is_v ? p.v_scale : p.k_scale;
    const long long head = static_cast<long long>(x >> 1) << p.page_shift;
    for (int y = threadIdx.x; y < p.M * CH; y += kAcceptThreads)
        if (from[y / CH] >= 0) rows[y] = reinterpret_cast<const uint4*>(cache + (from[y / CH] + head) * ROW)[y % CH];
    if (p.fp8)
        for (int j = threadIdx.x; j < p.M; j += kAcceptThreads)
            if (from[j] >= 0) scales[j] = scale[from[j] + head];
    __syncthreads();
    for (int y = threadIdx.x; y < p.M * CH; y += kAcceptThreads)
        if (from[y / CH] >= 0) reinterpret_cast<uint4*>(cache + (to[y / CH] + head) * ROW)[y % CH] = rows[y];
    if (p.fp8)
        for (int j = threadIdx.x; j < p.M; j += kAcceptThreads)
            if (from[j] >= 0) scale[to[j] + head] = scales[j];
}

template <int ROW>
cudaError_t accept_row(KvAcceptParams p, cudaStream_t stream) {
    const auto grid = [&](int blocks) {
        p.by_blocks = FastDiv(blocks);
        return static_cast<unsigned>(p.B) * blocks;
    };
    if (p.M <= kAcceptRows) {
        const unsigned n = grid((2 * p.H_kv * (ROW / 16) + kAcceptThreads - 1) / kAcceptThreads);
        if (p.M <= kAcceptRows / 2) kv_accept_kernel<ROW, kAcceptRows / 2><<<n, kAcceptThreads, 0, stream>>>(p);
        else kv_accept_kernel<ROW, kAcceptRows><<<n, kAcceptThreads, 0, stream>>>(p);
        return cudaGetLastError();
    }
    static std::atomic<unsigned long long> ready{0};
    cudaError_t e = once_per_device(ready, [] {
        return cudaFuncSetAttribute(kv_accept_long_kernel<ROW>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxAccepted * ROW);
    });
    if (e != cudaSuccess) return e;
    const unsigned n = grid(2 * p.H_kv);
    kv_accept_long_kernel<ROW><<<n, kAcceptThreads, p.M * ROW, stream>>>(p);
    return cudaGetLastError();
}

template <int D>
cudaError_t write_d(const KvWriteParams& p, cudaStream_t stream) {
    const long long threads = static_cast<long long>(p.T) * p.H_kv * (D / 16);
    const dim3 grid(static_cast<unsigned>((threads + kThreads - 1) / kThreads));
    if (p.fp8) kv_write_kernel<D, true><<<grid, kThreads, 0, stream>>>(p);
    else kv_write_kernel<D, false><<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <int D>
cudaError_t read_d(const KvReadParams& p, cudaStream_t stream) {
    const long long threads = static_cast<long long>(p.N) * p.H_kv * (D / 16);
    const dim3 grid(static_cast<unsigned>((threads + kThreads - 1) / kThreads), static_cast<unsigned>(p.B));
    if (p.fp8) kv_read_kernel<D, true><<<grid, kThreads, 0, stream>>>(p);
    else kv_read_kernel<D, false><<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t run_kv_write(const KvWriteParams& p, cudaStream_t stream) {
    return p.d == 64 ? write_d<64>(p, stream) : p.d == 128 ? write_d<128>(p, stream) : write_d<256>(p, stream);
}

cudaError_t run_kv_accept(const KvAcceptParams& p, cudaStream_t stream) {
    switch (p.d * (p.fp8 ? 1 : 2)) {
        case 64: return accept_row<64>(p, stream);
        case 128: return accept_row<128>(p, stream);
        case 256: return accept_row<256>(p, stream);
        default: return accept_row<512>(p, stream);
    }
}

cudaError_t run_kv_read(const KvReadParams& p, cudaStream_t stream) {
    return p.d == 64 ? read_d<64>(p, stream) : p.d == 128 ? read_d<128>(p, stream) : read_d<256>(p, stream);
}

}  // namespace attn
