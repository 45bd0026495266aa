// The paged key/value cache: launch parameters shared by the C ABI and the
// kernels (write, read back, and the attention over a shared prefix and each
// sequence's own pages).
//
// Cache layout: K and V are (num_pages, H_kv, page_size, d), d fastest, bf16 or
// e4m3; an e4m3 cache has one float32 scale per row, (num_pages, H_kv,
// page_size).  A head's rows of a page are contiguous, so a CTA that serves one
// key/value head streams whole lines, and the scales of 16 keys share two
// sectors.  Cache row of (page, head, row) = (page * H_kv + head) * page_size +
// row: the index of its scale, and of its d elements.  Row indices and byte
// offsets are 64-bit.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <atomic>
#include <cstddef>
#include <cstdint>
#include <utility>

namespace attn {

// Device status codes of indices that a kernel refused (nothing is read or
// written through them); codes below SITE_BAD_INDEX are waits that ran out.
enum : int {
    SITE_BAD_INDEX = 0x100,
    SITE_PAGED_SLOT = 0x101,     // attn_kv_write: slot beyond the cache
    SITE_PAGED_PAGE = 0x102,     // a page index outside [0, num_pages)
    SITE_PAGED_LENGTH = 0x103,   // a sequence length beyond its table
};

// n / d for n < 2^31 by a multiplication (d from the host; Granlund and
// Montgomery): with 2^s >= d and m = floor(2^32 (2^s - d) / d) + 1, n / d = (n +
// floor(m n / 2^32)) >> s.  A CTA finds its place by half a dozen of them, one after
// the other, before its first load; the compiler's own division by a variable
// took 1800 cycles of a tile CTA there.
struct FastDiv {
    unsigned d = 1, m = 1, s = 0;
    FastDiv() = default;
    explicit FastDiv(unsigned by) : d(by) {
        while ((1ull << s) < d) ++s;
        m = static_cast<unsigned>(((1ull << 32) * ((1ull << s) - d)) / d + 1);
    }
    __device__ __forceinline__ unsigned div(unsigned n) const { return (__umulhi(n, m) + n) >> s; }
    __device__ __forceinline__ unsigned mod(unsigned n) const { return n - div(n) * d; }
};

struct KvWriteParams {
    const void* k;               // bf16 rows: token t, head h at k + t * k_stride + h * d
    const void* v;
    long long k_stride, v_stride;
    const long long* slots;      // (T,)
    void* k_cache;
    void* v_cache;
    float* k_scale;
    float* v_scale;
    int T, H_kv, d, page_shift;
    FastDiv by_heads;            // H_kv
    long long num_slots;         // num_pages * page_size
    bool fp8;
    int* status;
};

struct KvReadParams {
    const void* k_cache;
    const void* v_cache;
    const float* k_scale;
    const float* v_scale;
    const int* table;            // (B, max_pages), row stride table_stride
    long long table_stride;
    const int* seq_lens;         // (B,)
    void* k;                     // bf16 (B, N, H_kv, d)
    void* v;
    int B, N, H_kv, d, num_pages, page_shift, max_pages;
    FastDiv by_heads;            // H_kv
    bool fp8;
    int* status;
};

// The attention.  A query row is (sequence b, query token i, head h); the rows
// of one key/value head's group share its keys.  Row index in q, o and the
// partial results: (b * Nq + i) * H + h.
struct PagedParams {
    const void* q;
    const void* k_cache;
    const void* v_cache;
    const float* k_scale;
    const float* v_scale;
    const int* prefix_table;
    const int* table;
    long long table_stride;
    const int* seq_lens;
    void* o;                     // bf16 (B, Nq, H, d)
    float* lse;                  // float32 (B, H, Nq)
    float* part_o;               // float32 (parts, B * Nq * H, d): normalised per part
    float* part_lse;             // float32 (parts, B * Nq * H): log2 units, -inf where the part is empty
    int B, Nq, H, H_kv, G, d;
    int num_pages, page_shift, max_pages;
    int prefix_len;
    int causal;
    int prefix_parts, own_parts; // parts [0, prefix_parts) are the prefix's
    int prefix_items, prefix_ctas;   // tile kernel: work items of the prefix; CTAs that share a row tile's keys
    int own_items, own_ctas;         // the same for the own tokens (0: the streaming kernel has them)
    int stream_tile;             // query rows of a streaming CTA: 8 or 16
    FastDiv by_G, by_per, by_heads;              // G, Nq G, H_kv
    FastDiv by_prefix_parts, by_own_parts;
    FastDiv by_prefix_rows, by_own_rows;         // streaming CTAs that share keys
    FastDiv by_prefix_groups, by_own_groups;     // tile kernel: CTAs that share keys,
    FastDiv by_prefix_shares, by_own_shares;     // and shares of a row tile's keys
    float scale_log2;
    bool fp8;
    unsigned long long wait_limit;
    int* status;
};

// How a call is cut up (host arithmetic only).
struct PagedPlan {
    int prefix_parts = 0;        // key ranges of the prefix, each a partial result
    int own_parts = 1;           // key ranges of a sequence's own tokens
    int prefix_items = 0, prefix_ctas = 0;   // tile kernel (see PagedParams)
    int own_items = 0, own_ctas = 0;
    bool prefix_stream = false;  // the streaming kernel has the prefix
    int stream_tile = 8;         // query rows of a streaming CTA
    bool direct = false;         // one part in all: the kernel writes o and lse itself
    long long blocks = 0;        // CTAs of the larger launch (an entry refuses 2^31 or more)
    size_t part_o_bytes = 0, bytes = 0;
};

// GB300 has 152 streaming multiprocessors; plans are made for that number on
// every device, so that a workspace size does not depend on the current one.
constexpr int kPlanSms = 152;

// A sequence's own tokens are cut into ranges of at least this many keys: a
// range's partial result (d floats a row, written and read again) then stays
// small beside the keys and values that it stands for.  16 sequences of 700 tokens
// behind a prefix of 2048, d = 256, bf16: 20.7, 18.0 and 16.2 us with 64, 128 and
// 256; 4 sequences of 97 behind 512, d = 128, e4m3: 8.4, 8.5 and 9.4 us.
__host__ __device__ constexpr int own_chunk(int d) { return d == 256 ? 256 : 128; }

// Query rows of one key/value head (of one sequence; over the prefix, of all)
// up to which the streaming kernel takes them; it reads the keys once per 8 or
// 16 rows, the tile kernel once per 128.  Microseconds of the streaming | the
// tile kernel at 8, 16, 32 and 48 rows, 8 heads:
//   own tokens, 32 sequences of up to 4096
//     d = 64   bf16   38 | 57    40 | 61    61 | 61    83 | 59
//              e4m3   31 | 80    37 | 80    63 | 81    87 | 83
//     d = 128  bf16   68 | 83    71 | 89    95 | 89   130 | 86
//              e4m3   46 | 112   55 | 111   89 | 114  117 | 116
//     d = 256  bf16  131 | 161  147 | 161  270 | 162  392 | 159
//              e4m3   79 | 195  101 | 195  173 | 196  241 | 196
//   and at 8, 16, 32 and 64 rows of a prefix of 32768 tokens
//     d = 64   bf16   19 | 24    22 | 25    25 | 25    35 | 26
//              e4m3   18 | 30    21 | 31    25 | 33    37 | 34
//     d = 128  bf16   29 | 39    33 | 40    34 | 41    52 | 38
//              e4m3   22 | 44    27 | 44    33 | 48    49 | 43
//     d = 256  bf16   57 | 54    60 | 55    90 | 58   161 | 63
//              e4m3   34 | 71    39 | 71    58 | 72    98 | 73
// (A plan does not depend on the cache's type, so that a workspace fits both.)
constexpr int stream_rows(int d) { return d == 256 ? 16 : 32; }

// Key ranges of a prefix, and of a sequence's own tokens, at most.
constexpr int kMaxParts = 256;

// A streaming CTA's fixed cost, in keys.
constexpr double kStreamFixed = 300.0;

// Fills in the divisors, from the other parameters.
void paged_divisors(PagedParams& p);

PagedPlan paged_plan(int B, int Nq, int H, int H_kv, int d, int prefix_len, int max_pages, int page_size);

// Runs `set` once per device (bit per ordinal; racing threads may run it twice,
// which is harmless).
template <class F>
inline cudaError_t once_per_device(std::atomic<unsigned long long>& done, F&& set) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    if ((e = set()) != cudaSuccess) return e;
    done.fetch_or(bit, std::memory_order_release);
    return cudaSuccess;
}

// Launches `kernel`; after: it follows a kernel of the same call on this stream and
// may start before that one has ended (it calls wait_prerequisites itself where
// it needs the results).
template <class... Params, class... Args>
inline cudaError_t launch_kernel(void (*kernel)(Params...), unsigned grid, unsigned threads, unsigned smem, bool after,
                                 cudaStream_t stream, Args&&... args) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = after ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

cudaError_t run_kv_write(const KvWriteParams& p, cudaStream_t stream);
cudaError_t run_kv_read(const KvReadParams& p, cudaStream_t stream);
// K and V of the cache as 4-D {d, page_size, H_kv, num_pages} tensors.  Box of the
// streaming kernel: 16 rows of up to 128 bytes; of the tile kernel: min(page_size,
// key tile) such rows.  128-byte swizzle (64-byte rows: 64).
struct PagedMaps {
    CUtensorMap k, v;
};

// The streaming kernel over the prefix and / or the own tokens, one translation
// unit per head dim; direct: it writes o and lse itself; after: the tile kernel
// runs before it.
cudaError_t run_paged_stream_d64(const PagedMaps& m, const PagedParams& p, bool prefix, bool own, bool direct, bool after,
                                 cudaStream_t stream);
cudaError_t run_paged_stream_d128(const PagedMaps& m, const PagedParams& p, bool prefix, bool own, bool direct, bool after,
                                  cudaStream_t stream);
cudaError_t run_paged_stream_d256(const PagedMaps& m, const PagedParams& p, bool prefix, bool own, bool direct, bool after,
                                  cudaStream_t stream);
// The tile kernel over its prefix_items and own_items.
cudaError_t run_paged_tile_d64(const PagedMaps& m, const PagedParams& p, bool direct, cudaStream_t stream);
cudaError_t run_paged_tile_d128(const PagedMaps& m, const PagedParams& p, bool direct, cudaStream_t stream);
cudaError_t run_paged_tile_d256(const PagedMaps& m, const PagedParams& p, bool direct, cudaStream_t stream);
cudaError_t run_paged_merge(const PagedParams& p, cudaStream_t stream);

}  // namespace attn
