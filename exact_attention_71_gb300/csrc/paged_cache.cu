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
#include <cuda_bf16.h>

#include "paged.cuh"
#include "sm103_ptx.cuh"

namespace attn {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void report(int* status, int site) { atomicCAS(status, 0, site); }

__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

struct Row16 {
    uint4 lo, hi;                  // 16 bf16
};

template <int D>
__device__ __forceinline__ Row16 load_row(const void* base, long long at, int lane) {
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + at) + lane;
    return {__ldg(src), __ldg(src + D / 16)};
}

template <int D>
__device__ __forceinline__ void store_row(void* base, long long at, int lane, const Row16& x) {
    uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + at) + lane;
    dst[0] = x.lo;
    dst[D / 16] = x.hi;
}

template <int D>
__device__ __forceinline__ void store_codes(void* base, long long at, int lane, const uint4& c) {
    uint2* dst = reinterpret_cast<uint2*>(static_cast<uint8_t*>(base) + at) + lane;
    dst[0] = make_uint2(c.x, c.y);
    dst[D / 16] = make_uint2(c.z, c.w);
}

template <int D>
__device__ __forceinline__ uint4 load_codes(const void* base, long long at, int lane) {
    const uint2* src = reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(base) + at) + lane;
    const uint2 a = __ldg(src), b = __ldg(src + D / 16);
    return make_uint4(a.x, a.y, b.x, b.y);
}

// The largest |x| of a row held by LANES lanes, as bf16 bits.  Unsigned
// comparison of the bits orders finite < inf < NaN, so an infinity or a NaN in
// the row is the result.
template <int LANES>
__device__ __forceinline__ uint32_t row_amax_bits(const Row16& x) {
    constexpr uint32_t kAbs = 0x7fff7fffu;
    const uint32_t a = __vmaxu2(__vmaxu2(x.lo.x & kAbs, x.lo.y & kAbs), __vmaxu2(x.lo.z & kAbs, x.lo.w & kAbs));
    const uint32_t b = __vmaxu2(__vmaxu2(x.hi.x & kAbs, x.hi.y & kAbs), __vmaxu2(x.hi.z & kAbs, x.hi.w & kAbs));
    uint32_t m = __vmaxu2(a, b);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    return max(m & 0xffffu, m >> 16);
}

// Four bf16 (two words) over the scale -> four codes.  x / scale is rounded once
// to binary32: q0 + (x - q0 scale) / scale, two elements an instruction, rounds to
// the quotient that division rounds to (the FP8 prep's div_by_scale).  The sign bits are
// or-ed in at the end, so that -0 stays -0.
__device__ __forceinline__ uint32_t quantise4(uint32_t a, uint32_t b, float2 neg_scale, float2 inv) {
    float q[4];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        const uint32_t w = y ? b : a;
        const float2 x = make_float2(bf16_lo(w), bf16_hi(w));
        const float2 q0 = __fmul2_rn(x, inv);
        const float2 r = __ffma2_rn(__ffma2_rn(q0, neg_scale, x), inv, q0);
        q[2 * y] = r.x;
        q[2 * y + 1] = r.y;
    }
    return pack_e4m3x4(q[0], q[1], q[2], q[3]) | (__byte_perm(a, b, 0x7531) & 0x80808080u);
}

// scale = amax / 448, 1 for a row of zeros, NaN for a row with an infinity or a
// NaN (every element of it then reads back as NaN).  Each quotient is rounded once
// to binary32 and once to e4m3, to nearest even, saturating at +-448.
template <int LANES>
__device__ __forceinline__ uint4 quantise_row(const Row16& x, float& scale) {
    const uint32_t bits = row_amax_bits<LANES>(x);
    const float amax = __uint_as_float(bits << 16);
    scale = bits >= 0x7f80u ? __uint_as_float(0x7fc00000u) : (bits ? __fdiv_rn(amax, 448.0f) : 1.0f);
    if (scale < 0x1p-100f) {
        // The reciprocal, or the residual, would leave the normal range.
        const uint32_t w[8] = {x.lo.x, x.lo.y, x.lo.z, x.lo.w, x.hi.x, x.hi.y, x.hi.z, x.hi.w};
        uint32_t c[4];
#pragma unroll
        for (int y = 0; y < 4; ++y)
            c[y] = pack_e4m3x4(__fdiv_rn(bf16_lo(w[2 * y]), scale), __fdiv_rn(bf16_hi(w[2 * y]), scale),
                               __fdiv_rn(bf16_lo(w[2 * y + 1]), scale), __fdiv_rn(bf16_hi(w[2 * y + 1]), scale));
        return make_uint4(c[0], c[1], c[2], c[3]);
    }
    const float inv = __frcp_rn(scale);
    const float2 n2 = make_float2(-scale, -scale), i2 = make_float2(inv, inv);
    return make_uint4(quantise4(x.lo.x, x.lo.y, n2, i2), quantise4(x.lo.z, x.lo.w, n2, i2),
                      quantise4(x.hi.x, x.hi.y, n2, i2), quantise4(x.hi.z, x.hi.w, n2, i2));
}

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

cudaError_t run_kv_read(const KvReadParams& p, cudaStream_t stream) {
    return p.d == 64 ? read_d<64>(p, stream) : p.d == 128 ? read_d<128>(p, stream) : read_d<256>(p, stream);
}

}  // namespace attn
