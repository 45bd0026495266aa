// Writing new tokens into the paged cache (quantised on the way for an e4m3
// cache) and reading sequences back out of it.
//
// Both are streams: a row of a token is read once and written once, so the
// bound is memory bandwidth.  A row is d / 8 lanes x 8 elements (16 bytes of
// bf16 a lane); K and V of a row go through the same thread, which keeps two
// independent loads in flight.
#include <cuda_bf16.h>

#include "fp8_prep.cuh"
#include "paged.cuh"
#include "sm103_ptx.cuh"

namespace attn {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void report(int* status, int site) { atomicCAS(status, 0, site); }

__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// The largest |x| of a row held by LANES lanes, as bf16 bits.  Unsigned
// comparison of the bits orders finite < inf < NaN, so an infinity or a NaN in
// the row is the result.
template <int LANES>
__device__ __forceinline__ uint32_t row_amax_bits(const uint4& x) {
    constexpr uint32_t kAbs = 0x7fff7fffu;
    uint32_t m = __vmaxu2(__vmaxu2(x.x & kAbs, x.y & kAbs), __vmaxu2(x.z & kAbs, x.w & kAbs));
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    return max(m & 0xffffu, m >> 16);
}

// scale = amax / 448, 1 for a row of zeros, NaN for a row with an infinity or a
// NaN (every element of it then reads back as NaN).  x / scale is rounded once
// to binary32 (div_by_scale; below 2^-100 its reciprocal would leave the
// normal range and the division instruction sequence is used) and once to
// e4m3, to nearest even, saturating at +-448.
template <int LANES>
__device__ __forceinline__ uint2 quantise_row(const uint4& x, float& scale) {
    const uint32_t bits = row_amax_bits<LANES>(x);
    const float amax = __uint_as_float(bits << 16);
    scale = bits >= 0x7f80u ? __uint_as_float(0x7fc00000u) : (bits ? __fdiv_rn(amax, 448.0f) : 1.0f);
    float v[8] = {bf16_lo(x.x), bf16_hi(x.x), bf16_lo(x.y), bf16_hi(x.y),
                  bf16_lo(x.z), bf16_hi(x.z), bf16_lo(x.w), bf16_hi(x.w)};
    if (scale < 0x1p-100f) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __fdiv_rn(v[e], scale);
    } else {
        const float inv = __frcp_rn(scale);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = div_by_scale(v[e], scale, inv);
    }
    return make_uint2(pack_e4m3x4(v[0], v[1], v[2], v[3]), pack_e4m3x4(v[4], v[5], v[6], v[7]));
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const KvWriteParams p) {
    constexpr int LANES = D / 8;
    // (32-bit indices: a 64-bit division would cost more than the row's work)
    const unsigned row = blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
    const int lane = threadIdx.x % LANES;
    const bool in = row < static_cast<unsigned>(p.T) * p.H_kv;
    const unsigned t = in ? row / p.H_kv : 0, h = in ? row % p.H_kv : 0;
    uint4 k = make_uint4(0, 0, 0, 0), v = k;
    long long slot = -1;
    if (in) {
        slot = __ldg(p.slots + t);
        k = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.k) + t * p.k_stride + h * D) + lane);
        v = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.v) + t * p.v_stride + h * D) + lane);
    }
    const bool store = slot >= 0 && slot < p.num_slots;
    if (slot >= p.num_slots) report(p.status, SITE_PAGED_SLOT);
    const long long page = slot >> p.page_shift;
    const long long at = ((page * p.H_kv + h) << p.page_shift) + (slot & ((1ll << p.page_shift) - 1));
    if constexpr (FP8) {
        // The shuffles inside need every lane; rows that are not stored take part.
        float ks, vs;
        const uint2 kc = quantise_row<LANES>(k, ks), vc = quantise_row<LANES>(v, vs);
        if (store) {
            reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.k_cache) + at * D)[lane] = kc;
            reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.v_cache) + at * D)[lane] = vc;
            if (lane == 0) {
                p.k_scale[at] = ks;
                p.v_scale[at] = vs;
            }
        }
    } else if (store) {
        reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.k_cache) + at * D)[lane] = k;
        reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.v_cache) + at * D)[lane] = v;
    }
}

// Eight codes and their row's scale -> eight bf16 (code * scale in binary32,
// rounded once).
__device__ __forceinline__ uint4 dequantise(const uint2& c, float scale) {
    uint4 r;
    uint32_t* out = &r.x;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const uint32_t x = w ? c.y : c.x;
#pragma unroll
        for (int hlf = 0; hlf < 2; ++hlf) {
            uint32_t f16;
            asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}"
                : "=r"(f16)
                : "r"(hlf ? x >> 16 : x & 0xffffu));
            const float2 f = f16x2_to_float2(f16);
            out[2 * w + hlf] = pack_bf16x2(f.x * scale, f.y * scale);
        }
    }
    return r;
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const KvReadParams p) {
    constexpr int LANES = D / 8;
    const int b = blockIdx.y;
    const unsigned row = blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
    const int lane = threadIdx.x % LANES;
    const int n = static_cast<int>(row / p.H_kv), h = static_cast<int>(row % p.H_kv);
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
    uint4 k, v;
    if constexpr (FP8) {
        const uint2 kc = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.k_cache) + at * D) + lane);
        const uint2 vc = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.v_cache) + at * D) + lane);
        k = dequantise(kc, __ldg(p.k_scale + at));
        v = dequantise(vc, __ldg(p.v_scale + at));
    } else {
        k = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.k_cache) + at * D) + lane);
        v = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.v_cache) + at * D) + lane);
    }
    reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.k) + to)[lane] = k;
    reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.v) + to)[lane] = v;
}

template <int D>
cudaError_t write_d(const KvWriteParams& p, cudaStream_t stream) {
    const long long threads = static_cast<long long>(p.T) * p.H_kv * (D / 8);
    const dim3 grid(static_cast<unsigned>((threads + kThreads - 1) / kThreads));
    if (p.fp8) kv_write_kernel<D, true><<<grid, kThreads, 0, stream>>>(p);
    else kv_write_kernel<D, false><<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <int D>
cudaError_t read_d(const KvReadParams& p, cudaStream_t stream) {
    const long long threads = static_cast<long long>(p.N) * p.H_kv * (D / 8);
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
