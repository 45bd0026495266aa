// Rows of the paged cache in registers: loading, storing and quantising them.
// A row of D elements is D / 16 lanes, 16 elements each: two chunks of eight,
// which are 16 bytes of bf16 or eight bytes of codes.
#pragma once

#include <cuda_bf16.h>

#include "sm103_ptx.cuh"

namespace attn {

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

// The same for a row in binary32 (rotated keys): v[0 .. 8) and v[8 .. 16) are the
// lane's chunks.  The scale is 1 also where amax / 448 is too small for binary32.
template <int LANES>
__device__ __forceinline__ uint4 quantise_row(const float (&v)[16], float& scale) {
    uint32_t bits = 0;
#pragma unroll
    for (int e = 0; e < 16; ++e) bits = max(bits, __float_as_uint(v[e]) & 0x7fffffffu);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, o));
    scale = bits >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : __fdiv_rn(__uint_as_float(bits), 448.0f);
    if (scale == 0.0f) scale = 1.0f;
    uint32_t c[4];
    if (scale < 0x1p-100f) {
        // The reciprocal, or the residual, would leave the normal range.
#pragma unroll
        for (int y = 0; y < 4; ++y)
            c[y] = pack_e4m3x4(__fdiv_rn(v[4 * y], scale), __fdiv_rn(v[4 * y + 1], scale), __fdiv_rn(v[4 * y + 2], scale),
                               __fdiv_rn(v[4 * y + 3], scale));
        return make_uint4(c[0], c[1], c[2], c[3]);
    }
    const float inv = __frcp_rn(scale);
    const float2 n2 = make_float2(-scale, -scale), i2 = make_float2(inv, inv);
#pragma unroll
    for (int y = 0; y < 4; ++y) {
        float q[4];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            const float2 x = make_float2(v[4 * y + 2 * z], v[4 * y + 2 * z + 1]);
            const float2 q0 = __fmul2_rn(x, i2);
            const float2 r = __ffma2_rn(__ffma2_rn(q0, n2, x), i2, q0);
            q[2 * z] = r.x;
            q[2 * z + 1] = r.y;
        }
        const uint32_t s01 = __byte_perm(__float_as_uint(v[4 * y]), __float_as_uint(v[4 * y + 1]), 0x0073);
        const uint32_t s23 = __byte_perm(__float_as_uint(v[4 * y + 2]), __float_as_uint(v[4 * y + 3]), 0x7300);
        c[y] = pack_e4m3x4(q[0], q[1], q[2], q[3]) | (__byte_perm(s01, s23, 0x7610) & 0x80808080u);
    }
    return make_uint4(c[0], c[1], c[2], c[3]);
}

}  // namespace attn
