// Rotary positions: of q and k rows in memory (attn_rope: the forward rotation, and
// its transpose for gradients), and on the way into the paged cache
// (attn_kv_append).
//
//     a' = a cos - b sin,   b' = a sin + b cos        (binary32, each product and sum
//                                                      rounded, as in the FP8 prep)
//
// for pair i of a row: elements (i, i + rot / 2) or (2i, 2i + 1) of the first
// `rot`; the table row that it turns by is the token's position on the pair's axis.
// One rounding follows: to bf16, or the quantiser of an e4m3 cache.
//
// Both are streams, bound by memory bandwidth.  A row is D / 16 lanes with two
// chunks of eight elements each: half-split pairs lie in the two chunks of one
// lane, neighbouring pairs in one chunk, so nothing crosses lanes but the largest
// magnitude that a row's scale needs.  A lane serves one head or several heads of a
// token: cosines and sines (twice the bytes of a head's row) are then loaded once for
// them.  CTAs of q and of k (append: of k and v together) follow one another in one
// launch, so no warp has both.
#include <algorithm>

#include "kv_rows.cuh"
#include "paged.cuh"

namespace attn {
namespace {

constexpr int kThreads = 256;

enum : int { ROPE = 0, APPEND_BF16 = 1, APPEND_E4M3 = 2 };

// The chunks of a lane and the pairs in them.
struct LaneMap {
    int c0, c1;                    // chunks (of eight elements)
    int p0, p1;                    // first pairs of their cosines' two groups of four
    bool r0, r1;                   // half-split: the lane's pairs turn; else: chunk c0's, chunk c1's do
};

template <int D>
__device__ __forceinline__ LaneMap lane_map(int lane, int rot, bool interleaved) {
    LaneMap m;
    if (interleaved) {
        m.c0 = lane;
        m.c1 = lane + D / 16;
        m.p0 = 4 * m.c0;
        m.p1 = 4 * m.c1;
        m.r0 = 8 * m.c0 < rot;
        m.r1 = 8 * m.c1 < rot;
        return m;
    }
    const int n = rot / 16;                                // lanes that turn; the others have chunks from rot on
    m.r0 = m.r1 = lane < n;
    m.c0 = lane < n ? lane : lane + n;
    m.c1 = lane < n ? lane + n : lane + D / 16;
    m.p0 = 8 * lane;
    m.p1 = 8 * lane + 4;
    return m;
}

// Cosines (or sines) of four pairs from pair i on.
template <bool AXES>
__device__ __forceinline__ float4 angles(const float* table, const RopeParams& p, const long long (&row)[4], int i) {
    if constexpr (!AXES) {
        return __ldg(reinterpret_cast<const float4*>(table + row[0] + i));
    } else {
        const uint32_t bits = (p.axes[i >> 4] >> (2 * (i & 15))) & 0xffu;
        const auto of = [&](uint32_t a) { return a == 0 ? row[0] : a == 1 ? row[1] : a == 2 ? row[2] : row[3]; };
        if (bits == (bits & 3u) * 0x55u) return __ldg(reinterpret_cast<const float4*>(table + of(bits & 3u) + i));
        return make_float4(__ldg(table + of(bits & 3u) + i), __ldg(table + of((bits >> 2) & 3u) + i + 1),
                           __ldg(table + of((bits >> 4) & 3u) + i + 2), __ldg(table + of(bits >> 6) + i + 3));
    }
}

// The lane's elements of a row in binary32, turned.
__device__ __forceinline__ void turn(const Row16& x, const LaneMap& m, bool interleaved, const float (&cs)[8],
                                     const float (&sn)[8], float (&v)[16]) {
    const uint32_t w[8] = {x.lo.x, x.lo.y, x.lo.z, x.lo.w, x.hi.x, x.hi.y, x.hi.z, x.hi.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        v[2 * e] = bf16_lo(w[e]);
        v[2 * e + 1] = bf16_hi(w[e]);
    }
    const auto pair = [&](float& a, float& b, int i) {
        const float x0 = __fsub_rn(__fmul_rn(a, cs[i]), __fmul_rn(b, sn[i]));
        b = __fadd_rn(__fmul_rn(a, sn[i]), __fmul_rn(b, cs[i]));
        a = x0;
    };
    if (interleaved) {
        if (m.r0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) pair(v[2 * i], v[2 * i + 1], i);
        }
        if (m.r1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) pair(v[8 + 2 * i], v[8 + 2 * i + 1], 4 + i);
        }
    } else if (m.r0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) pair(v[i], v[8 + i], i);
    }
}

__device__ __forceinline__ Row16 to_bf16(const float (&v)[16]) {
    return {make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])),
            make_uint4(pack_bf16x2(v[8], v[9]), pack_bf16x2(v[10], v[11]), pack_bf16x2(v[12], v[13]), pack_bf16x2(v[14], v[15]))};
}

// (plain loads: out may be the input itself; a thread reads what it writes first)
__device__ __forceinline__ Row16 load_chunks(const void* base, long long at, const LaneMap& m) {
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + at);
    return {src[m.c0], src[m.c1]};
}

__device__ __forceinline__ void store_chunks(void* base, long long at, const LaneMap& m, const Row16& x) {
    uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + at);
    dst[m.c0] = x.lo;
    dst[m.c1] = x.hi;
}

__device__ __forceinline__ void store_chunks8(void* base, long long at, const LaneMap& m, const uint4& c) {
    uint2* dst = reinterpret_cast<uint2*>(static_cast<uint8_t*>(base) + at);
    dst[m.c0] = make_uint2(c.x, c.y);
    dst[m.c1] = make_uint2(c.z, c.w);
}

// HQ heads a lane of q (and k of attn_rope), HK of the cache's k and v.
template <int D, int HQ, int HK, bool AXES, int MODE>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr int LANES = D / 16;
    const bool second = blockIdx.x >= p.q_blocks;          // k (append: k and v)
    const FastDiv by = second ? p.by_k_groups : p.by_q_groups;
    const unsigned x = (blockIdx.x - (second ? p.q_blocks : 0u)) * (kThreads / LANES) + threadIdx.x / LANES;
    const int lane = threadIdx.x % LANES;
    unsigned t = by.div(x);
    const unsigned group = x - t * by.d;
    const bool in = t < static_cast<unsigned>(p.T);
    if (!in) t = 0;
    const LaneMap m = lane_map<D>(lane, p.rot, p.interleaved);

    // Positions, and whether the token takes part (all lanes of a row alike).
    long long slot = 0;
    bool take = in;
    if constexpr (MODE != ROPE) {
        slot = in ? __ldg(p.slots + t) : -1;
        take = slot >= 0;
    }
    bool fine = true;
    long long row[4] = {0, 0, 0, 0};                       // (offsets of table rows)
    const unsigned n = p.period ? t - p.by_period.div(t) * p.by_period.d : t;
    if (p.positions == nullptr) {
        row[0] = static_cast<long long>(n) * (p.rot / 2);
    } else {
#pragma unroll
        for (int a = 0; a < (AXES ? 4 : 1); ++a) {
            if (a < p.n_axes && take) {
                const long long at = __ldg(p.positions + a * p.axis_stride + n);
                const bool ok = at >= 0 && at < p.rows;
                fine = fine && ok;
                row[a] = ok ? at * (p.rot / 2) : 0;
            }
        }
    }
    if (MODE != ROPE && slot >= p.num_slots) {
        report(p.status, SITE_PAGED_SLOT);
        take = false;
    }
    if (take && !fine) {
        report(p.status, SITE_ROPE_POSITION);
        take = false;
    }
    float cs[8], sn[8];
    const bool turns = take && (m.r0 || m.r1);
    {
        float4 c[2], s[2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const bool want = turns && (y ? m.r1 : m.r0);
            c[y] = want ? angles<AXES>(p.cos, p, row, y ? m.p1 : m.p0) : make_float4(0, 0, 0, 0);
            s[y] = want ? angles<AXES>(p.sin, p, row, y ? m.p1 : m.p0) : make_float4(0, 0, 0, 0);
        }
        const float f = p.inverse ? -1.0f : 1.0f;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            cs[4 * y] = c[y].x, cs[4 * y + 1] = c[y].y, cs[4 * y + 2] = c[y].z, cs[4 * y + 3] = c[y].w;
            sn[4 * y] = f * s[y].x, sn[4 * y + 1] = f * s[y].y, sn[4 * y + 2] = f * s[y].z, sn[4 * y + 3] = f * s[y].w;
        }
    }
    if (MODE == ROPE || !second) {
        const void* src = second ? p.k : p.q;
        void* dst = second ? p.k_out : p.q_out;
        const int heads = second ? p.H_kv : p.H;
        const long long from = t * (second ? p.k_stride : p.q_stride), to = t * (second ? p.k_out_stride : p.q_out_stride);
        const int h0 = group * HQ;
        Row16 r[HQ];
#pragma unroll
        for (int i = 0; i < HQ; ++i)
            if (take && h0 + i < heads) r[i] = load_chunks(src, from + (h0 + i) * D, m);
            else r[i] = Row16{};
#pragma unroll
        for (int i = 0; i < HQ; ++i) {
            if (!in || h0 + i >= heads) continue;
            float v[16];
            turn(r[i], m, p.interleaved, cs, sn, v);
            store_chunks(dst, to + (h0 + i) * D, m, to_bf16(v));
        }
    } else {
        const long long page = slot >> p.page_shift, in_page = slot & ((1ll << p.page_shift) - 1);
        const int h0 = group * HK;
        Row16 k[HK], v[HK];
#pragma unroll
        for (int i = 0; i < HK; ++i) {
            const bool have = take && h0 + i < p.H_kv;
            k[i] = have ? load_chunks(p.k, t * p.k_stride + (h0 + i) * D, m) : Row16{};
            v[i] = have ? load_chunks(p.v, t * p.v_stride + (h0 + i) * D, m) : Row16{};
        }
#pragma unroll
        for (int i = 0; i < HK; ++i) {
            float f[16];
            turn(k[i], m, p.interleaved, cs, sn, f);
            const bool store = take && h0 + i < p.H_kv;
            const long long at = ((page * p.H_kv + h0 + i) << p.page_shift) + in_page;
            if constexpr (MODE == APPEND_E4M3) {
                // The shuffles inside need every lane; rows that are not stored take part.
                float ks, vs;
                const uint4 kc = quantise_row<LANES>(f, ks), vc = quantise_row<LANES>(v[i], vs);
                if (store) {
                    store_chunks8(p.k_cache, at * D, m, kc);
                    store_chunks8(p.v_cache, at * D, m, vc);
                    if (lane == 0) {
                        p.k_scale[at] = ks;
                        p.v_scale[at] = vs;
                    }
                }
            } else if (store) {
                store_chunks(p.k_cache, at * D, m, to_bf16(f));
                store_chunks(p.v_cache, at * D, m, v[i]);
            }
        }
    }
}

template <int D, int HQ, int HK, bool AXES, int MODE>
cudaError_t launch(RopeParams p, cudaStream_t stream) {
    const auto groups = [](int heads, int per) { return (heads + per - 1) / per; };
    const int qg = groups(p.H, HQ), kg = groups(p.H_kv, MODE == ROPE ? HQ : HK);
    const auto blocks = [&](int g) {
        return static_cast<unsigned>((static_cast<long long>(p.T) * g * (D / 16) + kThreads - 1) / kThreads);
    };
    p.by_q_groups = FastDiv(std::max(qg, 1));
    p.by_k_groups = FastDiv(std::max(kg, 1));
    p.q_blocks = blocks(qg);
    rope_kernel<D, HQ, HK, AXES, MODE><<<p.q_blocks + blocks(kg), kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <int D, int MODE>
cudaError_t launch_mode(const RopeParams& p, cudaStream_t stream) {
    // Several heads a lane once the rows fill the machine.
    const long long lanes = static_cast<long long>(p.T) * (p.H + p.H_kv) * (D / 16);
    const bool many = lanes >= 2ll * kPlanSms * 2048;
    if (p.n_axes > 1)
        return many ? launch<D, 4, 2, true, MODE>(p, stream) : launch<D, 1, 1, true, MODE>(p, stream);
    return many ? launch<D, 4, 2, false, MODE>(p, stream) : launch<D, 1, 1, false, MODE>(p, stream);
}

template <int D>
cudaError_t launch_d(const RopeParams& p, cudaStream_t stream) {
    if (!p.append) return launch_mode<D, ROPE>(p, stream);
    return p.fp8 ? launch_mode<D, APPEND_E4M3>(p, stream) : launch_mode<D, APPEND_BF16>(p, stream);
}

}  // namespace

cudaError_t run_rope(const RopeParams& p, cudaStream_t stream) {
    return p.d == 64 ? launch_d<64>(p, stream) : p.d == 128 ? launch_d<128>(p, stream) : launch_d<256>(p, stream);
}

}  // namespace attn
