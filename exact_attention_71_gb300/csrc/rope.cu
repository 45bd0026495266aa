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
// chunks of eight elements each: half-split pairs lie in the two chunks of one lane,
// neighbouring pairs in one chunk, so nothing crosses lanes but the largest
// magnitude that a row's scale needs.  A lane has up to four heads of a token (two of k
// and v together), which share its pairs' angles.  One axis: they are two float4 each
// of the tables.  Several: a warp fetches its tokens' angles a pair a lane, whatever the
// pair's axis, and hands them round in shared memory (with float4 loads where four
// pairs share an axis, and single ones elsewhere: 4999 tokens of 24 heads on three
// alternating axes 15.8 us against 12.3, 7007 of 32 on sections 24.9 against 19.1; a
// CTA's angles together, behind a barrier: 13.4 and 20.7, and one axis 30 against 26).
//
// Order of the loads: the slot (padding has no position) and positions first, since the
// rows' loads would queue before them (32768 tokens of 48 heads into an e4m3 cache 145 us
// the other way round).
// Measured: 8192 tokens of 40 heads of 128, one axis, 26.0 us, 6.53 TB/s (96 % of the
// copy rate); those 32768 tokens 119.8 us, 6.32 TB/s (93 %), bf16 122.0 us, 6.74 TB/s;
// on three axes 155 and 151 us (a warp's chain of position, angles, rows); 32 tokens
// 2.9 us, a launch.
#include <algorithm>

#include "kv_rows.cuh"
#include "paged.cuh"

namespace attn {
namespace {

constexpr int kThreads = 128;
constexpr int kHeads = 4, kHeadsKv = 2;                    // heads a lane where there are many rows

enum : int { ROPE = 0, APPEND_BF16 = 1, APPEND_E4M3 = 2 };

// The chunks of a lane and the pairs that turn them.
struct LaneMap {
    int c0, c1;                    // chunks (of eight elements)
    int p0, p1;                    // first pairs of their angles' two quads
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

// A pair: a' = a c - b s, b' = a s + b c.
__device__ __forceinline__ void turn_pair(float& a, float& b, float c, float s) {
    const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    b = __fadd_rn(__fmul_rn(a, s), __fmul_rn(b, c));
    a = x;
}

// Two pairs of a row, in two words: half-split: v[0] and v[1] are elements i and i + 1,
// v[2] and v[3] those rot / 2 further on; neighbouring pairs: each word is one.
__device__ __forceinline__ void turn2(float (&v)[4], bool interleaved, float c0, float s0, float c1, float s1) {
    if (interleaved) {
        turn_pair(v[0], v[1], c0, s0);
        turn_pair(v[2], v[3], c1, s1);
    } else {
        turn_pair(v[0], v[2], c0, s0);
        turn_pair(v[1], v[3], c1, s1);
    }
}

// f(w0, w1, c, s, ..) for every two words of the lane's sixteen elements that turn
// together, and their two pairs' angles; a chunk that does not turn: f's last argument is
// false.
template <class F>
__device__ __forceinline__ void each_two(const LaneMap& m, bool interleaved, const float4 (&cos)[2], const float4 (&sin)[2], F&& f) {
    // words 0 .. 4 are chunk c0, 4 .. 8 chunk c1
    if (interleaved) {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            f(4 * y, 4 * y + 1, cos[y].x, sin[y].x, cos[y].y, sin[y].y, y ? m.r1 : m.r0);
            f(4 * y + 2, 4 * y + 3, cos[y].z, sin[y].z, cos[y].w, sin[y].w, y ? m.r1 : m.r0);
        }
    } else {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            f(2 * y, 2 * y + 4, cos[y].x, sin[y].x, cos[y].y, sin[y].y, m.r0);
            f(2 * y + 1, 2 * y + 5, cos[y].z, sin[y].z, cos[y].w, sin[y].w, m.r0);
        }
    }
}

// A row turned and rounded to bf16 in place.
__device__ __forceinline__ void turn_bf16(Row16& x, const LaneMap& m, bool interleaved, const float4 (&cos)[2],
                                          const float4 (&sin)[2]) {
    uint32_t w[8] = {x.lo.x, x.lo.y, x.lo.z, x.lo.w, x.hi.x, x.hi.y, x.hi.z, x.hi.w};
    each_two(m, interleaved, cos, sin, [&](int a, int b, float c0, float s0, float c1, float s1, bool turns) {
        float v[4] = {bf16_lo(w[a]), bf16_hi(w[a]), bf16_lo(w[b]), bf16_hi(w[b])};
        turn2(v, interleaved, c0, s0, c1, s1);
        w[a] = turns ? pack_bf16x2(v[0], v[1]) : w[a];
        w[b] = turns ? pack_bf16x2(v[2], v[3]) : w[b];
    });
    x = {make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7])};
}

// A row turned, in binary32.
__device__ __forceinline__ void turn_f32(const Row16& x, const LaneMap& m, bool interleaved, const float4 (&cos)[2],
                                         const float4 (&sin)[2], float (&out)[16]) {
    const uint32_t w[8] = {x.lo.x, x.lo.y, x.lo.z, x.lo.w, x.hi.x, x.hi.y, x.hi.z, x.hi.w};
    each_two(m, interleaved, cos, sin, [&](int a, int b, float c0, float s0, float c1, float s1, bool turns) {
        float v[4] = {bf16_lo(w[a]), bf16_hi(w[a]), bf16_lo(w[b]), bf16_hi(w[b])};
        if (turns) turn2(v, interleaved, c0, s0, c1, s1);
        out[2 * a] = v[0], out[2 * a + 1] = v[1], out[2 * b] = v[2], out[2 * b + 1] = v[3];
    });
}

// 16 bytes that are read once.  (Not a read-only load: out may be the input itself, a
// thread reads what it writes first.  volatile: the compiler moves plain loads down to
// the rows' use, one after the other: three axes 22.2 us against 19.3.)
__device__ __forceinline__ uint4 load_once(const void* at) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(at));
    return v;
}

template <bool ONCE>
__device__ __forceinline__ Row16 load_chunks(const void* base, long long at, const LaneMap& m) {
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + at);
    if constexpr (ONCE) return {load_once(src + m.c0), load_once(src + m.c1)};
    else return {src[m.c0], src[m.c1]};
}

// Whether a lane's rows are loaded between its position and its angles, by plain loads
// and with eight CTAs an SM instead of seven (64 registers: several heads a lane then spill 88
// bytes and read back 128, e4m3, 32 and 52, bf16): appending with one axis.  Microseconds,
// this way | the other: 32768 tokens of 48 heads of 128 bf16 cache 122.0 | 126.7, e4m3
// 119.8 | 125.5; of 64 65.2 | 65.1, 63.7 | 65.1; attn_rope's 8192 tokens of 40 heads 27.3 |
// 26.0; three axes: 7007 tokens of 32 heads 25.1 | 19.1, appending 4999 of 24 14.6 | 12.3.
template <bool AXES, int MODE>
constexpr bool kRowsEarly = MODE != ROPE && !AXES;

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
__global__ void __launch_bounds__(kThreads, kRowsEarly<AXES, MODE> ? 8 : 7) rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr int LANES = D / 16, PASS = kThreads / LANES, WARP = 32 / LANES;      // rows of a CTA, of a warp
    constexpr int HM = HQ > 2 * HK ? HQ : 2 * HK;          // rows in registers
    constexpr bool EARLY = kRowsEarly<AXES, MODE>;
    const bool second = blockIdx.x < p.k_blocks;           // k (append: k and v)
    const FastDiv by = second ? p.by_k_groups : p.by_q_groups;
    const unsigned x = (blockIdx.x - (second ? 0u : p.k_blocks)) * PASS + threadIdx.x / LANES;
    const int lane = threadIdx.x % LANES, half = p.rot / 2;
    const unsigned t = by.div(x), group = x - t * by.d;
    const bool in = t < static_cast<unsigned>(p.T);
    const LaneMap m = lane_map<D>(lane, p.rot, p.interleaved);
    const bool rows_of_one = MODE == ROPE || !second;      // (else: a head's k and v)
    const int heads = second ? p.H_kv : p.H, h0 = group * (rows_of_one ? HQ : HK);

    // Whether the token takes part (all lanes of a row alike).
    const auto position = [&](unsigned token, int axis) -> long long {
        const unsigned n = p.period ? token - p.by_period.div(token) * p.by_period.d : token;
        return p.positions == nullptr ? static_cast<long long>(n) : __ldg(p.positions + axis * p.axis_stride + n);
    };
    long long slot = 0, at = 0;
    bool take = in;
    if constexpr (MODE != ROPE) {
        slot = in ? __ldg(p.slots + t) : -1;
        if (slot >= p.num_slots) report(p.status, SITE_PAGED_SLOT);
        take = slot >= 0 && slot < p.num_slots;
    }
    // (Padding's positions are not read: there may be none.)
    bool fine = true;
#pragma unroll
    for (int a = 0; a < (AXES ? 4 : 1); ++a) {
        if (take && a < p.n_axes) {
            at = position(t, a);
            fine = fine && at >= 0 && at < p.rows;
        }
    }
    if (!fine) report(p.status, SITE_ROPE_POSITION);
    take = take && fine;

    Row16 r[HM];
    const auto load_rows = [&] {
        if (rows_of_one) {
            const void* src = second ? p.k : p.q;
            const long long from = t * (second ? p.k_stride : p.q_stride);
#pragma unroll
            for (int i = 0; i < HQ; ++i) r[i] = in && h0 + i < heads ? load_chunks<!EARLY>(src, from + (h0 + i) * D, m) : Row16{};
        } else {
#pragma unroll
            for (int i = 0; i < HK; ++i) {
                const bool have = in && h0 + i < heads;
                r[2 * i] = have ? load_chunks<!EARLY>(p.k, t * p.k_stride + (h0 + i) * D, m) : Row16{};
                r[2 * i + 1] = have ? load_chunks<!EARLY>(p.v, t * p.v_stride + (h0 + i) * D, m) : Row16{};
            }
        }
    };
    if constexpr (EARLY) load_rows();
    float4 cs[2], sn[2];
#pragma unroll
    for (int y = 0; y < 2; ++y) cs[y] = sn[y] = make_float4(0, 0, 0, 0);
    if constexpr (AXES) {
        // A pair a lane, whatever its axis, for the warp's tokens; handed round in shared
        // memory.  (Half-split: a lane needs quads 2l and 2l + 1; the even ones stand
        // before the odd ones, so that the lanes of a load are next to one another.)
        __shared__ float4 angles[kThreads / 32][WARP * D / 4];             // (token, cos / sin, pair)
        float* mine = reinterpret_cast<float*>(angles[threadIdx.x / 32]);
        const unsigned first = __shfl_sync(0xffffffffu, t, 0), last = min(__shfl_sync(0xffffffffu, t, 31), p.T - 1u);
        const int pairs = in || first < static_cast<unsigned>(p.T) ? static_cast<int>(last - first + 1) * half : 0;
        const auto place = [&](int i) { return p.interleaved ? i : ((i >> 2) & 1) * (half / 2) + ((i >> 3) << 2) + (i & 3); };
        // Where pair y's angles stand in the tables (-1: nowhere), and in `mine`.
        const auto table_at = [&](int y) -> long long {
            const int token = p.by_half.div(y), i = y - token * half;
            if constexpr (MODE != ROPE) {
                const long long slot = __ldg(p.slots + first + token);
                if (slot < 0 || slot >= p.num_slots) return -1;
            }
            const long long row = position(first + token, (p.axes[i >> 4] >> (2 * (i & 15))) & 3u);
            return row >= 0 && row < p.rows ? row * half + i : -1;
        };
        const auto put = [&](int y, long long from, float c, float s) {
            const int token = p.by_half.div(y), i = y - token * half;
            if (from < 0) return;
            mine[token * p.rot + place(i)] = c;
            mine[token * p.rot + half + place(i)] = s;
        };
        // The first two pairs of a lane (one token's, at 128 elements) together.
        const int y0 = threadIdx.x % 32;
        long long from[2];
        float c2[2], s2[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) from[k] = y0 + 32 * k < pairs ? table_at(y0 + 32 * k) : -1;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            c2[k] = from[k] >= 0 ? __ldg(p.cos + from[k]) : 0.0f;
            s2[k] = from[k] >= 0 ? __ldg(p.sin + from[k]) : 0.0f;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) put(y0 + 32 * k, from[k], c2[k], s2[k]);
        for (int y = y0 + 64; y < pairs; y += 32) {
            const long long at = table_at(y);
            if (at >= 0) put(y, at, __ldg(p.cos + at), __ldg(p.sin + at));
        }
        __syncwarp();
        if (take) {
            const float* c = mine + (t - first) * p.rot;
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                if (!(y ? m.r1 : m.r0)) continue;
                cs[y] = *reinterpret_cast<const float4*>(c + place(y ? m.p1 : m.p0));
                sn[y] = *reinterpret_cast<const float4*>(c + half + place(y ? m.p1 : m.p0));
            }
        }
    } else if (take) {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            if (!(y ? m.r1 : m.r0)) continue;
            cs[y] = __ldg(reinterpret_cast<const float4*>(p.cos + at * half + (y ? m.p1 : m.p0)));
            sn[y] = __ldg(reinterpret_cast<const float4*>(p.sin + at * half + (y ? m.p1 : m.p0)));
        }
    }
    if (p.inverse) {
#pragma unroll
        for (int y = 0; y < 2; ++y) sn[y] = make_float4(-sn[y].x, -sn[y].y, -sn[y].z, -sn[y].w);
    }

    if constexpr (!EARLY) load_rows();

    if (rows_of_one) {
        void* dst = second ? p.k_out : p.q_out;
        const long long to = t * (second ? p.k_out_stride : p.q_out_stride);
#pragma unroll
        for (int i = 0; i < HQ; ++i) {
            if (!in || h0 + i >= heads) continue;
            if (take) turn_bf16(r[i], m, p.interleaved, cs, sn);
            else r[i] = Row16{};
            store_chunks(dst, to + (h0 + i) * D, m, r[i]);
        }
    } else {
        const long long page = slot >> p.page_shift, in_page = slot & ((1ll << p.page_shift) - 1);
#pragma unroll
        for (int i = 0; i < HK; ++i) {
            const bool store = take && h0 + i < heads;
            const long long to = ((page * p.H_kv + h0 + i) << p.page_shift) + in_page;
            if constexpr (MODE == APPEND_E4M3) {
                // The shuffles inside need every lane; rows that are not stored take part.
                float f[16], ks, vs;
                turn_f32(r[2 * i], m, p.interleaved, cs, sn, f);
                const uint4 kc = quantise_row<LANES>(f, ks), vc = quantise_row<LANES>(r[2 * i + 1], vs);
                if (store) {
                    store_chunks8(p.k_cache, to * D, m, kc);
                    store_chunks8(p.v_cache, to * D, m, vc);
                    if (lane == 0) {
                        p.k_scale[to] = ks;
                        p.v_scale[to] = vs;
                    }
                }
            } else if (store) {
                turn_bf16(r[2 * i], m, p.interleaved, cs, sn);
                store_chunks(p.k_cache, to * D, m, r[2 * i]);
                store_chunks(p.v_cache, to * D, m, r[2 * i + 1]);
            }
        }
    }
}

template <int D, int HQ, int HK, bool AXES, int MODE>
cudaError_t launch(RopeParams p, cudaStream_t stream) {
    constexpr int PASS = kThreads / (D / 16);
    const auto groups = [](int heads, int per) { return (heads + per - 1) / per; };
    const int qg = groups(p.H, HQ), kg = groups(p.H_kv, MODE == ROPE ? HQ : HK);
    const auto blocks = [&](int g) { return static_cast<unsigned>((static_cast<long long>(p.T) * g + PASS - 1) / PASS); };
    p.by_q_groups = FastDiv(std::max(qg, 1));
    p.by_k_groups = FastDiv(std::max(kg, 1));
    p.by_half = FastDiv(p.rot / 2);
    p.k_blocks = blocks(kg);
    rope_kernel<D, HQ, HK, AXES, MODE><<<blocks(qg) + p.k_blocks, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <int D, int MODE>
cudaError_t launch_mode(const RopeParams& p, cudaStream_t stream) {
    // Several heads a lane once there are rows enough.  Microseconds, one head a lane |
    // several: attn_rope, 40 heads of 128, 64 tokens 2.3 | 2.6, 512 3.3 | 3.1, 1024 4.6 | 3.8,
    // 4096 13.7 | 11.5, 32 heads on three axes, 512 4.5 | 4.3, 4096 20.3 | 12.2; appending, 40 and
    // 8 heads, 32 tokens 2.8 | 3.8, 512 3.8 | 4.6, 1024 5.8 | 5.5, 2048 11.1 | 9.7.
    const long long lanes = static_cast<long long>(p.T) * (p.H + p.H_kv) * (D / 16);
    const bool many = lanes >= kPlanSms * (MODE == ROPE ? 1024ll : 2048ll);
    if (p.n_axes > 1)
        return many ? launch<D, kHeads, kHeadsKv, true, MODE>(p, stream) : launch<D, 1, 1, true, MODE>(p, stream);
    return many ? launch<D, kHeads, kHeadsKv, false, MODE>(p, stream) : launch<D, 1, 1, false, MODE>(p, stream);
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
