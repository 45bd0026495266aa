// Attention of a few query rows against a key range of the paged cache: the
// memory-bound side of the paged attention (decoding steps).
//
//     m = max_j s_j,  l = sum_j exp2(s_j - m),  O = sum_j exp2(s_j - m) v_j / l
//     s_j = scale * log2(e) * q . k_j        (times k's row scale: e4m3 cache)
//
// taken in one pass over the keys with a running m, l and O.
//
// A CTA serves 16 query rows of one key/value head (the group's heads of one
// sequence, or rows of several sequences over the prefix they share) and one
// key range; its four warps take the range's 16-key steps in turn, each with
// its own m, l and O, joined once at the end.  Every key row is read once per
// CTA, so the bound is the cache's bytes: at 16 rows a step does 16 FLOP per
// byte of K and V (bf16), a twentieth of what the tensor cores could do per
// byte of HBM bandwidth.  The products therefore use the warp-level m16n8k16
// MMA with operands in registers: tcgen05 would leave 112 of its 128 tile rows
// empty and need the tile to be assembled in shared memory first.
//
// No data crosses threads on the way in.  The MMA's k index may be permuted
// freely (both operands alike), and so may O's columns, so each thread is given
// whole 16-byte chunks of the rows its B fragments need:
//   S = Q K^T   thread (g, t) = (lane / 4, lane % 4) holds key rows g and 8 + g,
//               d elements [c * 4E + t * E, + E) of them (E elements a chunk)
//   O += P V    it holds value rows 2t, 2t+1, 2t+8, 2t+9, columns
//               [c * 8E + g * E, + E); pairs of rows are interleaved by byte
//               permutes, which for e4m3 is part of the conversion to bf16
// A thread copies its own chunks with cp.async into its own slots of a
// shared-memory ring and reads them back after cp.async.wait_group: a
// per-thread queue, STAGES - 1 steps deep, without any barrier.
#pragma once

#include <cuda_bf16.h>

#include "paged.cuh"
#include "sm103_ptx.cuh"

namespace attn {

// 16 (or 8) bytes global -> shared; nothing is read and zeros are written when
// `valid` is false.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, bool valid) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(valid ? 8 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// D (16 x 8, fp32) += A (16 x 16, bf16) B (16 x 8, bf16).
__device__ __forceinline__ void mma_m16n8k16(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two e4m3 codes -> two bf16, exactly.  sel picks [code, sign, code, sign]
// bytes (the sign byte by the permute's sign replication); shifted left by 4,
// code bit 7 (and its copies) reach bit 15 and the exponent and mantissa bits
// 10..4, i.e. a bf16 of value 2^-120 times the code's; the product with 2^120
// is exact, subnormal codes included (they are subnormal bf16 before it).  A
// NaN code becomes +-480: such rows have a NaN scale, which decides.
template <uint32_t SEL>
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t a, uint32_t b) {
    uint32_t x, r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(x) : "r"(a), "r"(b), "n"(SEL));
    x = (x << 4) & 0x87f087f0u;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(0x7b807b80u));
    return r;
}

template <int D_, bool FP8_>
struct StreamCfg {
    static constexpr int D = D_;
    static constexpr bool FP8 = FP8_;
    static constexpr int ES = FP8 ? 1 : 2;
    static constexpr int E = 16 / ES;                              // elements of a K chunk
    static constexpr int KC = D / (4 * E);                         // K chunks per row and thread
    static constexpr int VB = D * ES / 8 >= 16 ? 16 : 8;           // bytes of a V chunk
    static constexpr int VE = VB / ES;
    static constexpr int VC = D / (8 * VE);                        // V chunks per row and thread
    static constexpr int WARPS = 4;
    static constexpr int THREADS = WARPS * 32;
    static constexpr int STEP = 16;                                // keys per warp step
    static constexpr int K_BYTES = 2 * KC * 16 * THREADS;
    static constexpr int V_BYTES = 4 * VC * VB * THREADS;
    static constexpr int S_BYTES = FP8 ? 4 * 8 * THREADS : 0;      // scales: K and V, two key pairs each
    static constexpr int STAGE_BYTES = K_BYTES + V_BYTES + S_BYTES;
    static constexpr int CTAS = D == 64 ? 4 : D == 128 ? 3 : FP8 ? 2 : 1;     // per SM
    static constexpr int STAGES = D == 64 ? (FP8 ? 4 : 3) : D == 128 ? (FP8 ? 3 : 2) : 3;
    static constexpr int RING_BYTES = STAGES * STAGE_BYTES;
    static constexpr int JOIN_BYTES = WARPS * 16 * (D + 2) * 4;
    static constexpr int SMEM_BYTES = RING_BYTES > JOIN_BYTES ? RING_BYTES : JOIN_BYTES;
    static constexpr int NT = D / 8;                               // O's column tiles
    static_assert(CTAS * (SMEM_BYTES + 1024) <= 228 * 1024, "shared memory");
};

// Replaces the infinities and NaN among this thread's V chunks (value rows 2t,
// 2t+1, 2t+8, 2t+9 of the step, those from `from` on) by 0; bit r of the result: the step's row r had
// one.  Called by whole warps.
template <class Cfg>
__device__ __noinline__ uint32_t clear_nonfinite(uint8_t* sv, int t, int from) {
    uint32_t hit = 0;
    for (int x = 0; x < 4; ++x) {
        const int row = 2 * t + (x & 1) + (x >> 1) * 8;
        bool any = false;
        if (row < from) continue;
        for (int c = 0; c < Cfg::VC; ++c) {
            uint32_t* at = reinterpret_cast<uint32_t*>(sv + (x * Cfg::VC + c) * Cfg::VB * Cfg::THREADS);
            for (int y = 0; y < Cfg::VB / 4; ++y) {
                uint32_t w = at[y];
                if ((w & 0x7f80u) == 0x7f80u) { w &= 0xffff0000u; any = true; }
                if ((w & 0x7f800000u) == 0x7f800000u) { w &= 0xffffu; any = true; }
                at[y] = w;
            }
        }
        if (any) hit |= 1u << row;
    }
    return __reduce_or_sync(0xffffffffu, hit);
}

// PREFIX: the rows are all sequences' rows over the shared prefix; otherwise
// one sequence's (blockIdx.y) over its own tokens.  DIRECT: this is the only
// part, o and lse are written; otherwise a partial result.
template <class Cfg, bool PREFIX, bool DIRECT>
__global__ void __launch_bounds__(Cfg::THREADS, Cfg::CTAS) paged_stream_kernel(const PagedParams p) {
    constexpr int D = Cfg::D, KC = Cfg::KC, VC = Cfg::VC, NT = Cfg::NT, STAGES = Cfg::STAGES;
    constexpr bool FP8 = Cfg::FP8;
    extern __shared__ __align__(16) uint8_t smem[];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int rows = (PREFIX ? p.B : 1) * p.Nq * p.G;
    const int tiles = (rows + 15) / 16;
    // Row tiles of the same keys run next to one another.
    const int tile = blockIdx.x % tiles;
    const int kvh = blockIdx.x / tiles % p.H_kv, part = blockIdx.x / tiles / p.H_kv;
    const int seq = PREFIX ? 0 : blockIdx.y;

    // The key range.
    int len = PREFIX ? p.prefix_len : __ldg(p.seq_lens + seq);
    const long long room = static_cast<long long>(p.max_pages) << p.page_shift;
    if (!PREFIX && len > room) {
        if (tid == 0) atomicCAS(p.status, 0, SITE_PAGED_LENGTH);
        len = static_cast<int>(room);
    }
    len = max(len, 0);
    const int parts = PREFIX ? p.prefix_parts : p.own_parts;
    const int chunk = max(((len + parts - 1) / parts + 63) / 64 * 64, PREFIX ? 64 : kOwnChunk);
    const int k0 = static_cast<int>(min(static_cast<long long>(part) * chunk, static_cast<long long>(len)));
    const int k1 = min(k0 + chunk, len);
    const int* table = PREFIX ? p.prefix_table : p.table + seq * p.table_stride;

    // This thread's two query rows: g and g + 8 of the tile.
    int row_out[2], limit[2];      // index in q / o / the partials (-1: none); keys it sees
    uint32_t qa[2][D / 8];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int r = tile * 16 + g + 8 * x;
        row_out[x] = -1;
        limit[x] = 0;
        const uint4* src = nullptr;
        if (r < rows) {
            const int per = p.Nq * p.G;
            const int b = PREFIX ? r / per : seq, i = (PREFIX ? r % per : r) / p.G, h = kvh * p.G + r % p.G;
            row_out[x] = (b * p.Nq + i) * p.H + h;
            limit[x] = PREFIX || !p.causal ? len : max(0, len - p.Nq + 1 + i);
            src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                 static_cast<long long>(row_out[x]) * D);
        }
        // chunk c of the k permutation: elements [c * 4E + t * E, + E)
#pragma unroll
        for (int c = 0; c < KC; ++c) {
#pragma unroll
            for (int y = 0; y < Cfg::E / 8; ++y) {
                const uint4 v = src ? __ldg(src + (c * 4 + t) * (Cfg::E / 8) + y) : make_uint4(0, 0, 0, 0);
                const int at = (c * (Cfg::E / 8) + y) * 4;
                qa[x][at] = v.x;
                qa[x][at + 1] = v.y;
                qa[x][at + 2] = v.z;
                qa[x][at + 3] = v.w;
            }
        }
    }

    // From this key on some row of the tile may not see what another does.
    int diag = len;
    if (!PREFIX && p.causal) diag = max(0, len - p.Nq + 1 + (tile * 16) / p.G);

    const int first = k0 / 16 + warp;                      // this warp's steps: first, first + 4, ...
    const int steps_end = k0 < k1 ? (k1 + 15) / 16 : 0;    // an empty range ends at len, inside a step
    const uint32_t ring = smem_u32(smem);
    uint32_t bad = 0;                                      // bit (step / 4) & 31: the step's page is invalid

    auto page_of = [&](int step) -> int { return step < steps_end ? __ldg(table + ((step * 16) >> p.page_shift)) : 0; };
    auto issue = [&](int step, int stage, int page) {
        if (step < steps_end) {
            const bool ok = page >= 0 && page < p.num_pages;
            const uint32_t bit = 1u << ((step >> 2) & 31);
            bad = ok ? bad & ~bit : bad | bit;
            if (!ok && lane == 0) atomicCAS(p.status, 0, SITE_PAGED_PAGE);
            const int key0 = step * 16;
            const long long at = ((static_cast<long long>(ok ? page : 0) * p.H_kv + kvh) << p.page_shift) +
                                 (key0 & ((1 << p.page_shift) - 1));
            const int n = ok ? min(k1 - key0, 16) : 0;     // valid rows of the step
            const uint8_t* kb = static_cast<const uint8_t*>(p.k_cache) + at * (D * Cfg::ES);
            const uint8_t* vb = static_cast<const uint8_t*>(p.v_cache) + at * (D * Cfg::ES);
            const uint32_t ks = ring + stage * Cfg::STAGE_BYTES + tid * 16;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int r = x * 8 + g;
                const uint8_t* src = kb + (r < n ? r : 0) * (D * Cfg::ES) + t * 16;
#pragma unroll
                for (int c = 0; c < KC; ++c) cp_async16(ks + (x * KC + c) * 16 * Cfg::THREADS, src + c * 64, r < n);
            }
            const uint32_t vs = ring + stage * Cfg::STAGE_BYTES + Cfg::K_BYTES + tid * Cfg::VB;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int r = 2 * t + (x & 1) + (x >> 1) * 8;
                const uint8_t* src = vb + (r < n ? r : 0) * (D * Cfg::ES) + g * Cfg::VB;
#pragma unroll
                for (int c = 0; c < VC; ++c) {
                    const uint32_t dst = vs + (x * VC + c) * Cfg::VB * Cfg::THREADS;
                    if constexpr (Cfg::VB == 16) cp_async16(dst, src + c * 128, r < n);
                    else cp_async8(dst, src + c * 64, r < n);
                }
            }
            if constexpr (FP8) {
                // Scales of keys 2t, 2t+1 and 2t+8, 2t+9.  Rows past n are
                // never used (their scores are masked); the pair stays inside
                // the page.
                const uint32_t ss = ring + stage * Cfg::STAGE_BYTES + Cfg::K_BYTES + Cfg::V_BYTES + tid * 8;
                cp_async8(ss, p.k_scale + at + 2 * t, 2 * t < n);
                cp_async8(ss + 8 * Cfg::THREADS, p.k_scale + at + 2 * t + 8, 2 * t + 8 < n);
                cp_async8(ss + 16 * Cfg::THREADS, p.v_scale + at + 2 * t, 2 * t < n);
                cp_async8(ss + 24 * Cfg::THREADS, p.v_scale + at + 2 * t + 8, 2 * t + 8 < n);
            }
        }
        cp_async_commit();
    };

    float o[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

    int next_page = page_of(first);
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) {
        const int step = first + 4 * s;
        const int page = next_page;
        next_page = page_of(step + 4);
        issue(step, s, page);
    }
    int stage = 0;
    for (int step = first; step < steps_end; step += 4) {
        {
            const int ahead = step + 4 * (STAGES - 1);
            const int page = next_page;
            next_page = page_of(ahead + 4);
            issue(ahead, stage == 0 ? STAGES - 1 : stage - 1, page);
        }
        cp_async_wait<STAGES - 1>();
        const uint8_t* st = smem + stage * Cfg::STAGE_BYTES;
        stage = stage + 1 == STAGES ? 0 : stage + 1;

        // ---------------------------------------------------------- S = Q K^T
        float s[2][4];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            s[x][0] = s[x][1] = s[x][2] = s[x][3] = 0.0f;
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                const uint4 kk = *reinterpret_cast<const uint4*>(st + (x * KC + c) * 16 * Cfg::THREADS + tid * 16);
                if constexpr (FP8) {
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t word = w == 0 ? kk.x : w == 1 ? kk.y : w == 2 ? kk.z : kk.w;
                        const int at = c * 8 + w * 2;
                        mma_m16n8k16(s[x], qa[0][at], qa[1][at], qa[0][at + 1], qa[1][at + 1],
                                     e4m3_pair<0x9180>(word, 0), e4m3_pair<0xb3a2>(word, 0));
                    }
                } else {
                    const int at = c * 4;
                    mma_m16n8k16(s[x], qa[0][at], qa[1][at], qa[0][at + 1], qa[1][at + 1], kk.x, kk.y);
                    mma_m16n8k16(s[x], qa[0][at + 2], qa[1][at + 2], qa[0][at + 3], qa[1][at + 3], kk.z, kk.w);
                }
            }
        }
        // s[x][0..1]: row g, keys x * 8 + 2t, + 1; s[x][2..3]: row g + 8.
        float2 vscale[2];
        const uint8_t* sc = st + Cfg::K_BYTES + Cfg::V_BYTES + tid * 8;
        const bool skip = (bad >> ((step >> 2) & 31)) & 1u;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            float2 mul = make_float2(p.scale_log2, p.scale_log2);
            if constexpr (FP8) {
                const float2 ks = *reinterpret_cast<const float2*>(sc + x * 8 * Cfg::THREADS);
                vscale[x] = *reinterpret_cast<const float2*>(sc + (2 + x) * 8 * Cfg::THREADS);
                mul.x *= ks.x;
                mul.y *= ks.y;
            }
            const int key = step * 16 + x * 8 + 2 * t;
            // A masked score is -inf whatever was read for it.
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int lim = skip ? 0 : min(limit[r], k1);
                s[x][2 * r] = key < lim ? s[x][2 * r] * mul.x : -INFINITY;
                s[x][2 * r + 1] = key + 1 < lim ? s[x][2 * r + 1] * mul.y : -INFINITY;
            }
        }
        // ------------------------------------------------------ running maximum
        // The reference moves only when some score exceeds it by more than 8
        // (log2 units), so that the quad's shuffles and O's rescaling are rare;
        // O and l share the reference, so the result does not depend on it.
        const float x0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
        const float x1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
        const bool move = x0 > m[0] + 8.0f || x1 > m[1] + 8.0f;
        if (__any_sync(0xffffffffu, move)) {
            float mx[2] = {x0, x1};
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
                mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
                // (per row: a row's result does not depend on its neighbours)
                const float mn = mx[r] > m[r] + 8.0f ? mx[r] : m[r];
                const float a = mn == m[r] ? 1.0f : ex2_approx(m[r] - mn);
                m[r] = mn;
                l[r] *= a;
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    o[j][2 * r] *= a;
                    o[j][2 * r + 1] *= a;
                }
            }
        }
        const float n0 = m[0] == -INFINITY ? 0.0f : m[0], n1 = m[1] == -INFINITY ? 0.0f : m[1];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            s[x][0] = ex2_approx(s[x][0] - n0);
            s[x][1] = ex2_approx(s[x][1] - n0);
            s[x][2] = ex2_approx(s[x][2] - n1);
            s[x][3] = ex2_approx(s[x][3] - n1);
            l[0] += s[x][0] + s[x][1];
            l[1] += s[x][2] + s[x][3];
            if constexpr (FP8) {
                // V's row scale rides on P; l sums the plain probabilities.
                // A weight of 0 stays 0 beside a NaN scale: a row that does not
                // see the key must not notice it.
                s[x][0] = s[x][0] == 0.0f ? 0.0f : s[x][0] * vscale[x].x;
                s[x][1] = s[x][1] == 0.0f ? 0.0f : s[x][1] * vscale[x].y;
                s[x][2] = s[x][2] == 0.0f ? 0.0f : s[x][2] * vscale[x].x;
                s[x][3] = s[x][3] == 0.0f ? 0.0f : s[x][3] * vscale[x].y;
            }
        }
        // P is rounded to bf16 for the product (relative 2^-9 at most per
        // weight, as the dense forward does); l keeps the unrounded values.
        const uint32_t a0 = pack_bf16x2(s[0][0], s[0][1]), a1 = pack_bf16x2(s[0][2], s[0][3]);
        const uint32_t a2 = pack_bf16x2(s[1][0], s[1][1]), a3 = pack_bf16x2(s[1][2], s[1][3]);
        // ---------------------------------------------------------- O += P V
        const uint8_t* sv = st + Cfg::K_BYTES + tid * Cfg::VB;
        if constexpr (!FP8 && !PREFIX) {
            // 0 * NaN is NaN: where rows of the tile see different keys, a
            // non-finite value is taken out of the product and the rows that
            // do see its key become NaN as a whole.
            if (diag < len && step * 16 + 16 > diag) {
                const uint32_t hit = clear_nonfinite<Cfg>(const_cast<uint8_t*>(sv), t, diag - step * 16);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int n = min(max(min(limit[r], k1) - step * 16, 0), 16);
                    if (hit & ((1u << n) - 1u)) l[r] = __uint_as_float(0x7fc00000u);
                }
            }
        }
#pragma unroll
        for (int c = 0; c < VC; ++c) {
            uint32_t w[4][Cfg::VB / 4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const uint8_t* at = sv + (x * VC + c) * Cfg::VB * Cfg::THREADS;
                if constexpr (Cfg::VB == 16) {
                    const uint4 v = *reinterpret_cast<const uint4*>(at);
                    w[x][0] = v.x;
                    w[x][1] = v.y;
                    w[x][Cfg::VB / 4 - 2] = v.z;
                    w[x][Cfg::VB / 4 - 1] = v.w;
                } else {
                    const uint2 v = *reinterpret_cast<const uint2*>(at);
                    w[x][0] = v.x;
                    w[x][1] = v.y;
                }
            }
#pragma unroll
            for (int y = 0; y < Cfg::VB / 4; ++y) {
                float(*oo)[4] = &o[c * Cfg::VE + y * (4 / Cfg::ES)];
                if constexpr (FP8) {
                    mma_m16n8k16(oo[0], a0, a1, a2, a3, e4m3_pair<0xc480>(w[0][y], w[1][y]),
                                 e4m3_pair<0xc480>(w[2][y], w[3][y]));
                    mma_m16n8k16(oo[1], a0, a1, a2, a3, e4m3_pair<0xd591>(w[0][y], w[1][y]),
                                 e4m3_pair<0xd591>(w[2][y], w[3][y]));
                    mma_m16n8k16(oo[2], a0, a1, a2, a3, e4m3_pair<0xe6a2>(w[0][y], w[1][y]),
                                 e4m3_pair<0xe6a2>(w[2][y], w[3][y]));
                    mma_m16n8k16(oo[3], a0, a1, a2, a3, e4m3_pair<0xf7b3>(w[0][y], w[1][y]),
                                 e4m3_pair<0xf7b3>(w[2][y], w[3][y]));
                } else {
                    mma_m16n8k16(oo[0], a0, a1, a2, a3, __byte_perm(w[0][y], w[1][y], 0x5410),
                                 __byte_perm(w[2][y], w[3][y], 0x5410));
                    mma_m16n8k16(oo[1], a0, a1, a2, a3, __byte_perm(w[0][y], w[1][y], 0x7632),
                                 __byte_perm(w[2][y], w[3][y], 0x7632));
                }
            }
        }
    }
    cp_async_wait<0>();

    // ------------------------------------------------------------ join the warps
    // o[c * VE + e][2r + z] is row g + 8r, column c * 8 * VE + (2t + z) * VE + e.
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    }
    __syncthreads();                       // every warp is done with the ring
    float* js = reinterpret_cast<float*>(smem);                        // (warp, 16, D)
    float* jm = js + Cfg::WARPS * 16 * D;                              // (warp, 16)
    float* jl = jm + Cfg::WARPS * 16;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        float* dst = js + (warp * 16 + g + 8 * r) * D;
#pragma unroll
        for (int c = 0; c < VC; ++c)
#pragma unroll
            for (int z = 0; z < 2; ++z)
#pragma unroll
                for (int e = 0; e < Cfg::VE; e += 4)
                    *reinterpret_cast<float4*>(dst + c * 8 * Cfg::VE + (2 * t + z) * Cfg::VE + e) =
                        make_float4(o[c * Cfg::VE + e][2 * r + z], o[c * Cfg::VE + e + 1][2 * r + z],
                                    o[c * Cfg::VE + e + 2][2 * r + z], o[c * Cfg::VE + e + 3][2 * r + z]);
        if (t == 0) {
            jm[warp * 16 + g + 8 * r] = m[r];
            jl[warp * 16 + g + 8 * r] = l[r];
        }
    }
    __syncthreads();
    // A thread takes 4 columns of a row at a time; D / 4 threads a row.
    for (int x = tid; x < 16 * (D / 4); x += Cfg::THREADS) {
        const int rr = x / (D / 4), c4 = x % (D / 4);
        const int r = tile * 16 + rr;
        if (r >= rows) continue;
        const int per = p.Nq * p.G;
        const int b = PREFIX ? r / per : seq, i = (PREFIX ? r % per : r) / p.G, h = kvh * p.G + r % p.G;
        const long long out = (static_cast<long long>(b) * p.Nq + i) * p.H + h;
        float mm = jm[rr];
#pragma unroll
        for (int w = 1; w < Cfg::WARPS; ++w) mm = fmaxf(mm, jm[w * 16 + rr]);
        const float ref = mm == -INFINITY ? 0.0f : mm;
        float ll = 0.0f;
        float4 acc = make_float4(0, 0, 0, 0);
#pragma unroll
        for (int w = 0; w < Cfg::WARPS; ++w) {
            const float a = ex2_approx(jm[w * 16 + rr] - ref);
            const float4 v = *reinterpret_cast<const float4*>(js + (w * 16 + rr) * D + c4 * 4);
            ll += a * jl[w * 16 + rr];
            acc.x += a * v.x;
            acc.y += a * v.y;
            acc.z += a * v.z;
            acc.w += a * v.w;
        }
        // l = 0: the row sees no key of this range (O = 0, lse = -inf)
        const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
        acc.x *= inv;
        acc.y *= inv;
        acc.z *= inv;
        acc.w *= inv;
        const float lse2 = ll == 0.0f ? -INFINITY : ref + __log2f(ll);
        if constexpr (DIRECT) {
            reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + out * D)[c4] =
                make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
            if (c4 == 0) p.lse[(static_cast<long long>(b) * p.H + h) * p.Nq + i] = lse2 * 0.69314718055994530942f;
        } else {
            const long long pr = static_cast<long long>(PREFIX ? part : p.prefix_parts + part) *
                                     (static_cast<long long>(p.B) * p.Nq * p.H) + out;
            // An empty part's O is not read by the join.
            if (lse2 != -INFINITY) reinterpret_cast<float4*>(p.part_o + pr * D)[c4] = acc;
            if (c4 == 0) p.part_lse[pr] = lse2;
        }
    }
}

}  // namespace attn
