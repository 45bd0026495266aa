// Attention of a tree's nodes over one another, and the join with the partial
// results over the tokens before them (the prefix, and a sequence's own tokens:
// every node sees all of those, so the kernels of the paged attention take them
// without a mask).
//
//     s_j = scale * log2(e) * q . k_j  for the nodes j that are i or an ancestor of i
//     m = max(max_j s_j, max_p lse_p)
//     l = sum_j exp2(s_j - m) + sum_p exp2(lse_p - m)
//     O = (sum_j exp2(s_j - m) v_j + sum_p exp2(lse_p - m) O_p) / l
//
// A node sees few others: its depth, a dozen of sixty-four.  W warps take 16 query
// rows of one key/value head (the nodes' heads of its group), collect the nodes that
// any of them sees into a list, and multiply blocks of 16 of the list, so the work
// goes by the paths and not by the square of the drafts.  What a row does not see of
// the list is masked.  Everything before wait_prerequisites needs no partial result
// and runs beside the kernels that make them.
//
// Products: m16n8k16 on bf16, queries the 16 rows, operands straight from global
// memory into registers: the k index may be permuted (both operands alike), and O's
// columns too, so every lane takes whole chunks of a row (K: chunks 4c + t of row g;
// V: chunks 8c + g of the rows 2t, 2t + 1, 2t + 8, 2t + 9, pairs of rows interleaved
// by byte permutes).  O's fragment is then 16 consecutive columns a lane, the shape in
// which partial results are read and O is written.  e4m3 codes are bf16 values; K's
// scales multiply the scores, V's ride on the weights, and the weights enter as two
// bf16 parts (2^-17), which costs nothing here.
//
// A value that is not finite, of a node that some row of the list does not see, must
// not meet a weight of 0: it is taken out, and the rows that see its node become NaN.
#include <cuda_bf16.h>

#include "paged.cuh"
#include "paged_stream_kernel.cuh"
#include "sm103_bulk.cuh"

namespace attn {
namespace {

constexpr int kRows = 16, kWarps = 4, kWords = kMaxTree / 32;

// What the warps of a row tile share.
struct TreeTile {
    uint32_t vis[kRows][kWords + 1];       // token of the tile: its path, a bit per node
    int parents[kMaxTree];
    unsigned short list[kMaxTree];         // nodes that some row sees
    int count;
    uint32_t node;                         // bit per token: it is a node
};

__device__ __forceinline__ uint32_t codes_to_bf16x2(uint32_t f16x2) {
    const float2 x = f16x2_to_float2(f16x2);
    return pack_bf16x2(x.x, x.y);
}

__device__ __forceinline__ bool not_finite_bf16x2(uint32_t w) { return (((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u) != 0; }

__device__ __forceinline__ uint32_t finite_bf16x2(uint32_t w) {
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
    return w;
}

template <int D, bool FP8, int W>
struct TreeCfg {
    static constexpr int TILES = kWarps / W;
    static constexpr int JD = D + 4;                       // row stride of the join (banks)
    static constexpr int SMEM_BYTES = W == 1 ? 0 : kWarps * kRows * (JD + 2) * 4;
};

template <int D, bool FP8, int W>
__global__ void __launch_bounds__(kWarps * 32) paged_tree_kernel(const __grid_constant__ PagedParams p, const int tiles,
                                                                const FastDiv by_tiles) {
    using Cfg = TreeCfg<D, FP8, W>;
    constexpr int CC = D / 64;                             // O's groups of 64 columns
    constexpr int KC = FP8 ? D / 64 : D / 32;              // 16-byte chunks of a K row and lane
    constexpr int ROW = D * (FP8 ? 1 : 2);                 // bytes of a cache row
    constexpr bool QREG = D <= 128;
    extern __shared__ float join[];
    __shared__ TreeTile shared[Cfg::TILES];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, w = warp % W;
    TreeTile& s = shared[warp / W];
    const unsigned x = blockIdx.x * Cfg::TILES + warp / W;
    const bool in = x < static_cast<unsigned>(tiles);
    unsigned y = by_tiles.div(in ? x : 0);
    const int tile = (in ? x : 0) - y * by_tiles.d;
    const int seq = p.by_heads.div(y), kvh = y - seq * p.H_kv;
    const int z0 = tile * kRows, live = in ? min(kRows, p.Nq * p.G - z0) : 0;
    const int i0 = p.by_G.div(z0), i1 = live > 0 ? p.by_G.div(z0 + live - 1) : i0 - 1;         // tokens of the tile

    // ------------------------------------------------------------ paths and list
    int len = max(0, __ldg(p.seq_lens + seq));
    len = static_cast<int>(min(static_cast<long long>(len), static_cast<long long>(p.max_pages) << p.page_shift));
    const int* parents = p.parents + seq * p.parents_stride;
    for (int j = w * 32 + lane; j < p.Nq; j += W * 32) s.parents[j] = __ldg(parents + j);
    __syncthreads();
    const int words = (p.Nq + 31) >> 5;
    if (w == 0) {
        bool node = false;
        if (lane < kRows) {
            for (int y = 0; y < words; ++y) s.vis[lane][y] = 0;
            int at = i0 + lane;
            if (at <= i1 && s.parents[at] >= -1) {
                node = true;
                for (int steps = 0; at >= 0; ++steps) {
                    if (at >= p.Nq || steps >= p.Nq) {
                        node = false;
                        break;
                    }
                    s.vis[lane][at >> 5] |= 1u << (at & 31);
                    at = s.parents[at];
                }
                if (at < -1) node = false;
                if (!node) {
                    atomicCAS(p.status, 0, SITE_TREE_PARENT);
                    for (int y = 0; y < words; ++y) s.vis[lane][y] = 0;
                }
            }
        }
        const uint32_t nodes = __ballot_sync(0xffffffffu, node);
        int count = 0;
        for (int y = 0; y < words; ++y) {
            const uint32_t any = __reduce_or_sync(0xffffffffu, lane < kRows ? s.vis[lane][y] : 0u);
            const int j = y * 32 + lane;
            // (drafts before the sequence's first token are not there)
            const bool have = ((any >> lane) & 1u) && len - p.Nq + j >= 0;
            const uint32_t all = __ballot_sync(0xffffffffu, have);
            if (have) s.list[count + __popc(all & ((1u << lane) - 1u))] = static_cast<unsigned short>(j);
            count += __popc(all);
        }
        if (lane == 0) {
            s.count = count;
            s.node = nodes;
        }
    }
    __syncthreads();
    const int count = s.count;

    // Rows g and g + 8 of the tile: their tokens, and their indices in q and o.
    long long out[2];
    int token[2], lse_at[2];
    bool node[2], row_in[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        row_in[r] = g + 8 * r < live;
        const int z = z0 + (row_in[r] ? g + 8 * r : 0), i = p.by_G.div(z), h = kvh * p.G + z - i * p.G;
        token[r] = min(i - i0, kRows - 1);
        node[r] = row_in[r] && ((s.node >> token[r]) & 1u);
        out[r] = (static_cast<long long>(seq) * p.Nq + i) * p.H + h;
        lse_at[r] = (seq * p.H + h) * p.Nq + i;
    }
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q);
    constexpr int QW = FP8 ? 8 : 4;                        // Q's words of a chunk and row
    auto load_q = [&](int c, uint32_t (&a)[2][QW]) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int i = 0; i < QW / 4; ++i) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (row_in[r]) v = __ldg(reinterpret_cast<const uint4*>(q + out[r] * D) + (4 * c + t) * (QW / 4) + i);
                a[r][4 * i] = v.x;
                a[r][4 * i + 1] = v.y;
                a[r][4 * i + 2] = v.z;
                a[r][4 * i + 3] = v.w;
            }
    };
    uint32_t qf[QREG ? KC : 1][2][QW];
    if constexpr (QREG) {
        if (w * 16 < count) {
#pragma unroll
            for (int c = 0; c < KC; ++c) load_q(c, qf[c]);
        }
    }

    // acc[c][j]: rows g, columns 64 c + 16 t + j and + 8 + j; rows g + 8 the same.
    float acc[CC][8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < CC; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[c][j][0] = acc[c][j][1] = acc[c][j][2] = acc[c][j][3] = 0.0f;

#pragma unroll 1
    for (int b0 = w * 16; b0 < count; b0 += W * 16) {
        // Lane x has key x of the block: its node and its cache row (-1: none).
        int mine = -1;
        long long at = -1;
        if (lane < 16 && b0 + lane < count) {
            mine = s.list[b0 + lane];
            const int pos = len - p.Nq + mine;
            const int page = __ldg(p.table + seq * p.table_stride + (pos >> p.page_shift));
            if (page < 0 || page >= p.num_pages) {
                atomicCAS(p.status, 0, SITE_PAGED_PAGE);
                mine = -1;
            } else {
                at = ((static_cast<long long>(page) * p.H_kv + kvh) << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
            }
        }
        // The lane's keys 2t, 2t + 1, 2t + 8, 2t + 9: rows in the cache, bits for both rows.
        long long v_at[4];
        uint32_t sees[2] = {0, 0};
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const int key = 2 * t + (y & 1) + 8 * (y >> 1);
            v_at[y] = __shfl_sync(0xffffffffu, at, key);
            const int j = __shfl_sync(0xffffffffu, mine, key);
#pragma unroll
            for (int r = 0; r < 2; ++r)
                if (j >= 0 && node[r] && ((s.vis[token[r]][j >> 5] >> (j & 31)) & 1u)) sees[r] |= 1u << y;
        }
        // ------------------------------------------------------------ S = Q K^T
        float sc[2][4];                    // keys 0 .. 8 and 8 .. 16: (row g, 2t), (row g, 2t + 1), (row g + 8, ..)
#pragma unroll
        for (int h = 0; h < 2; ++h) sc[h][0] = sc[h][1] = sc[h][2] = sc[h][3] = 0.0f;
        uint4 kv[2][KC];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const long long row = __shfl_sync(0xffffffffu, at, 8 * h + g);
            const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.k_cache) + row * ROW);
#pragma unroll
            for (int c = 0; c < KC; ++c) kv[h][c] = row >= 0 ? __ldg(src + 4 * c + t) : make_uint4(0, 0, 0, 0);
        }
        float k_scale[4], v_scale[4];
        if constexpr (FP8) {
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                k_scale[y] = v_at[y] >= 0 ? __ldg(p.k_scale + v_at[y]) : 0.0f;
                v_scale[y] = v_at[y] >= 0 ? __ldg(p.v_scale + v_at[y]) : 0.0f;
            }
        }
#pragma unroll
        for (int c = 0; c < KC; ++c) {
            uint32_t a[2][QW];
            if constexpr (QREG) {
#pragma unroll
                for (int i = 0; i < QW; ++i) a[0][i] = qf[c][0][i], a[1][i] = qf[c][1][i];
            } else {
                load_q(c, a);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t kw[4] = {kv[h][c].x, kv[h][c].y, kv[h][c].z, kv[h][c].w};
#pragma unroll
                for (int i = 0; i < QW / 2; ++i) {
                    uint32_t b0w, b1w;
                    if constexpr (FP8) {
                        b0w = codes_to_bf16x2(f16x2_of_lo(kw[i]));
                        b1w = codes_to_bf16x2(f16x2_of_hi(kw[i]));
                    } else {
                        b0w = kw[2 * i];
                        b1w = kw[2 * i + 1];
                    }
                    mma_m16n8k16<false>(sc[h], a[0][2 * i], a[1][2 * i], a[0][2 * i + 1], a[1][2 * i + 1], b0w, b1w);
                }
            }
        }
        // ------------------------------------------------------------ weights
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float& v = sc[y >> 1][2 * r + (y & 1)];
                if constexpr (FP8) v *= k_scale[y];
                v = (sees[r] >> y) & 1u ? v * p.scale_log2 : -INFINITY;
                mx[r] = fmaxf(mx[r], v);
            }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
            const float to = fmaxf(m[r], mx[r]), f = to == m[r] ? 1.0f : ex2_approx(m[r] - to);
            m[r] = to;
            l[r] *= f;
#pragma unroll
            for (int c = 0; c < CC; ++c)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    acc[c][j][2 * r] *= f;
                    acc[c][j][2 * r + 1] *= f;
                }
        }
        uint32_t loud = 0;                 // bit y: the scale of key y is not finite
        if constexpr (FP8) {
#pragma unroll
            for (int y = 0; y < 4; ++y)
                if (!(fabsf(v_scale[y]) < INFINITY)) {
                    loud |= 1u << y;
                    v_scale[y] = 0.0f;
                }
        }
        uint32_t hi[4], lo[4];             // P as the A operand: rows g, g + 8 of keys 0 .. 8, then of 8 .. 16
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float ref = m[r] == -INFINITY ? 0.0f : m[r];
                float e0 = ex2_approx(sc[h][2 * r] - ref), e1 = ex2_approx(sc[h][2 * r + 1] - ref);
                l[r] += e0 + e1;
                if constexpr (FP8) {
                    e0 *= v_scale[2 * h];
                    e1 *= v_scale[2 * h + 1];
                }
                const uint32_t top = pack_bf16x2(e0, e1);
                hi[2 * h + r] = top;
                lo[2 * h + r] = pack_bf16x2(e0 - __uint_as_float(top << 16), e1 - __uint_as_float(top & 0xffff0000u));
            }
        // ------------------------------------------------------------ O += P V
#pragma unroll
        for (int c = 0; c < CC; ++c) {
            uint32_t v[4][4];
            bool bad = false;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const uint8_t* src = static_cast<const uint8_t*>(p.v_cache) + v_at[y] * ROW;
                if constexpr (FP8) {
                    const uint2 u = v_at[y] >= 0 ? __ldg(reinterpret_cast<const uint2*>(src) + 8 * c + g) : make_uint2(0, 0);
                    v[y][0] = codes_to_bf16x2(f16x2_of_lo(u.x));
                    v[y][1] = codes_to_bf16x2(f16x2_of_hi(u.x));
                    v[y][2] = codes_to_bf16x2(f16x2_of_lo(u.y));
                    v[y][3] = codes_to_bf16x2(f16x2_of_hi(u.y));
                } else {
                    const uint4 u = v_at[y] >= 0 ? __ldg(reinterpret_cast<const uint4*>(src) + 8 * c + g) : make_uint4(0, 0, 0, 0);
                    v[y][0] = u.x;
                    v[y][1] = u.y;
                    v[y][2] = u.z;
                    v[y][3] = u.w;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) bad = bad || not_finite_bf16x2(v[y][i]);
            }
            if (__any_sync(0xffffffffu, bad)) {
#pragma unroll
                for (int y = 0; y < 4; ++y)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (not_finite_bf16x2(v[y][i])) {
                            loud |= 1u << y;
                            v[y][i] = finite_bf16x2(v[y][i]);
                        }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t sel = j & 1 ? 0x7632u : 0x5410u;
                const uint32_t b0w = __byte_perm(v[0][j / 2], v[1][j / 2], sel), b1w = __byte_perm(v[2][j / 2], v[3][j / 2], sel);
                mma_m16n8k16<false>(acc[c][j], hi[0], hi[1], hi[2], hi[3], b0w, b1w);
                mma_m16n8k16<false>(acc[c][j], lo[0], lo[1], lo[2], lo[3], b0w, b1w);
            }
        }
        if (__any_sync(0xffffffffu, loud != 0)) {
            // (lanes of one t have chunks of the same keys)
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) loud |= __shfl_xor_sync(0xffffffffu, loud, o);
#pragma unroll
            for (int r = 0; r < 2; ++r)
                if (loud & sees[r]) l[r] = __uint_as_float(0x7fc00000u);
        }
    }

    // ------------------------------------------------------------ the partial results
    wait_prerequisites();
    const int parts = p.prefix_parts + p.own_parts;
    const long long rows = static_cast<long long>(p.B) * p.Nq * p.H;
    {
        float top[2] = {m[0], m[1]};
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            if (node[r])
                for (int x = w + W * t; x < parts; x += 4 * W) top[r] = fmaxf(top[r], p.part_lse[x * rows + out[r]]);
            top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
            top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
            const float f = top[r] == m[r] ? 1.0f : ex2_approx(m[r] - top[r]);
            m[r] = top[r];
            l[r] *= f;
#pragma unroll
            for (int c = 0; c < CC; ++c)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    acc[c][j][2 * r] *= f;
                    acc[c][j][2 * r + 1] *= f;
                }
        }
    }
#pragma unroll 1
    for (int x = w; x < parts; x += W) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float lse2 = node[r] ? p.part_lse[x * rows + out[r]] : -INFINITY;
            // (an empty part's O was not written)
            if (lse2 == -INFINITY) continue;
            const float wt = ex2_approx(lse2 - m[r]);
            if (t == 0) l[r] += wt;
            const float4* src = reinterpret_cast<const float4*>(p.part_o + (x * rows + out[r]) * D);
#pragma unroll
            for (int c = 0; c < CC; ++c) {
                float4 f[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) f[i] = src[c * 16 + t * 4 + i];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float u[4] = {f[i].x, f[i].y, f[i].z, f[i].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float& o = acc[c][(i & 1) * 4 + e][2 * r + (i >> 1)];
                        o = fmaf(wt, u[e], o);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    }

    // ------------------------------------------------------------ out
    auto finish = [&](int r, float mm, float ll, auto&& value) {
        const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;           // (0: the row sees nothing)
        uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + out[r] * D);
#pragma unroll
        for (int c = 0; c < CC; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                dst[c * 8 + t * 2 + h] = make_uint4(pack_bf16x2(value(c, h, 0) * inv, value(c, h, 1) * inv),
                                                    pack_bf16x2(value(c, h, 2) * inv, value(c, h, 3) * inv),
                                                    pack_bf16x2(value(c, h, 4) * inv, value(c, h, 5) * inv),
                                                    pack_bf16x2(value(c, h, 6) * inv, value(c, h, 7) * inv));
        if (t == 0) p.lse[lse_at[r]] = ll == 0.0f ? -INFINITY : (mm + __log2f(ll)) * 0.69314718055994530942f;
    };
    if constexpr (W == 1) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
            if (row_in[r]) finish(r, m[r], l[r], [&](int c, int h, int j) { return acc[c][j][2 * r + h]; });
    } else {
        constexpr int JD = Cfg::JD;
        float* jm = join + kWarps * kRows * JD;                    // (warp, kRows)
        float* jl = jm + kWarps * kRows;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float* dst = join + (warp * kRows + g + 8 * r) * JD;
#pragma unroll
            for (int c = 0; c < CC; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<float4*>(dst + c * 64 + t * 16 + i * 4) =
                        make_float4(acc[c][(i & 1) * 4][2 * r + (i >> 1)], acc[c][(i & 1) * 4 + 1][2 * r + (i >> 1)],
                                    acc[c][(i & 1) * 4 + 2][2 * r + (i >> 1)], acc[c][(i & 1) * 4 + 3][2 * r + (i >> 1)]);
            if (t == 0) {
                jm[warp * kRows + g + 8 * r] = m[r];
                jl[warp * kRows + g + 8 * r] = l[r];
            }
        }
        __syncthreads();
        // Warp w of the tile joins the rows w * 16 / W ..: D / 8 lanes a row, eight columns each.
        constexpr int PER = kRows / W, LR = D / 8;
        const int first = warp - w;
        for (int y = lane; y < PER * LR; y += 32) {
            const int rr = w * PER + y / LR, c8 = y % LR;
            if (rr >= live) break;
            float mm = jm[first * kRows + rr];
#pragma unroll
            for (int k = 1; k < W; ++k) mm = fmaxf(mm, jm[(first + k) * kRows + rr]);
            const float ref = mm == -INFINITY ? 0.0f : mm;
            float ll = 0.0f, v[8] = {};
#pragma unroll
            for (int k = 0; k < W; ++k) {
                const float a = ex2_approx(jm[(first + k) * kRows + rr] - ref);
                ll += a * jl[(first + k) * kRows + rr];
                const float* src = join + ((first + k) * kRows + rr) * JD + c8 * 8;
                const float4 f0 = *reinterpret_cast<const float4*>(src), f1 = *reinterpret_cast<const float4*>(src + 4);
                const float u[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = fmaf(a, u[e], v[e]);
            }
            const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
            const int z = z0 + rr, i = p.by_G.div(z), h = kvh * p.G + z - i * p.G;
            const long long o = (static_cast<long long>(seq) * p.Nq + i) * p.H + h;
            reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + o * D)[c8] =
                make_uint4(pack_bf16x2(v[0] * inv, v[1] * inv), pack_bf16x2(v[2] * inv, v[3] * inv),
                           pack_bf16x2(v[4] * inv, v[5] * inv), pack_bf16x2(v[6] * inv, v[7] * inv));
            if (c8 == 0) p.lse[(seq * p.H + h) * p.Nq + i] = ll == 0.0f ? -INFINITY : (ref + __log2f(ll)) * 0.69314718055994530942f;
        }
    }
}

template <int D, bool FP8, int W>
cudaError_t launch_tree(const PagedParams& p, cudaStream_t stream) {
    using Cfg = TreeCfg<D, FP8, W>;
    auto kernel = paged_tree_kernel<D, FP8, W>;
    static std::atomic<unsigned long long> ready{0};
    cudaError_t e = once_per_device(ready, [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM_BYTES);
    });
    if (e != cudaSuccess) return e;
    const int per = (p.Nq * p.G + kRows - 1) / kRows, tiles = p.B * p.H_kv * per;
    return launch_kernel(kernel, (tiles + Cfg::TILES - 1) / Cfg::TILES, kWarps * 32, Cfg::SMEM_BYTES, true, stream, p, tiles,
                         FastDiv(per));
}

template <int D, bool FP8>
cudaError_t tree_d(const PagedParams& p, cudaStream_t stream) {
    // Warps that share a tile's rows: more for many partial results (their reading is
    // what a tile then does), one where the tiles fill the machine.
    const int parts = p.prefix_parts + p.own_parts;
    if (parts > 4) return launch_tree<D, FP8, 4>(p, stream);
    if (parts > 2) return launch_tree<D, FP8, 2>(p, stream);
    return launch_tree<D, FP8, 1>(p, stream);
}

}  // namespace

cudaError_t run_paged_tree(const PagedParams& p, cudaStream_t stream) {
    if (p.d == 64) return p.fp8 ? tree_d<64, true>(p, stream) : tree_d<64, false>(p, stream);
    if (p.d == 128) return p.fp8 ? tree_d<128, true>(p, stream) : tree_d<128, false>(p, stream);
    return p.fp8 ? tree_d<256, true>(p, stream) : tree_d<256, false>(p, stream);
}

}  // namespace attn
