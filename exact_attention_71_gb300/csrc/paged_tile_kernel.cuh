// Attention of many query rows against one key range of the paged cache, on
// the tensor cores: the shared prefix of a batch (all sequences' rows of a
// key/value head's group), and long query chunks over a sequence's own tokens.
//
//     m = max_j s_j,  l = sum_j exp2(s_j - m),  O = sum_j exp2(s_j - m) v_j / l
//     s_j = scale * log2(e) * q . k_j        (times k's row scale: e4m3 cache)
//
// A CTA takes a work item: one segment (the prefix, or one sequence's own
// tokens), one key/value head, one or two tiles of 128 query rows and a key
// range.  Two softmax warpgroups ("streams") each hold one tile's S and O in
// tensor memory.  With two row tiles (pair) both streams take every key tile;
// with one (alt) each stream takes half of the range with the same rows, so that
// one stream's softmax still runs beside the other's products, and the two
// results are joined at the end.  At d = 256 tensor memory holds one stream.
//
//   warps [0, 4 NS)       softmax (one thread per row); they also bring in Q
//   e4m3: 4 warps         convert the codes of a V tile to fp16, times the row's
//                         scale over vref (a power of two that keeps the products in
//                         fp16's range: see the streaming kernel).  The ratio and
//                         the product are rounded to fp16, 2^-11 each; with the
//                         ratio on P instead, in the softmax, a chunk of 512
//                         queries over 8192 keys took 165 us against 160.
//                         K is multiplied as it is: q is split into two e4m3
//                         parts, q = (q1 + q2) 2^shift, so that S = q1 K^T + q2 K^T
//                         in the 8-bit products that run at twice the rate.  The
//                         tensor cores add them up in 25 bits (measured: 2^-22 of
//                         sum |q k|).
//   load warp             walks the page table: a head's rows of a page are
//                         contiguous, so a bf16 tile is BN / page_size TMA boxes
//                         per 64 columns, written swizzled into a ring of half
//                         stages (K and V alternating); e4m3: K tiles likewise
//                         (per 128 columns) into a ring of their own, and V tiles
//                         as BN / page_size bulk copies into a ring of raw tiles
//   MMA warps             one per stream, issue tcgen05.mma: S = Q K^T, O += P V
//                         (one warp for both streams left the pipe idle between
//                         steps)
//
// Measured: 2048 query rows of each of 8 heads over a prefix of 65536 tokens, d =
// 128: bf16 337 us, 1630 TFLOP/s (83 % of the measured peak), 2770 cycles a step of
// two tiles, of which the products take 2740: bound by the tensor pipe (a block of
// P V and S takes 1370 cycles where the rate alone would be 1024: at N = 128 the
// operands in shared memory ask for all of its bandwidth).  e4m3 442 us, 1240
// TFLOP/s: bound by the latency of the softmax, 1800 cycles a tile where bf16 takes
// 1260 (the scales, and rows spread over four threads), which two streams do not
// hide behind 1440 cycles of products.  A CTA costs 6 us besides (query rows, first
// copies, epilogue), 9 with an e4m3 cache.
//
// The scores of rows past the range, and of a page outside the cache, are
// masked; their V rows are zeroed before a product reads them (0 times stale NaN
// would be NaN).
#pragma once

#include <cuda_bf16.h>

#include <type_traits>

#include "paged.cuh"
#include "paged_stream_kernel.cuh"
#include "sm103_bulk.cuh"
#include "sm103_ptx.cuh"

namespace attn {

enum : int {
    SITE_TILE_EMPTY = 0xa1,
    SITE_TILE_Q = 0xa2,
    SITE_TILE_FULL = 0xa3,
    SITE_TILE_P = 0xa4,
    SITE_TILE_S = 0xa5,
    SITE_TILE_O = 0xa6,
    SITE_TILE_SCALE = 0xa7,
    SITE_TILE_LOADED = 0xa8,
    SITE_TILE_DRAIN = 0xa9,
    SITE_TILE_TURN = 0xaa,
    SITE_TILE_JOIN = 0xab,
};

template <int D_, bool FP8_>
struct TileCfg {
    static constexpr int D = D_;
    static constexpr bool FP8 = FP8_;
    static constexpr int BM = 128;
    static constexpr int BN = D == 256 ? 64 : 128;
    static constexpr int NS = D == 256 ? 1 : 2;                    // streams
    static constexpr int NCB = D / 64;                             // 128-byte column boxes per row
    static constexpr int Q_BYTES = BM * D * 2;
    static constexpr int HALF_BYTES = BN * D * 2;                  // one K or V tile, 16-bit
    // bf16: one ring of K and V tiles.  e4m3: a ring of K tiles as they are, one of
    // V tiles as they are (raw) and one of V tiles in fp16.
    static constexpr int RAW_BYTES = FP8 ? BN * D : 0;
    static constexpr int NH = FP8 ? (D == 64 ? 4 : 2) : (D == 64 ? 8 : 5);
    static constexpr int NK = FP8 ? (D == 64 ? 6 : 3) : 0;
    static constexpr int NR = FP8 ? (D == 64 ? 4 : 2) : 0;
    static constexpr int SWK = D >= 128 ? 128 : 64;                // e4m3 K and q: swizzle span, 64-byte rows at d = 64
    static constexpr int SLOTS = 8;                                // key tiles whose scales are held
    static constexpr int SC_BYTES = FP8 ? SLOTS * 2 * BN * 4 : 0;
    static constexpr int DIAG_TILES = 8;
    static constexpr int CONV_WARP = 4 * NS;                       // e4m3: 4 converting warps
    static constexpr int LOAD_WARP = 4 * NS + (FP8 ? 4 : 0), MMA_WARP = LOAD_WARP + 1;   // one MMA warp per stream
    static constexpr int THREADS = NS * 128 + (FP8 ? 256 : 128);
    static constexpr int LAUNCH_REGS = 65536 / THREADS > 255 ? 248 : (65536 / THREADS) / 8 * 8;
    static constexpr int CONV_REGS = FP8 ? 80 : 0, LOW_REGS = FP8 ? 64 : 104;
    static constexpr int HIGH_RAW = (LAUNCH_REGS * THREADS - (CONV_REGS + LOW_REGS) * 128) / (NS * 128) / 8 * 8;
    static constexpr int HIGH_REGS = HIGH_RAW > 248 ? 248 : HIGH_RAW;
    static constexpr int BAR_BYTES = FP8 ? 2688 : 2048;           // (of TileBarriers)
    // Output staging: 4 KB per softmax warp, over query tiles that no product
    // reads any more (d = 64: its query tiles are too small for that).
    static constexpr int EPI_BYTES = D == 64 ? NS * 16384 : 0;
    static constexpr int SMEM_BYTES = 1024 + NS * Q_BYTES + NH * HALF_BYTES + (NK + NR) * RAW_BYTES + SC_BYTES +
                                      EPI_BYTES + BAR_BYTES;
    static_assert(HIGH_REGS * NS * 128 + (CONV_REGS + LOW_REGS) * 128 <= LAUNCH_REGS * THREADS, "register split");
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
    // A slot (validity bits, scales) is rewritten for the eighth key tile after its
    // own.  bf16: that is at least 15 ring entries after its K, when the entry NH
    // before has been released; it is past the tile's V (at most 3 entries after
    // its K).  e4m3: when the S of the tile NK before has been taken, which follows
    // P V of all tiles but the last of each stream.
    static_assert(FP8 ? 8 - NK >= 2 : 15 - NH >= 3, "scale slots");
    static_assert(NS == 1 || NH * HALF_BYTES >= BM * D * 4, "the streams' join");
};

template <bool FP8>
struct TileBarriers {
    uint64_t q_full, loaded, drain[2], fix, joined;
    uint64_t s_full[2], p_full[2], o_full[2];
    uint64_t ring_full[8], ring_empty[8];
    uint64_t raw_full[8], raw_empty[8], k_full[8], k_empty[8];
    uint64_t sc_full[8], vs_ready[8];
    uint32_t valid[8][4];          // per slot: bit per key of the tile
    // Per diagonal tile, bit per key: its V row is not finite (poison); from 8 on, e4m3:
    // it is left out of the products and added at the end (loud).
    uint32_t poison[FP8 ? 16 : 8][4];
    float most[2];                 // e4m3, streams that begin with a diagonal tile: V scales that may move vref there
    float vref[8];                 // e4m3, per slot: the slot's V scales are divided by it
    float red[2][4];               // e4m3: the converting warps' maxima
    float q_log2[FP8 ? 128 * 2 : 1];   // e4m3: raw score -> log2 units, per query row
    float lse1[128];               // alt mode: stream 1's result
    uint32_t tmem_base;
    int abort_flag;
    int turn;                      // blocks of products issued
};

// Bounded wait: false when the shared abort flag is raised or the cycle budget
// runs out (then it raises the flag and records `site`).
__device__ __forceinline__ bool tile_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                          const PagedParams& p, int site) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (true) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (static_cast<unsigned long long>(clock64() - t0) > p.wait_limit) {
            *abort_flag = 1;
            atomicCAS(p.status, 0, site);
            return false;
        }
    }
}
__device__ __forceinline__ bool tile_warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                               const PagedParams& p, int site) {
    return __all_sync(0xffffffffu, tile_wait(bar, parity, abort_flag, p, site));
}

// Bounded wait (whole warp) until `k` blocks of products have been issued.
__device__ __forceinline__ bool tile_turn(volatile int* turn, int k, volatile int* abort_flag, const PagedParams& p) {
    bool ok = true;
    if (*turn < k) {
        const long long t0 = clock64();
        while (*turn < k) {
            if (*abort_flag) {
                ok = false;
                break;
            }
            if (static_cast<unsigned long long>(clock64() - t0) > p.wait_limit) {
                *abort_flag = 1;
                atomicCAS(p.status, 0, SITE_TILE_TURN);
                ok = false;
                break;
            }
        }
    }
    return __all_sync(0xffffffffu, ok);
}

// Teardown wait for the CTA's own asynchronous work, which always completes: it
// ignores the abort flag and lasts at least a second.
__device__ __forceinline__ void tile_drain(uint64_t* bar, uint32_t parity, const PagedParams& p, int site) {
    const unsigned long long lim = p.wait_limit > 2000000000ull ? p.wait_limit : 2000000000ull;
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity)) {
        if (static_cast<unsigned long long>(clock64() - t0) > lim) {
            atomicCAS(p.status, 0, site);
            return;
        }
    }
}

// Byte offset of 16-byte chunk c of row r in a swizzled K / V tile.
template <class Cfg>
__device__ __forceinline__ uint32_t tile_offset(int r, int c) { 
    return static_cast<uint32_t>((c >> 3) * (Cfg::BN * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// One warp's pass over a bf16 V tile in shared memory: rows that were not
// copied, or lie past the range (row >= len), become 0; in rows from `diag` on
// infinities and NaN become 0 and the row's bit in poison is set.
template <class Cfg>
__device__ __noinline__ void fix_v_tile(uint8_t* tile, uint32_t copies, int log2_box, int len, int diag,
                                        uint32_t* poison, int lane) {
    constexpr int CPR = Cfg::D / 8, LPR = CPR < 32 ? CPR : 32;     // 16-byte chunks, lanes of a row
    // Rows below `from` are as they should be.
    int from = max(min(len, diag), 0);
    const uint32_t missing = ~copies & ((1u << (Cfg::BN >> log2_box)) - 1u);
    if (missing) from = min(from, (__ffs(missing) - 1) << log2_box);
    // One warp does this while the products wait, so the usual case, finite rows, is
    // kept short: eight row groups at a time (latency), and 2^7 added to an
    // exponent field of ones carries into the sign bit.  (A row group after the
    // other, with comparisons, held up a tile of 128 rows by 12000 cycles.)
    constexpr int AT = 8, RPI = 32 / LPR;
    for (int r0 = from + lane / LPR; r0 < Cfg::BN; r0 += AT * RPI) {
#pragma unroll
        for (int c = lane % LPR; c < CPR; c += LPR) {
            uint4 v[AT];
#pragma unroll
            for (int i = 0; i < AT; ++i) {
                const int r = r0 + i * RPI;
                const bool have = r < len && r < Cfg::BN && ((copies >> (r >> log2_box)) & 1u);
                if (have) v[i] = *reinterpret_cast<const uint4*>(tile + tile_offset<Cfg>(r, c));
                else v[i] = make_uint4(0, 0, 0, 0);
                if (!have && r < Cfg::BN) *reinterpret_cast<uint4*>(tile + tile_offset<Cfg>(r, c)) = v[i];
            }
            uint32_t bad[AT], any = 0;
#pragma unroll
            for (int i = 0; i < AT; ++i) {
                const uint32_t* w = &v[i].x;
                bad[i] = 0;
#pragma unroll
                for (int y = 0; y < 4; ++y) bad[i] |= (w[y] & 0x7f807f80u) + 0x00800080u;
                any |= bad[i];
            }
            if (any & 0x80008000u) {
#pragma unroll
                for (int i = 0; i < AT; ++i) {
                    const int r = r0 + i * RPI;
                    if (!(bad[i] & 0x80008000u) || r < diag) continue;
                    uint32_t* w = &v[i].x;
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        if ((w[y] & 0x7f80u) == 0x7f80u) w[y] &= 0xffff0000u;
                        if ((w[y] & 0x7f800000u) == 0x7f800000u) w[y] &= 0xffffu;
                    }
                    *reinterpret_cast<uint4*>(tile + tile_offset<Cfg>(r, c)) = v[i];
                    atomicOr(&poison[r >> 5], 1u << (r & 31));
                }
            }
        }
    }
    __syncwarp();
}

// Lane r's value of row r, from the accumulator layout (v[i] of the threads
// 4 q .. 4 q + 3 belongs to row q + 8 i).
__device__ __forceinline__ float to_row(const float (&v)[4], int lane) {
    float r = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float x = __shfl_sync(0xffffffffu, v[i], (lane & 7) * 4);
        if ((lane >> 3) == i) r = x;
    }
    return r;
}

// What a CTA computes; every role derives it alike.
struct TileItem {
    bool prefix, pair;
    int seq, kvh;
    int rows;            // query rows of the segment for this head
    int rt[2];           // row tile of each stream (-1: none)
    int part;            // part index of the result
    int j0[2], n[2];     // first key tile and number of key tiles of each stream
    int len;             // keys of the segment
    const int* table;
};

// Keys that row r of the segment sees.
__device__ __forceinline__ int row_limit(const PagedParams& p, const TileItem& w, int r) {
    if (w.prefix || !p.causal) return w.len;
    return max(0, w.len - p.Nq + 1 + static_cast<int>(p.by_G.div(r)));
}

template <class Cfg>
__device__ __forceinline__ TileItem tile_item(const PagedParams& p) {
    TileItem w;
    unsigned x = blockIdx.x;
    w.prefix = x < static_cast<unsigned>(p.prefix_items);
    if (!w.prefix) x -= p.prefix_items;
    const int per = p.Nq * p.G;
    w.rows = w.prefix ? p.B * per : per;
    const int tiles = (w.rows + Cfg::BM - 1) / Cfg::BM;
    w.pair = Cfg::NS == 2 && tiles > 1;
    // Row groups of the same keys run next to one another.
    const FastDiv by_groups = w.prefix ? p.by_prefix_groups : p.by_own_groups;
    const FastDiv by_ctas = w.prefix ? p.by_prefix_parts : p.by_own_parts;
    unsigned y = by_groups.div(x);
    const int group = by_groups.d - 1 - (x - y * by_groups.d);     // (those that see the most keys first)
    x = p.by_heads.div(y);
    w.kvh = y - x * p.H_kv;
    y = by_ctas.div(x);
    const int split = x - y * by_ctas.d;
    w.seq = w.prefix ? 0 : y;
    w.table = w.prefix ? p.prefix_table : p.table + w.seq * p.table_stride;
    int len = p.prefix_len;
    if (!w.prefix) {
        len = max(0, __ldg(p.seq_lens + w.seq));
        const long long room = static_cast<long long>(p.max_pages) << p.page_shift;
        if (len > room) {
            if (threadIdx.x == 0) atomicCAS(p.status, 0, SITE_PAGED_LENGTH);
            len = static_cast<int>(room);
        }
    }
    w.len = len;
    w.part = (w.prefix ? 0 : p.prefix_parts) + split;
    // Even shares of the key tiles; the first `more` have one tile more.
    const int all = (len + Cfg::BN - 1) / Cfg::BN;
    const bool two = Cfg::NS == 2 && !w.pair;
    const FastDiv by_shares = w.prefix ? p.by_prefix_shares : p.by_own_shares;
    const int least = by_shares.div(all), more = all - least * static_cast<int>(by_shares.d);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        if (t >= Cfg::NS) {
            w.rt[t] = -1;
            w.j0[t] = w.n[t] = 0;
            continue;
        }
        w.rt[t] = w.pair ? group * 2 + t : group;
        if (w.rt[t] >= tiles) w.rt[t] = -1;
        const int share = two ? 2 * split + t : split;
        w.j0[t] = least * share + min(share, more);
        int j1 = w.j0[t] + least + (share < more ? 1 : 0);
        if (w.rt[t] >= 0) {
            // Tiles past what the tile's last row sees are left out.
            const int last = min(w.rt[t] * Cfg::BM + Cfg::BM, w.rows) - 1;
            j1 = min(j1, (row_limit(p, w, last) + Cfg::BN - 1) / Cfg::BN);
        }
        w.n[t] = w.rt[t] >= 0 ? max(0, j1 - w.j0[t]) : 0;
    }
    return w;
}

// Calls f(stream, u, is_v) for every ring entry in order: in pair mode K_u, V_u
// of the shared tiles; in alt mode the streams' entries in the order in which
// the products use them.
template <class Cfg, class F>
__device__ __forceinline__ void tile_entries(const TileItem& w, F&& f) {
    if (w.pair || Cfg::NS == 1) {
        const int n = max(w.n[0], w.n[1]);
        for (int u = 0; u < n; ++u) {
            if (!f(0, u, false) || !f(0, u, true)) return;
        }
    } else {
        const int n = max(w.n[0], w.n[1]);
        for (int u = 0; u <= n; ++u) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (u >= 1 && u <= w.n[t] && !f(t, u - 1, true)) return;
                if (u < w.n[t] && !f(t, u, false)) return;
            }
        }
    }
}

// Ring index of stream t's V_(u-1) (is_v) or K_u in tile_entries order.
template <class Cfg>
__device__ __forceinline__ uint32_t tile_entry(const TileItem& w, int t, int u, bool is_v) {
    if (w.pair || Cfg::NS == 1) return is_v ? 2 * u - 1 : 2 * u;
    const int b = max(u - 1, 0);
    int x = min(b, w.n[0]) + min(u, w.n[0]) + min(b, w.n[1]) + min(u, w.n[1]);      // rounds before u
    const int v0 = u >= 1 && u <= w.n[0], k0 = u < w.n[0], v1 = u >= 1 && u <= w.n[1];
    if (t == 1) x += v0 + k0;
    if (!is_v) x += t == 0 ? v0 : v1;
    return static_cast<uint32_t>(x);
}

// Position of stream t's key tile u among the K entries (its scale slot).
template <class Cfg>
__device__ __forceinline__ int tile_slot(const TileItem& w, int t, int u) {
    if (w.pair || Cfg::NS == 1) return u;
    return u + (t == 0 ? min(u, w.n[1]) : min(u + 1, w.n[0]));
}

// Whether a V row of the keys [lo, hi) is not finite (whole warp; rows of pages
// outside the cache, which are hidden, do not count).
template <class Cfg>
__device__ __forceinline__ bool v_rows_not_finite(const PagedParams& p, const TileItem& w, int lo, int hi, int lane) {
    constexpr int CPR = Cfg::FP8 ? Cfg::D / 16 : Cfg::D / 8;       // 16-byte chunks of a row (32 at most)
    bool bad = false;
#pragma unroll 1
    for (int key = lo + lane / CPR; key < hi; key += 32 / CPR) {
        const int page = __ldg(w.table + (key >> p.page_shift));
        if (page < 0 || page >= p.num_pages) continue;
        const long long at = ((static_cast<long long>(page) * p.H_kv + w.kvh) << p.page_shift) + (key & ((1 << p.page_shift) - 1));
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.v_cache) + at * (CPR * 16)) + lane % CPR);
        const uint32_t* x = &v.x;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            if constexpr (Cfg::FP8) bad |= __vcmpeq4(x[y] & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0;
            else bad |= (((x[y] & 0x7f807f80u) + 0x00800080u) & 0x80008000u) != 0;
        }
        if constexpr (Cfg::FP8) bad |= !(__ldg(p.v_scale + at) < INFINITY);
    }
    return __any_sync(0xffffffffu, bad);
}

// O of a warp's rows, one a lane, comes in units of vref and leaves in units of
// kLoudUnit (a weight may be 2^15), with the values of the loud keys of the tiles
// [x0, x1) that each row sees: weights exp2(s - m) from the cache, in binary32.  Whole
// warp; out: the row's index in q, limit: the keys that it sees.
constexpr float kLoudUnit = 0x1p20f;
template <class Cfg>
__device__ __noinline__ void add_loud(const PagedParams& p, const int* table, int kvh, const uint32_t (*loud)[4], int diag,
                                      int x0, int x1, int limit, int out, float m, float vref, uint32_t o_tmem) {
    constexpr int D = Cfg::D;
    auto update = [&](auto&& f) {
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(o_tmem + c * 32, o);
            tmem_wait_ld();
            reg_fence32(o);
#pragma unroll
            for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(f(c * 32 + y, __uint_as_float(o[y])));
            tmem_st32(o_tmem + c * 32, o);
            tmem_wait_st();
        }
    };
    update([&](int, float o) { return o * (vref * (1.0f / kLoudUnit)); });
#pragma unroll 1
    for (int x = x0; x < x1; ++x) {
#pragma unroll 1
        for (int c = 0; c < Cfg::BN / 32; ++c) {
#pragma unroll 1
            for (uint32_t bits = loud[min(x - diag, Cfg::DIAG_TILES - 1)][c]; bits; bits &= bits - 1) {
                const int key = x * Cfg::BN + c * 32 + __ffs(bits) - 1;
                const long long at = ((static_cast<long long>(__ldg(table + (key >> p.page_shift))) * p.H_kv + kvh) << p.page_shift) +
                                     (key & ((1 << p.page_shift) - 1));
                const uint32_t* kc = reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(p.k_cache) + at * D);
                const uint32_t* vc = reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(p.v_cache) + at * D);
                float e = 0.0f;
                if (key < limit) {
                    const uint2* q = reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.q) + static_cast<long long>(out) * D);
                    float dot = 0.0f;
#pragma unroll 1
                    for (int y = 0; y < D / 4; ++y) dot = dot4(__ldg(q + y), __ldg(kc + y), dot);
                    e = ex2_approx(dot * __ldg(p.k_scale + at) * p.scale_log2 - m) * (__ldg(p.v_scale + at) * (1.0f / kLoudUnit));
                }
                __syncwarp();
                // (a row that does not see the key keeps what it has)
                update([&](int y, float o) {
                    const uint32_t codes = __ldg(vc + y / 4);
                    const float2 v = f16x2_to_float2(y & 2 ? f16x2_of_hi(codes) : f16x2_of_lo(codes));
                    return e == 0.0f ? o : fmaf(e, y & 1 ? v.y : v.x, o);
                });
            }
        }
    }
}

template <class Cfg, bool DIRECT>
__global__ void __launch_bounds__(Cfg::THREADS, 1)
    paged_tile_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                      const __grid_constant__ PagedParams p) {
    constexpr int D = Cfg::D, BN = Cfg::BN, BM = Cfg::BM, NS = Cfg::NS, NH = Cfg::NH;
    constexpr bool FP8 = Cfg::FP8;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sQ = smem;
    uint8_t* sRing = smem + NS * Cfg::Q_BYTES;
    uint8_t* sK = sRing + NH * Cfg::HALF_BYTES;                // e4m3: K tiles
    uint8_t* sRaw = sK + Cfg::NK * Cfg::RAW_BYTES;             // e4m3: V tiles
    float* sScale = reinterpret_cast<float*>(sRaw + Cfg::NR * Cfg::RAW_BYTES);     // (slot, k / v, BN)
    uint8_t* sEpi = reinterpret_cast<uint8_t*>(sScale) + Cfg::SC_BYTES;            // d = 64: output staging
    using Barriers = TileBarriers<FP8>;
    static_assert(sizeof(Barriers) <= Cfg::BAR_BYTES, "barrier block");
    Barriers* bars = reinterpret_cast<Barriers*>(sEpi + Cfg::EPI_BYTES);
    volatile int* abort_flag = &bars->abort_flag;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    launch_dependents();           // (nothing of this call that follows reads what precedes it)
    const TileItem w = tile_item<Cfg>(p);
    // From this key on the CTA's rows may see different keys; its tile.
    int diag_key = w.len;
    if (!w.prefix && p.causal) diag_key = row_limit(p, w, max(w.rt[0], 0) * BM);
    const int diag = diag_key < w.len ? diag_key / BN : w.len / BN + 1;

    // Softmax threads: their query row.
    const int stream = warp >> 2;
    const int row = (stream == 0 ? w.rt[0] : w.rt[1]) * BM + (tid & 127);
    bool in = false;
    int out = -1, lse_at = 0;      // row index in q, o and the partials; in lse
    if (warp < 4 * NS) {
        in = (stream == 0 ? w.rt[0] : w.rt[1]) >= 0 && row < w.rows;
        if (in) {
            const int per = p.Nq * p.G;
            const int y = w.prefix ? p.by_per.div(row) : 0, z = row - y * per;             // row z of its sequence
            const int b = w.prefix ? y : w.seq, i = p.by_G.div(z);
            const int h = w.kvh * p.G + z - i * p.G;
            out = (b * p.Nq + i) * p.H + h;
            lse_at = (b * p.H + h) * p.Nq + i;
        }
    }
    if (tid == Cfg::LOAD_WARP * 32) {
        mbar_init(&bars->q_full, NS * 128);
        mbar_init(&bars->loaded, 1);
        mbar_init(&bars->fix, 1);
        mbar_init(&bars->joined, 128);
        for (int t = 0; t < 2; ++t) {
            mbar_init(&bars->drain[t], 1);
            mbar_init(&bars->s_full[t], 1);
            mbar_init(&bars->p_full[t], 128);
            mbar_init(&bars->o_full[t], 1);
        }
        for (int s = 0; s < 8; ++s) {
            mbar_init(&bars->ring_full[s], FP8 ? 128 : 1);
            mbar_init(&bars->ring_empty[s], w.pair ? 2 : 1);       // the MMA warps that use an entry
            mbar_init(&bars->raw_full[s], 1);
            mbar_init(&bars->raw_empty[s], 128);
            mbar_init(&bars->k_full[s], 1);
            mbar_init(&bars->k_empty[s], w.pair ? 2 : 1);
            mbar_init(&bars->sc_full[s], 1);
            mbar_init(&bars->vs_ready[s], 128);
            for (int x = 0; x < 4; ++x) {
                bars->poison[s][x] = 0;
                if (FP8) bars->poison[FP8 ? 8 + s : 0][x] = 0;
            }
        }
        bars->abort_flag = 0;
        bars->turn = 0;
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    if (warp == Cfg::MMA_WARP) {
        tmem_alloc(&bars->tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;

    if (warp >= Cfg::LOAD_WARP) {
        regs_decrease<Cfg::LOW_REGS>();
        if (warp >= Cfg::MMA_WARP && warp < Cfg::MMA_WARP + NS) {
            // -------------------------------------------------------- MMA issuers
            // Step u of a stream: O += P(u-1) V(u-1), then S(u), as one block.
            // The streams' blocks go to the tensor pipe in turns, so that one
            // stream's softmax runs beside the other's block (without turns the
            // two interleave, finish together and leave the pipe idle while both
            // exponentiate: 3350 cycles a step; 2750 with them, of which the
            // products, at 1370 cycles a block, take all but a few).  P comes
            // last and is awaited last: a block starts as soon as it is there.  In pair mode both warps release every
            // ring entry, always after waiting for it.
            constexpr uint32_t fmt = FP8 ? 0u : 1u;            // fp16 or bf16 operands
            constexpr uint32_t idesc_s = make_idesc(FP8 ? 0u : 1u, 128, BN, 0), idesc_o = make_idesc(fmt, 128, D, 1);
            const int t = warp - Cfg::MMA_WARP;
            const int nt = t == 0 ? w.n[0] : w.n[1];
            const int rounds = max(w.n[0], w.n[1]);
            const int n = w.pair ? rounds : nt;
            const uint32_t ring = smem_u32(sRing);
            const uint32_t s_tmem = tmem + t * 128, o_tmem = tmem + 256 + t * D;
            constexpr int SWQ = FP8 ? Cfg::SWK : 128;
            const uint64_t qd = sdesc_swz<SWQ>(smem_u32(sQ) + (w.pair ? t : 0) * Cfg::Q_BYTES, 16, 8 * SWQ);
            constexpr uint32_t NKR = FP8 ? Cfg::NK : NH;           // K's ring
            uint64_t* const k_full = FP8 ? bars->k_full : bars->ring_full;
            uint64_t* const k_empty = FP8 ? bars->k_empty : bars->ring_empty;
            volatile int* turn = &bars->turn;
            bool ok = n == 0 || tile_warp_wait(&bars->q_full, 0, abort_flag, p, SITE_TILE_Q);
            for (int u = 0; u <= rounds && ok; ++u) {
                const bool has_v = u > 0 && u <= n, has_k = u < n;
                const uint32_t xv = FP8 ? tile_slot<Cfg>(w, t, max(u - 1, 0)) : tile_entry<Cfg>(w, t, u, true);
                const uint32_t xk = FP8 ? tile_slot<Cfg>(w, t, u) : tile_entry<Cfg>(w, t, u, false);
                if (has_v) ok = tile_warp_wait(&bars->ring_full[xv % NH], (xv / NH) & 1, abort_flag, p, SITE_TILE_FULL);
                if (ok && has_k) ok = tile_warp_wait(&k_full[xk % NKR], (xk / NKR) & 1, abort_flag, p, SITE_TILE_FULL);
                if (NS > 1 && ok) ok = tile_turn(turn, 2 * u + t, abort_flag, p);
                if (ok && u > 0 && u <= nt) ok = tile_warp_wait(&bars->p_full[t], (u - 1) & 1, abort_flag, p, SITE_TILE_P);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    if (has_v) {
                        if (u <= nt) {
                            const uint64_t vd = sdesc_sw128(ring + (xv % NH) * Cfg::HALF_BYTES, BN * 128, 1024);
#pragma unroll
                            for (int kk = 0; kk < BN / 16; ++kk)
                                mma_f16_ts(o_tmem, s_tmem + kk * 8, vd + ((kk * 16 * 128) >> 4), idesc_o,
                                           (kk > 0 || u > 1) ? 1u : 0u);
                            if (u == nt) mma_commit(&bars->o_full[t]);
                            mma_commit(&bars->ring_empty[xv % NH]);
                        } else {
                            mbar_arrive(&bars->ring_empty[xv % NH]);
                        }
                    }
                    if (has_k) {
                        if (u < nt) {
                            const uint64_t kd = FP8 ? sdesc_swz<SWQ>(smem_u32(sK) + (xk % NKR) * Cfg::RAW_BYTES, 16, 8 * SWQ)
                                                    : sdesc_sw128(ring + (xk % NKR) * Cfg::HALF_BYTES, 16, 1024);
                            // 32 bytes of a row per instruction; e4m3: both parts of q.
                            constexpr int KPB = SWQ / 32, STEPS = FP8 ? D / 32 : D / 16;
#pragma unroll
                            for (int z = 0; z < (FP8 ? 2 : 1); ++z)
#pragma unroll
                                for (int kk = 0; kk < STEPS; ++kk) {
                                    const uint32_t a = z * (BM * D) + (kk / KPB) * (BM * SWQ) + (kk % KPB) * 32;
                                    const uint32_t b = (kk / KPB) * (BN * SWQ) + (kk % KPB) * 32;
                                    if constexpr (FP8)
                                        mma_f8_ss(s_tmem, qd + (a >> 4), kd + (b >> 4), idesc_s, z + kk > 0 ? 1u : 0u);
                                    else
                                        mma_f16_ss(s_tmem, qd + (a >> 4), kd + (b >> 4), idesc_s, kk > 0 ? 1u : 0u);
                                }
                            mma_commit(&bars->s_full[t]);
                            mma_commit(&k_empty[xk % NKR]);
                        } else {
                            mbar_arrive(&k_empty[xk % NKR]);
                        }
                    }
                    if (NS > 1) {
                        __threadfence_block();
                        *turn = 2 * u + t + 1;
                    }
                }
                __syncwarp();
            }
            // Every MMA issued here has finished before teardown.
            if (elect_one()) {
                mma_commit(&bars->drain[t]);
                tile_drain(&bars->drain[t], 0, p, SITE_TILE_DRAIN);
            }
            __syncwarp();
        }
        if (warp == Cfg::LOAD_WARP) {
            // -------------------------------------------------------- load warp
            const int ps = 1 << p.page_shift;
            const int box = min(ps, BN), boxes = BN / box;      // rows of a copy; copies of a tile (per 64 columns)
            const uint64_t pol = l2_policy_evict_last();
            uint32_t e = 0, ktiles = 0, fixes = 0;
            // Lane x < boxes looks up the page of copy x, a tile ahead; V's entry
            // uses its K's.
            auto page_of = [&](int t, int u) -> int {
                const int key = ((t == 0 ? w.j0[0] : w.j0[1]) + u) * BN + lane * box;
                const bool any = u < (w.pair ? max(w.n[0], w.n[1]) : t == 0 ? w.n[0] : w.n[1]);
                return any && lane < boxes && key < w.len ? __ldg(w.table + (key >> p.page_shift)) : -1;
            };
            if (FP8 && lane < NS) {
                // (a stream that begins with a diagonal tile: see the converting warps)
                const int key = (lane == 0 ? w.j0[0] : w.j0[1]) * BN;
                float v = 0.0f;
                if (key / BN >= diag && key < w.len) {
                    const int page = __ldg(w.table + (key >> p.page_shift));
                    if (page >= 0 && page < p.num_pages)
                        v = __ldg(p.v_scale + (((static_cast<long long>(page) * p.H_kv + w.kvh) << p.page_shift) + (key & (ps - 1))));
                }
                bars->most[lane] = v < INFINITY ? 16.0f * v : 0.0f;
            }
            __syncwarp();
            int page0 = -1, page1 = -1, next0 = page_of(0, 0), next1 = NS > 1 && !w.pair ? page_of(1, 0) : -1;
            tile_entries<Cfg>(w, [&](int t, int u, bool is_v) -> bool {
                const int key0 = ((t == 0 ? w.j0[0] : w.j0[1]) + u) * BN;
                const int key = key0 + lane * box;
                if (!is_v) {
                    if (t == 0) {
                        page0 = next0;
                        next0 = page_of(0, u + 1);
                    } else {
                        page1 = next1;
                        next1 = page_of(1, u + 1);
                    }
                }
                const int page = t == 0 ? page0 : page1;
                const bool want = lane < boxes && key < w.len;
                const bool have = want && page >= 0 && page < p.num_pages;
                const uint32_t copies = __ballot_sync(0xffffffffu, have);
                const int row = key & (ps - 1);
                const uint32_t kt = tile_slot<Cfg>(w, t, u), slot = kt % Cfg::SLOTS;
                constexpr uint32_t NK = FP8 ? Cfg::NK : 1, NR = FP8 ? Cfg::NR : 1;
                uint64_t* gate = !FP8 ? &bars->ring_empty[e % NH] : is_v ? &bars->raw_empty[kt % NR] : &bars->k_empty[kt % NK];
                const uint32_t round = !FP8 ? e / NH : is_v ? kt / NR : kt / NK;
                if (!tile_warp_wait(gate, (round & 1) ^ 1, abort_flag, p, SITE_TILE_EMPTY)) return false;
                if (!is_v) {
                    // Validity of the tile's keys (the slot is free: see SLOTS).
                    if (want && !have) atomicCAS(p.status, 0, SITE_PAGED_PAGE);
                    if (lane < BN / 32) {
                        uint32_t bits = 0;
                        if (box >= 32) bits = (copies >> (lane * 32 / box)) & 1u ? 0xffffffffu : 0u;
                        else bits = ((copies >> (2 * lane)) & 1u ? 0xffffu : 0u) | ((copies >> (2 * lane + 1)) & 1u ? 0xffff0000u : 0u);
                        const int n = min(max(w.len - key0 - lane * 32, 0), 32);
                        bars->valid[slot][lane] = bits & (n == 32 ? 0xffffffffu : (1u << n) - 1u);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive_expect_tx(&bars->sc_full[slot], FP8 ? __popc(copies) * box * 8 : 0);
                    __syncwarp();
                    if constexpr (FP8) {
                        if (have) {
                            const long long at = ((static_cast<long long>(page) * p.H_kv + w.kvh) << p.page_shift) + row;
                            float* dst = sScale + slot * 2 * BN + lane * box;
                            bulk_load(dst, p.k_scale + at, box * 4, &bars->sc_full[slot]);
                            bulk_load(dst + BN, p.v_scale + at, box * 4, &bars->sc_full[slot]);
                        }
                    }
                    ++ktiles;
                }
                if constexpr (FP8) {
                    uint64_t* full = is_v ? &bars->raw_full[kt % NR] : &bars->k_full[kt % NK];
                    if (lane == 0) mbar_arrive_expect_tx(full, __popc(copies) * box * D);
                    __syncwarp();
                    if (have) {
                        if (is_v) {
                            const long long at = ((static_cast<long long>(page) * p.H_kv + w.kvh) << p.page_shift) + row;
                            bulk_load(sRaw + (kt % NR) * Cfg::RAW_BYTES + lane * box * D,
                                      static_cast<const uint8_t*>(p.v_cache) + at * D, box * D, full);
                        } else {
                            uint8_t* tile = sK + (kt % NK) * Cfg::RAW_BYTES;
#pragma unroll
                            for (int cb = 0; cb < D / Cfg::SWK; ++cb)
                                tma_load_4d(tile + cb * (BN * Cfg::SWK) + lane * box * Cfg::SWK, &tmap_k, full, cb * Cfg::SWK, row,
                                            w.kvh, page, pol);
                        }
                    }
                } else {
                    // A V tile with rows that must not reach the product as they
                    // are: past the range, of a refused page, or not finite where
                    // only some query rows see them.
                    const bool fix = is_v && (key0 + BN > w.len || __popc(copies) != boxes || key0 / BN >= diag);
                    uint64_t* full = fix ? &bars->fix : &bars->ring_full[e % NH];
                    uint8_t* tile = sRing + (e % NH) * Cfg::HALF_BYTES;
                    if (lane == 0) mbar_arrive_expect_tx(full, __popc(copies) * box * D * 2);
                    __syncwarp();
                    if (have) {
#pragma unroll
                        for (int cb = 0; cb < Cfg::NCB; ++cb)
                            tma_load_4d(tile + cb * (BN * 128) + lane * box * 128, is_v ? &tmap_v : &tmap_k, full, cb * 64,
                                        row, w.kvh, page, pol);
                    }
                    if (fix) {
                        __syncwarp();
                        tile_drain(&bars->fix, fixes++ & 1, p, SITE_TILE_LOADED);
                        fix_v_tile<Cfg>(tile, copies, __ffs(box) - 1, w.len - key0, max(diag_key - key0, 0),
                                        bars->poison[min(max(key0 / BN - diag, 0), Cfg::DIAG_TILES - 1)], lane);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bars->ring_full[e % NH]);
                    }
                }
                __syncwarp();
                ++e;
                return true;
            });
            if (lane == 0) mbar_arrive(&bars->loaded);
            // Every copy issued here lands before the CTA can exit (on the normal
            // path these phases have completed already).
            if constexpr (FP8) {
                constexpr uint32_t NK = FP8 ? Cfg::NK : 1, NR = FP8 ? Cfg::NR : 1;
                const uint32_t vtiles = e - ktiles;
                for (uint32_t x = vtiles > NR ? vtiles - NR : 0; x < vtiles; ++x)
                    tile_drain(&bars->raw_full[x % NR], (x / NR) & 1, p, SITE_TILE_DRAIN);
                for (uint32_t x = ktiles > NK ? ktiles - NK : 0; x < ktiles; ++x)
                    tile_drain(&bars->k_full[x % NK], (x / NK) & 1, p, SITE_TILE_DRAIN);
                for (uint32_t x = ktiles > Cfg::SLOTS ? ktiles - Cfg::SLOTS : 0; x < ktiles; ++x)
                    tile_drain(&bars->sc_full[x % Cfg::SLOTS], (x / Cfg::SLOTS) & 1, p, SITE_TILE_DRAIN);
            } else {
                for (uint32_t x = e > NH ? e - NH : 0; x < e; ++x)
                    tile_drain(&bars->ring_full[x % NH], (x / NH) & 1, p, SITE_TILE_DRAIN);
            }
        }
    } else if (FP8 && warp >= Cfg::CONV_WARP) {
        regs_decrease<Cfg::CONV_REGS>();
        if constexpr (FP8) {
            // ---------------------------------------------------- converting warps
            // A thread's chunks (16 codes, column c) lie in rows r0 + i * RPP.  Its two
            // stores per chunk go to 16-byte columns 2c and 2c + 1 of the swizzle;
            // threads with c % 8 >= 4 do the second first, so that a quarter
            // warp's store covers all eight columns once.
            constexpr int CPR = D / 16;                         // chunks of a row
            constexpr int RPP = 128 / CPR;                      // rows per pass of the 128 threads
            const int ct = tid - Cfg::CONV_WARP * 32;
            const int c = ct % CPR, r0 = ct / CPR;
            const bool odd = D != 64 && (c & 4);
            float vref0 = 0.0f, vref1 = 0.0f;                   // per stream (pair: the first)
            tile_entries<Cfg>(w, [&](int t, int u, bool is_v) -> bool {
                if (!is_v) return true;
                constexpr uint32_t NR = Cfg::NR;
                const uint32_t e = tile_slot<Cfg>(w, t, u), slot = e % Cfg::SLOTS;
                const int key0 = ((t == 0 ? w.j0[0] : w.j0[1]) + u) * BN;
                // The tile's V scales, divided by the stream's vref (which follows
                // their maximum).  0 for keys that are not there (stale) and where
                // only some query rows see a key with a NaN scale: those rows learn
                // it from the poison bits, since a weight of 0 beside it must stay
                // 0.  A scale that only some rows see must not move vref, in which the
                // others' weights would vanish: its key is left out (loud), and the
                // rows that see it add its values at the end.  In a stream's first
                // tile vref may follow up to 16 times the scale of its first key,
                // which every row sees that sees one of the stream's: that is still
                // below it.  Every thread reaches the one barrier of a tile,
                // whatever its waits say; all leave together.
                bool ok = tile_wait(&bars->sc_full[slot], (e / Cfg::SLOTS) & 1, abort_flag, p, SITE_TILE_SCALE);
                const uint32_t* valid = bars->valid[slot];
                uint32_t all = valid[0] & valid[1];
                if constexpr (BN == 128) all &= valid[2] & valid[3];
                const bool whole = all == 0xffffffffu;
                const bool diagonal = key0 / BN >= diag;
                uint32_t* poison = bars->poison[min(max(key0 / BN - diag, 0), Cfg::DIAG_TILES - 1)];
                float v = 0.0f;
                if (ct < BN && ((valid[ct >> 5] >> (ct & 31)) & 1u)) {
                    v = sScale[slot * 2 * BN + BN + ct];
                    if (diagonal && key0 + ct >= diag_key) {
                        const float ref = w.pair || t == 0 ? vref0 : vref1;
                        const float most = fmaxf(64.0f * ref, bars->most[t]);
                        if (!(v <= most)) {
                            atomicOr(&poison[(v < INFINITY ? 32 : 0) + (ct >> 5)], 1u << (ct & 31));
                            v = 0.0f;
                        }
                    }
                }
                const uint32_t top = __reduce_max_sync(0xffffffffu, v > 0.0f && v < INFINITY ? __float_as_uint(v) : 0u);
                if (lane == 0) bars->red[e & 1][ct >> 5] = __uint_as_float(top);
                if (!named_barrier_and(1, 128, ok)) return false;
                {
                    const float* red = bars->red[e & 1];
                    const float vm = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
                    float ref = w.pair || t == 0 ? vref0 : vref1;
                    if (vm > 64.0f * ref) ref = vref_of(vm);
                    if (w.pair || t == 0) vref0 = ref;
                    else vref1 = ref;
                    if (ct < BN) sScale[slot * 2 * BN + BN + ct] = v * (ref == 0.0f ? 0.0f : 1.0f / ref);
                    if (ct == 0) bars->vref[slot] = ref;
                    mbar_arrive(&bars->vs_ready[slot]);
                }
                if (!tile_wait(&bars->raw_full[e % NR], (e / NR) & 1, abort_flag, p, SITE_TILE_FULL)) ok = false;
                if (ok && !tile_wait(&bars->ring_empty[e % NH], ((e / NH) & 1) ^ 1, abort_flag, p, SITE_TILE_EMPTY)) ok = false;
                if (!named_barrier_and(1, 128, ok)) return false;
                const uint8_t* src = sRaw + (e % NR) * Cfg::RAW_BYTES + r0 * D + c * 16;
                uint8_t* dst = sRing + (e % NH) * Cfg::HALF_BYTES;
                const float* vs = sScale + slot * 2 * BN + BN;
                // (d < 256: two chunks at a time.  The kernel is at the limit of the
                // instruction caches: a chunk of 512 queries over 8192 keys took 151 us
                // with all eight unrolled, 139.6 with two.)
                auto convert = [&](auto check) {
#pragma unroll (D == 256 ? BN / RPP : 2)
                    for (int i = 0; i < BN / RPP; ++i) {
                        const int r = r0 + i * RPP;
                        uint4 v = *reinterpret_cast<const uint4*>(src + i * RPP * D);
                        if constexpr (decltype(check)::value) {
                            if (!((valid[r >> 5] >> (r & 31)) & 1u)) v = make_uint4(0, 0, 0, 0);
                            if (diagonal && key0 + r >= diag_key) {
                                uint32_t* wd = &v.x;
                                uint32_t nan = 0;
#pragma unroll
                                for (int y = 0; y < 4; ++y) {
                                    const uint32_t n4 = __vcmpeq4(wd[y] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                                    wd[y] &= ~n4;
                                    nan |= n4;
                                }
                                if (nan) atomicOr(&poison[r >> 5], 1u << (r & 31));
                            }
                        }
                        const float s1 = vs[r];
                        const uint32_t s2 = pack_f16x2(s1, s1);
                        const uint4 lo = make_uint4(mul_f16x2(f16x2_of_lo(v.x), s2), mul_f16x2(f16x2_of_hi(v.x), s2),
                                                    mul_f16x2(f16x2_of_lo(v.y), s2), mul_f16x2(f16x2_of_hi(v.y), s2));
                        const uint4 hi = make_uint4(mul_f16x2(f16x2_of_lo(v.z), s2), mul_f16x2(f16x2_of_hi(v.z), s2),
                                                    mul_f16x2(f16x2_of_lo(v.w), s2), mul_f16x2(f16x2_of_hi(v.w), s2));
                        *reinterpret_cast<uint4*>(dst + tile_offset<Cfg>(r, 2 * c + odd)) = odd ? hi : lo;
                        *reinterpret_cast<uint4*>(dst + tile_offset<Cfg>(r, 2 * c + !odd)) = odd ? lo : hi;
                    }
                };
                if (whole && !diagonal) convert(std::false_type{});
                else convert(std::true_type{});
                fence_proxy_async_smem();
                mbar_arrive(&bars->ring_full[e % NH]);
                mbar_arrive(&bars->raw_empty[e % NR]);
                return true;
            });
        }
    } else {
        regs_increase<Cfg::HIGH_REGS>();
        // ------------------------------------------------------------ softmax
        const int t = stream;
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_tmem = tmem + lane_off + t * 128, o_tmem = tmem + lane_off + 256 + t * D;
        const int nt = t == 0 ? w.n[0] : w.n[1];
        const int j0 = t == 0 ? w.j0[0] : w.j0[1], part = w.part;
        const int limit = in ? row_limit(p, w, row) : w.len;   // (a row that is not there needs no mask)
        // A warp brings in its 32 query rows, swizzled, zero where there is none;
        // in alt mode both streams use stream 0's tile.  A lane has chunk qc of the
        // rows q_row(x).
        constexpr int LPR = D / 8 < 32 ? D / 8 : 32, RPI = 32 / LPR;   // lanes per row (16 bytes each), rows at a time
        const int qc = lane % LPR;
        auto q_row = [&](int x) { return (warp & 3) * 32 + x * RPI + lane / LPR; };
        auto q_at = [&](int r) -> uint32_t { return (qc >> 3) * (BM * 128) + r * 128 + (((qc & 7) ^ (r & 7)) << 4); };
        // (e4m3, d = 64: a row's two parts do not lie where its bf16 elements would)
        uint8_t* const rows16 = FP8 && D == 64 ? sEpi + t * 16384 : sQ + t * Cfg::Q_BYTES;
        if (w.pair || t == 0) {
            const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + qc * 8;
#pragma unroll 8
            for (int x = 0; x < LPR; ++x) {
                const int src = __shfl_sync(0xffffffffu, out, x * RPI + lane / LPR);
                cp_async16(smem_u32(rows16) + q_at(q_row(x)), q + static_cast<long long>(max(src, 0)) * D, src >= 0);
            }
        }
        cp_async_commit();
        cp_async_wait<0>();
        if constexpr (FP8) {
            // Into two e4m3 parts, in place.  (A loop of few instructions: with a
            // row a thread and everything unrolled, fetching the code took most of
            // 21000 cycles.)
            if (w.pair || t == 0) {
                uint8_t* tile = sQ + t * Cfg::Q_BYTES;
                constexpr int AT = 4;                              // row groups at a time (latency)
#pragma unroll 1
                for (int x = 0; x < LPR; x += AT) {
                    uint4 v[AT];
                    uint32_t top[AT];
#pragma unroll
                    for (int i = 0; i < AT; ++i) {
                        v[i] = *reinterpret_cast<const uint4*>(rows16 + q_at(q_row(x + i)));
                        top[i] = bf16x8_amax(v[i]);
                    }
#pragma unroll
                    for (int y = 1; y < LPR; y <<= 1)
#pragma unroll
                        for (int i = 0; i < AT; ++i) top[i] = max(top[i], __shfl_xor_sync(0xffffffffu, top[i], y));
#pragma unroll
                    for (int i = 0; i < AT; ++i) {
                        const int r = q_row(x + i), shift = q_shift(top[i], 7);
                        uint2 q1, q2;
                        q_split(v[i], top[i] >= 0x7f80u ? __uint_as_float(0x7fc00000u) : pow2f(shift), q1, q2);
                        const int c = qc >> 1;                     // 16 codes
                        constexpr int PER = Cfg::SWK / 16;
                        const int z = Cfg::SWK == 128 ? (c % PER) ^ (r & 7) : (c % PER) ^ ((r >> 1) & 3);
                        uint8_t* at = tile + (c / PER) * (BM * Cfg::SWK) + r * Cfg::SWK + (z << 4) + (qc & 1) * 8;
                        *reinterpret_cast<uint2*>(at) = q1;
                        *reinterpret_cast<uint2*>(at + BM * D) = q2;
                        // (not 0: -inf, the masked score, stays -inf when multiplied)
                        if (qc == 0) bars->q_log2[t * 128 + r] = fmaxf(p.scale_log2 * pow2f(-shift), 0x1p-126f);
                    }
                    __syncwarp();
                }
            }
        }
        fence_proxy_async_smem();
        mbar_arrive(&bars->q_full);
        // e4m3: rows lane / 4 + 8 i of the warp's 32 (see below).
        float vref = 0.0f;
        float tl4[4], m4[4], l4[4];
        int limit4[4];
        if constexpr (FP8) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                tl4[i] = l4[i] = 0.0f;
                m4[i] = -INFINITY;
                limit4[i] = __shfl_sync(0xffffffffu, limit, (lane >> 2) + 8 * i);
            }
        }
        float m = -INFINITY, l = 0.0f;
        bool ok = true;
        for (int u = 0; u < nt; ++u) {
            // Scale slot of this tile: its position among the K entries.
            const int kt = tile_slot<Cfg>(w, t, u);
            const int slot = kt % Cfg::SLOTS;
            bool wt = tile_wait(&bars->sc_full[slot], (kt / Cfg::SLOTS) & 1, abort_flag, p, SITE_TILE_SCALE);
            if (FP8) wt = wt && tile_wait(&bars->vs_ready[slot], (kt / Cfg::SLOTS) & 1, abort_flag, p, SITE_TILE_SCALE);
            // What does not need S is done while the products run.
            const int key0 = (j0 + u) * BN;
            const float2* ks = reinterpret_cast<const float2*>(sScale + slot * 2 * BN) + (lane & 3);
            constexpr int NG = BN / 8;
            float vfall = 1.0f;                    // e4m3: O is in units of vref
            uint32_t seen[BN / 32], all = 0xffffffffu;
            if constexpr (FP8) {
                const float now = bars->vref[slot];
                if (now != vref) {
                    vfall = vref * (1.0f / now);
                    vref = now;
                }
                const int low = min(min(limit4[0], limit4[1]), min(limit4[2], limit4[3]));
#pragma unroll
                for (int c = 0; c < BN / 32; ++c) all &= bars->valid[slot][c];
                if (key0 + BN > low) all = 0;
            } else {
#pragma unroll
                for (int c = 0; c < BN / 32; ++c) {
                    const int n = min(max(limit - key0 - c * 32, 0), 32);
                    seen[c] = bars->valid[slot][c] & (n == 32 ? 0xffffffffu : (1u << n) - 1u);
                    all &= seen[c];
                }
            }
            const bool masked = __any_sync(0xffffffffu, all != 0xffffffffu);
            wt = wt && tile_wait(&bars->s_full[t], u & 1, abort_flag, p, SITE_TILE_S);
            if (!__all_sync(0xffffffffu, wt)) {
                ok = false;
                break;
            }
            tc_fence_after();
            if constexpr (FP8) {
                // A key's scales are common to all rows: in the accumulator layout
                // (a thread has four rows and two of every eight columns) it reads a
                // quarter of them; one row a thread read 512 bytes of K scales and 512
                // of V scales a tile, which with the conversion's traffic bounded the
                // kernel by shared memory (6300 cycles a step of two tiles).
                if (u == 0) {                      // (in alt mode stream 0's threads wrote it: S comes after)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        tl4[i] = bars->q_log2[(w.pair ? t * 128 : 0) + (warp & 3) * 32 + (lane >> 2) + 8 * i];
                }
                uint32_t sr[8 * NG];               // (half of the rows, group, row bit, column bit)
#pragma unroll
                for (int h = 0; h < 2; ++h) tmem_ld_frag<NG>(s_tmem + (static_cast<uint32_t>(16 * h) << 16), sr + h * 4 * NG);
                tmem_wait_ld();
#pragma unroll
                for (int x = 0; x < 8 * NG; x += 32) reg_fence32(sr + x);
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const float2 k2 = ks[4 * g];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t* e = sr + (i >> 1) * 4 * NG + g * 4 + (i & 1) * 2;
                        const float2 v = __fmul2_rn(make_float2(__uint_as_float(e[0]), __uint_as_float(e[1])), k2);
                        e[0] = __float_as_uint(v.x);
                        e[1] = __float_as_uint(v.y);
                    }
                }
                if (masked) {
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        const int key = 8 * g + 2 * (lane & 3);
                        const uint32_t bits = bars->valid[slot][g / 4] >> (key & 31);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t* e = sr + (i >> 1) * 4 * NG + g * 4 + (i & 1) * 2;
                            if (!(bits & 1u) || key0 + key >= limit4[i]) e[0] = 0xff800000u;
                            if (!(bits & 2u) || key0 + key + 1 >= limit4[i]) e[1] = 0xff800000u;
                        }
                    }
                }
#pragma unroll
                for (int g = 0; g < NG; ++g)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t* e = sr + (i >> 1) * 4 * NG + g * 4 + (i & 1) * 2;
                        mx[i] = fmax3(mx[i], __uint_as_float(e[0]), __uint_as_float(e[1]));
                    }
                // A reference is set 7 (log2 units) below its row's maximum and moves
                // when that is more than 15 above it: P lies below 2^15, and what
                // fp16 rounds to 0 below 2^-25 is 2^-32 of the largest weight.  O and
                // l share them.
                bool move = false;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    mx[i] *= tl4[i];
                    move = move || mx[i] > m4[i] + 15.0f;
                }
                float fall4[4] = {vfall, vfall, vfall, vfall};
                if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
                        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
                        const float mn = mx[i] > m4[i] + 15.0f ? mx[i] - 7.0f : m4[i];
                        const float a = mn == m4[i] ? 1.0f : ex2_approx(m4[i] - mn);
                        m4[i] = mn;
                        l4[i] *= a;
                        fall4[i] *= a;
                    }
                }
                float2 acc[4];
                float2 neg[4], mul[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float ref = m4[i] == -INFINITY ? 0.0f : m4[i];
                    neg[i] = make_float2(-ref, -ref);
                    mul[i] = make_float2(tl4[i], tl4[i]);
                    acc[i] = make_float2(0.0f, 0.0f);
                }
#pragma unroll
                for (int g = 0; g < NG; ++g) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t* e = sr + (i >> 1) * 4 * NG + g * 4 + (i & 1) * 2;
                        float2 f = __ffma2_rn(make_float2(__uint_as_float(e[0]), __uint_as_float(e[1])), mul[i], neg[i]);
                        f.x = ex2_approx(f.x);
                        f.y = ex2_approx(f.y);
                        acc[i] = __fadd2_rn(acc[i], f);
                        // (packed into the half's first registers: all of it is read by now)
                        sr[(i >> 1) * 4 * NG + g * 2 + (i & 1)] = pack_f16x2(f.x, f.y);
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) tmem_st_frag<NG>(s_tmem + (static_cast<uint32_t>(16 * h) << 16), sr + h * 4 * NG);
#pragma unroll
                for (int i = 0; i < 4; ++i) l4[i] += acc[i].x + acc[i].y;
                const bool fell = fall4[0] != 1.0f || fall4[1] != 1.0f || fall4[2] != 1.0f || fall4[3] != 1.0f;
                if (u > 0 && __any_sync(0xffffffffu, fell)) {
                    // O's rows lie one per lane.
                    const float fall = to_row(fall4, lane);
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld32(o_tmem + c * 32, o);
                        tmem_wait_ld();
                        reg_fence32(o);
#pragma unroll
                        for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * fall);
                        tmem_st32(o_tmem + c * 32, o);
                    }
                }
            } else {
                uint32_t sr[BN];
#pragma unroll
                for (int c = 0; c < BN / 32; ++c) tmem_ld32(s_tmem + c * 32, sr + c * 32);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < BN / 32; ++c) reg_fence32(sr + c * 32);
                if (masked) {
#pragma unroll
                    for (int x = 0; x < BN; ++x)
                        if (!((seen[x / 32] >> (x % 32)) & 1u)) sr[x] = 0xff800000u;
                }
                float mx0 = __uint_as_float(sr[0]), mx1 = __uint_as_float(sr[1]);
                float mx2 = __uint_as_float(sr[2]), mx3 = __uint_as_float(sr[3]);
#pragma unroll
                for (int c = 4; c + 8 <= BN; c += 8) {
                    mx0 = fmax3(mx0, __uint_as_float(sr[c + 0]), __uint_as_float(sr[c + 1]));
                    mx1 = fmax3(mx1, __uint_as_float(sr[c + 2]), __uint_as_float(sr[c + 3]));
                    mx2 = fmax3(mx2, __uint_as_float(sr[c + 4]), __uint_as_float(sr[c + 5]));
                    mx3 = fmax3(mx3, __uint_as_float(sr[c + 6]), __uint_as_float(sr[c + 7]));
                }
                mx0 = fmax3(mx0, mx1, __uint_as_float(sr[BN - 4]));
                mx2 = fmax3(mx2, mx3, __uint_as_float(sr[BN - 3]));
                const float mx = fmax3(mx0, mx2, fmaxf(__uint_as_float(sr[BN - 2]), __uint_as_float(sr[BN - 1]))) * p.scale_log2;
                // The reference moves only by jumps of more than 8 (log2 units).
                float mn = m;
                if (mx > m + 8.0f) mn = mx;
                const float ref = mn == -INFINITY ? 0.0f : mn;
                const float alpha = mn == m ? 1.0f : ex2_approx(m - ref);
                const float2 mul2 = make_float2(p.scale_log2, p.scale_log2), neg2 = make_float2(-ref, -ref);
                float2 acc0 = make_float2(0.0f, 0.0f), acc1 = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int c = 0; c < BN / 32; ++c) {
                    uint32_t pk[16];
#pragma unroll
                    for (int x = 0; x < 16; x += 2) {
                        const int e = c * 32 + 2 * x;
                        float2 f = __ffma2_rn(make_float2(__uint_as_float(sr[e]), __uint_as_float(sr[e + 1])), mul2, neg2);
                        float2 g = __ffma2_rn(make_float2(__uint_as_float(sr[e + 2]), __uint_as_float(sr[e + 3])), mul2, neg2);
                        f.x = ex2_approx(f.x);
                        f.y = ex2_approx(f.y);
                        g.x = ex2_approx(g.x);
                        g.y = ex2_approx(g.y);
                        acc0 = __fadd2_rn(acc0, f);
                        acc1 = __fadd2_rn(acc1, g);
                        pk[x] = pack_bf16x2(f.x, f.y);
                        pk[x + 1] = pack_bf16x2(g.x, g.y);
                    }
                    tmem_st16(s_tmem + c * 16, pk);
                }
                l = l * alpha + ((acc0.x + acc0.y) + (acc1.x + acc1.y));
                if (u > 0 && __any_sync(0xffffffffu, alpha != 1.0f)) {
                    // The commit that signalled S(u) covers O += P(u-1) V(u-1).
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld32(o_tmem + c * 32, o);
                        tmem_wait_ld();
                        reg_fence32(o);
#pragma unroll
                        for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * alpha);
                        tmem_st32(o_tmem + c * 32, o);
                    }
                }
                m = mn;
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&bars->p_full[t]);
        }
        if constexpr (FP8) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                l4[i] += __shfl_xor_sync(0xffffffffu, l4[i], 1);
                l4[i] += __shfl_xor_sync(0xffffffffu, l4[i], 2);
            }
            l = to_row(l4, lane);
            m = to_row(m4, lane);
        }
        const long long rows_all = static_cast<long long>(p.B) * p.Nq * p.H;
        if (ok && nt > 0) {
            bool wt = tile_wait(&bars->o_full[t], 0, abort_flag, p, SITE_TILE_O);
            if (!FP8 && diag < j0 + nt) wt = wt && tile_wait(&bars->loaded, 0, abort_flag, p, SITE_TILE_LOADED);
            ok = __all_sync(0xffffffffu, wt);
        }
        if (ok) {
            tc_fence_after();
            if (diag < j0 + nt) {
                for (int x = max(diag, j0); x < j0 + nt; ++x) {
#pragma unroll
                    for (int c = 0; c < BN / 32; ++c) {
                        const int n = min(max(limit - x * BN - c * 32, 0), 32);
                        const uint32_t bits = bars->poison[min(x - diag, Cfg::DIAG_TILES - 1)][c];
                        if (bits & (n == 32 ? 0xffffffffu : (1u << n) - 1u)) l = __uint_as_float(0x7fc00000u);
                    }
                }
            }
            if constexpr (FP8) {
                // (rare) Values that were left out of the products; l has their weights.
                bool any = false;
                for (int x = max(diag, j0); x < j0 + nt; ++x)
#pragma unroll
                    for (int c = 0; c < BN / 32; ++c) any |= bars->poison[FP8 ? 8 + min(x - diag, Cfg::DIAG_TILES - 1) : 0][c] != 0;
                if (any) {
                    add_loud<Cfg>(p, w.table, w.kvh, bars->poison + 8, diag, max(diag, j0), j0 + nt, in ? limit : 0, out, m, vref, o_tmem);
                    vref = kLoudUnit;
                }
            }
            float inv = (l == 0.0f ? 0.0f : 1.0f / l) * (FP8 ? vref : 1.0f);
            float lse2 = l == 0.0f ? -INFINITY : m + __log2f(l);
            const bool some = nt > 0;
            // alt: stream 1 leaves its rows in the ring (no product reads it any
            // more once both streams are done), stream 0 adds them to its own.
            const bool alt = NS == 2 && !w.pair;
            float weight1 = 0.0f;
            const uint8_t* other = sRing + (tid & 127) * (D * 4);
            bool take = !(alt && t == 1);
            if (alt) {
                const int n_other = t == 0 ? w.n[1] : w.n[0];
                bool wt = n_other == 0 || tile_wait(&bars->o_full[1 - t], 0, abort_flag, p, SITE_TILE_O);
                if (t == 1) {
                    if (__all_sync(0xffffffffu, wt)) {
                        if (some) {
                            uint8_t* mine = const_cast<uint8_t*>(other);
#pragma unroll 1
                            for (int c = 0; c < D / 32; ++c) {
                                uint32_t o[32];
                                tmem_ld32(o_tmem + c * 32, o);
                                tmem_wait_ld();
                                reg_fence32(o);
#pragma unroll
                                for (int x = 0; x < 8; ++x)
                                    *reinterpret_cast<float4*>(mine + (((c * 8 + x) ^ (lane & 7)) << 4)) =
                                        make_float4(__uint_as_float(o[4 * x]) * inv, __uint_as_float(o[4 * x + 1]) * inv,
                                                    __uint_as_float(o[4 * x + 2]) * inv, __uint_as_float(o[4 * x + 3]) * inv);
                            }
                        }
                        bars->lse1[tid & 127] = lse2;
                    }
                    mbar_arrive(&bars->joined);
                } else {
                    wt = wt && tile_wait(&bars->joined, 0, abort_flag, p, SITE_TILE_JOIN);
                    take = __all_sync(0xffffffffu, wt);
                    if (take) {
                        const float l1 = bars->lse1[tid & 127];
                        if (l1 != -INFINITY) {             // (NaN included)
                            const float top = fmaxf(lse2, l1), ref = top == -INFINITY ? 0.0f : top;
                            const float a = lse2 == -INFINITY ? 0.0f : ex2_approx(lse2 - ref), b = ex2_approx(l1 - ref);
                            const float s = 1.0f / (a + b);
                            weight1 = b * s;
                            inv *= a * s;
                            lse2 = ref + __log2f(a + b);
                        }
                    }
                }
            }
            if (take) {
                if constexpr (DIRECT) {
                    if (in) p.lse[lse_at] = lse2 * 0.69314718055994530942f;
                } else {
                    if (in) p.part_lse[part * rows_all + out] = lse2;
                }
            }
            // O leaves through this warp's 4 KB of shared memory (32 rows x 128
            // bytes, swizzled by 16-byte chunk), so that every store instruction
            // writes whole 128-byte lines instead of 16 bytes of 32 rows.  (An
            // empty part's O is not written: the join does not read it.)
            uint8_t* epi = D == 64 ? sEpi + t * 16384
                         : w.pair || NS == 1 ? sQ + t * Cfg::Q_BYTES
                                             : sQ + Cfg::Q_BYTES + t * 16384;
            epi += (warp & 3) * 4096;
            const int mine = in && take && (DIRECT || lse2 != -INFINITY) ? out : -1;
            const bool add = __any_sync(0xffffffffu, weight1 != 0.0f);
            constexpr int COLS = DIRECT ? 64 : 32;             // columns per 128 bytes
            float2 not_finite = make_float2(0.0f, 0.0f);       // NaN once an element was not
#pragma unroll 1
            for (int c = 0; c < D / COLS; ++c) {         // (not unrolled: its code is fetched cold, once)
                if (!take) break;
                uint32_t o[COLS];
                if (some) {
#pragma unroll
                    for (int y = 0; y < COLS; y += 32) tmem_ld32(o_tmem + c * COLS + y, o + y);
                    tmem_wait_ld();
#pragma unroll
                    for (int y = 0; y < COLS; y += 32) reg_fence32(o + y);
#pragma unroll
                    for (int y = 0; y < COLS; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * inv);
                } else {
#pragma unroll
                    for (int y = 0; y < COLS; ++y) o[y] = 0u;
                }
                if (add) {
#pragma unroll
                    for (int y = 0; y < COLS / 4; ++y) {
                        const float4 v = *reinterpret_cast<const float4*>(other + (((c * (COLS / 4) + y) ^ (lane & 7)) << 4));
                        const float* e = &v.x;
#pragma unroll
                        for (int z = 0; z < 4; ++z)
                            if (weight1 != 0.0f) o[4 * y + z] = __float_as_uint(__uint_as_float(o[4 * y + z]) + e[z] * weight1);
                    }
                }
#pragma unroll
                for (int y = 0; y < COLS; y += 2)
                    not_finite = __ffma2_rn(make_float2(__uint_as_float(o[y]), __uint_as_float(o[y + 1])), make_float2(0.0f, 0.0f), not_finite);
                __syncwarp();
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    uint4 v;
                    uint32_t* q = &v.x;
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        q[y] = DIRECT ? pack_bf16x2(__uint_as_float(o[(DIRECT ? 8 : 4) * x + 2 * y]),
                                                    __uint_as_float(o[(DIRECT ? 8 : 4) * x + 2 * y + 1]))
                                      : o[4 * x + y];
                    *reinterpret_cast<uint4*>(epi + lane * 128 + ((x ^ (lane & 7)) << 4)) = v;
                }
                __syncwarp();
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const int rr = x * 4 + lane / 8, ch = lane % 8;
                    const int dst = __shfl_sync(0xffffffffu, mine, rr);
                    const uint4 v = *reinterpret_cast<const uint4*>(epi + rr * 128 + ((ch ^ (rr & 7)) << 4));
                    if (dst >= 0) {
                        if constexpr (DIRECT)
                            reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + static_cast<long long>(dst) * D + c * COLS)[ch] = v;
                        else
                            reinterpret_cast<uint4*>(p.part_o + (part * rows_all + dst) * D + c * COLS)[ch] = v;
                    }
                }
            }
            // Keys that all of these rows see but some earlier query of the sequence
            // does not: a V row among them that is not finite makes the rows NaN, as
            // the poison bits do for keys that only some of the rows see, so that a
            // query's result does not depend on the CTA that has it.  All rows' O then
            // shows it; so the values are read again only if O is not finite in all of
            // a warp's rows, and not by their scores alone.  (alt: the one row tile has
            // the first query; there are no such keys.)
            if (take && !alt && !w.prefix && p.causal) {
                const int lo = max(max(0, w.len - p.Nq + 1), j0 * BN), hi = min(diag_key, (j0 + nt) * BN);
                const bool odd = not_finite.x + not_finite.y != 0.0f, known = lse2 - lse2 == 0.0f;
                if (lo < hi && __all_sync(0xffffffffu, !in || odd) && __any_sync(0xffffffffu, in && known) &&
                    v_rows_not_finite<Cfg>(p, w, lo, hi, lane)) {
                    __syncwarp();
                    if (in) {
                        if constexpr (DIRECT) {
                            p.lse[lse_at] = __uint_as_float(0x7fc00000u);
                            uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + static_cast<long long>(out) * D);
#pragma unroll 1
                            for (int c = 0; c < D / 8; ++c) dst[c] = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
                        } else {
                            p.part_lse[part * rows_all + out] = __uint_as_float(0x7fc00000u);   // (the join does the rest)
                        }
                    }
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == Cfg::MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace attn
