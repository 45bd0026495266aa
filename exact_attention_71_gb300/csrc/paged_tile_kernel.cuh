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
// with one (alt) each stream takes half of the range with the same rows and
// leaves a partial result of its own, so that one stream's softmax still runs
// beside the other's products.  At d = 256 tensor memory holds one stream.
//
//   warps [0, 4 NS)       softmax (one thread per row)
//   next warpgroup        loaders: gather K and V rows through the page table
//                         into 128-byte-swizzled tiles (a ring of half stages,
//                         K and V alternating); e4m3 rows pass through a queue
//                         of raw 16-byte chunks that each thread fills with
//                         cp.async, reads back and converts to bf16 (exact; the
//                         row scales go to the scores and to P)
//   next warp             issues tcgen05.mma: S = Q K^T, O += P V
//
// The rows of a tile past the range are zero-filled (stale cache contents never
// reach a product) and their scores masked; so are the rows of a page outside
// the cache.
#pragma once

#include <cuda_bf16.h>

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
};

template <int D_, bool FP8_>
struct TileCfg {
    static constexpr int D = D_;
    static constexpr bool FP8 = FP8_;
    static constexpr int ES = FP8 ? 1 : 2;
    static constexpr int BM = 128;
    static constexpr int BN = D == 256 ? 64 : 128;
    static constexpr int NS = D == 256 ? 1 : 2;                    // streams
    static constexpr int NCB = D / 64;                             // 128-byte column boxes per row
    static constexpr int Q_BYTES = BM * D * 2;
    static constexpr int HALF_BYTES = BN * D * 2;                  // one K or V tile
    static constexpr int NH = D == 64 ? (FP8 ? 6 : 8) : (FP8 ? 3 : 5);
    static constexpr int AHEAD = 2;                                // bf16: copies in flight per thread (half stages)
    static constexpr int RAW_BYTES = FP8 ? BN * D : 0;
    static constexpr int NR = FP8 ? (D == 64 ? 5 : 3) : 0;
    static constexpr int SLOTS = 8;                                // key tiles whose scales are held
    static constexpr int SC_BYTES = FP8 ? SLOTS * 2 * BN * 4 : 0;
    static constexpr int DIAG_TILES = 8;
    static constexpr int LOAD_WARP = 4 * NS, MMA_WARP = 4 * NS + 4;
    static constexpr int THREADS = NS * 128 + 256;
    static constexpr int LAUNCH_REGS = (65536 / THREADS) / 8 * 8;
    static constexpr int LOAD_REGS = 72, MMA_REGS = 40;
    static constexpr int HIGH_RAW = (LAUNCH_REGS * THREADS - (LOAD_REGS + MMA_REGS) * 128) / (NS * 128) / 8 * 8;
    static constexpr int HIGH_REGS = HIGH_RAW > 248 ? 248 : HIGH_RAW;
    static constexpr int BAR_BYTES = 1024;
    static constexpr int SMEM_BYTES = 1024 + NS * Q_BYTES + NH * HALF_BYTES + NR * RAW_BYTES + SC_BYTES + BAR_BYTES;
    static_assert(HIGH_REGS * NS * 128 + (LOAD_REGS + MMA_REGS) * 128 <= LAUNCH_REGS * THREADS, "register split");
    static_assert(AHEAD < NH && (!FP8 || NR >= 2), "ring depth");
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
    // A slot (validity bits, scales) is rewritten at least 15 ring entries after
    // its tile's K; the entry NH + NR before that has been released by then.  It
    // is past the tile's V (at most 3 entries after its K), so the tile's softmax
    // is done with the slot.
    static_assert(15 - NH - NR >= 3, "scale slots");
};

struct TileBarriers {
    uint64_t q_full, loaded, drain;
    uint64_t s_full[2], p_full[2], o_full[2];
    uint64_t ring_full[8], ring_empty[8];
    uint64_t sc_full[8];
    uint32_t valid[8][4];          // per slot: bit per key of the tile
    uint32_t poison[8][4];         // per diagonal tile: bit per key whose V row is not finite
    uint32_t tmem_base;
    int abort_flag;
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

// What a CTA computes; every role derives it alike.
struct TileItem {
    bool prefix, pair;
    int seq, kvh;
    int rows;            // query rows of the segment for this head
    int rt[2];           // row tile of each stream (-1: none)
    int part[2];         // part index of each stream's result
    int j0[2], n[2];     // first key tile and number of key tiles of each stream
    int len;             // keys of the segment
    const int* table;
};

// Keys that row r of the segment sees.
__device__ __forceinline__ int row_limit(const PagedParams& p, const TileItem& w, int r) {
    if (w.prefix || !p.causal) return w.len;
    return max(0, w.len - p.Nq + 1 + r / p.G);
}

template <class Cfg>
__device__ __forceinline__ TileItem tile_item(const PagedParams& p) {
    TileItem w;
    int x = blockIdx.x;
    w.prefix = x < p.prefix_items;
    if (!w.prefix) x -= p.prefix_items;
    const int per = p.Nq * p.G;
    w.rows = w.prefix ? p.B * per : per;
    const int tiles = (w.rows + Cfg::BM - 1) / Cfg::BM;
    w.pair = Cfg::NS == 2 && tiles > 1;
    const int groups = w.pair ? (tiles + 1) / 2 : tiles;
    // Row groups of the same keys run next to one another.
    const int group = x % groups;
    x /= groups;
    w.kvh = x % p.H_kv;
    x /= p.H_kv;
    // Streams that split a range count as two parts.
    const int per_cta = (Cfg::NS == 2 && !w.pair) ? 2 : 1;
    const int ctas = w.prefix ? p.prefix_ctas : p.own_ctas;
    const int split = x % ctas;
    w.seq = w.prefix ? 0 : x / ctas;
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
    const int parts = ctas * per_cta;
    const int base = w.prefix ? 0 : p.prefix_parts;
    const int all = (len + Cfg::BN - 1) / Cfg::BN;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        if (t >= Cfg::NS) {
            w.rt[t] = -1;
            w.part[t] = w.j0[t] = w.n[t] = 0;
            continue;
        }
        w.rt[t] = w.pair ? group * 2 + t : group;
        if (w.rt[t] >= tiles) w.rt[t] = -1;
        const int part = w.pair || Cfg::NS == 1 ? split : 2 * split + t;
        w.part[t] = base + part;
        // Even shares of the key tiles.
        w.j0[t] = static_cast<int>(static_cast<long long>(all) * part / parts);
        int j1 = static_cast<int>(static_cast<long long>(all) * (part + 1) / parts);
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

template <class Cfg>
__device__ __forceinline__ uint32_t tile_offset(int r, int c) {     // 16-byte chunk c of row r
    return static_cast<uint32_t>((c >> 3) * (Cfg::BN * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

template <class Cfg, bool DIRECT>
__global__ void __launch_bounds__(Cfg::THREADS, 1) paged_tile_kernel(const PagedParams p) {
    constexpr int D = Cfg::D, BN = Cfg::BN, BM = Cfg::BM, NS = Cfg::NS, NH = Cfg::NH;
    constexpr bool FP8 = Cfg::FP8;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sQ = smem;
    uint8_t* sRing = smem + NS * Cfg::Q_BYTES;
    uint8_t* sRaw = sRing + NH * Cfg::HALF_BYTES;
    float* sScale = reinterpret_cast<float*>(sRaw + Cfg::NR * Cfg::RAW_BYTES);     // (slot, k / v, BN)
    TileBarriers* bars = reinterpret_cast<TileBarriers*>(reinterpret_cast<uint8_t*>(sScale) + Cfg::SC_BYTES);
    volatile int* abort_flag = &bars->abort_flag;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        mbar_init(&bars->q_full, 128);
        mbar_init(&bars->loaded, 128);
        mbar_init(&bars->drain, 1);
        for (int t = 0; t < 2; ++t) {
            mbar_init(&bars->s_full[t], 1);
            mbar_init(&bars->p_full[t], 128);
            mbar_init(&bars->o_full[t], 1);
        }
        for (int s = 0; s < 8; ++s) {
            mbar_init(&bars->ring_full[s], 128);
            mbar_init(&bars->ring_empty[s], 1);
            mbar_init(&bars->sc_full[s], 128);
            for (int x = 0; x < 4; ++x) bars->poison[s][x] = 0;
        }
        bars->abort_flag = 0;
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    if (warp == 0) {
        tmem_alloc(&bars->tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    const TileItem w = tile_item<Cfg>(p);
    // From this key on the CTA's rows may see different keys; its tile.
    int diag_key = w.len;
    if (!w.prefix && p.causal) diag_key = row_limit(p, w, max(w.rt[0], 0) * BM);
    const int diag = diag_key < w.len ? diag_key / BN : w.len / BN + 1;

    if (warp >= Cfg::MMA_WARP) {
        regs_decrease<Cfg::MMA_REGS>();
        if (warp == Cfg::MMA_WARP) {
            // -------------------------------------------------------- MMA issuer
            constexpr uint32_t idesc_s = make_idesc(1u, 128, BN, 0), idesc_o = make_idesc(1u, 128, D, 1);
            const uint32_t ring = smem_u32(sRing);
            uint32_t e = 0;                         // ring entries consumed
            uint32_t pc[2] = {0, 0};                // P tiles consumed per stream
            bool ok = (w.n[0] + w.n[1] == 0) || tile_warp_wait(&bars->q_full, 0, abort_flag, p, SITE_TILE_Q);
            auto entry = [&](uint32_t x) { return tile_warp_wait(&bars->ring_full[x % NH], (x / NH) & 1, abort_flag, p, SITE_TILE_FULL); };
            auto issue_s = [&](int t, uint32_t x) {
                const uint64_t qd = sdesc_sw128(smem_u32(sQ) + (w.pair ? t : 0) * Cfg::Q_BYTES, 16, 1024);
                const uint64_t kd = sdesc_sw128(ring + (x % NH) * Cfg::HALF_BYTES, 16, 1024);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t a = (kk / 4) * (BM * 128) + (kk % 4) * 32, b = (kk / 4) * (BN * 128) + (kk % 4) * 32;
                        mma_f16_ss(tmem + t * 128, qd + (a >> 4), kd + (b >> 4), idesc_s, kk > 0 ? 1u : 0u);
                    }
                    mma_commit(&bars->s_full[t]);
                }
                __syncwarp();
            };
            auto issue_o = [&](int t, uint32_t x, bool acc, bool last) {
                const uint64_t vd = sdesc_sw128(ring + (x % NH) * Cfg::HALF_BYTES, BN * 128, 1024);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < BN / 16; ++kk)
                        mma_f16_ts(tmem + 256 + t * D, tmem + t * 128 + kk * 8, vd + ((kk * 16 * 128) >> 4), idesc_o,
                                   (kk > 0 || acc) ? 1u : 0u);
                    if (last) mma_commit(&bars->o_full[t]);
                }
                __syncwarp();
            };
            auto release = [&](uint32_t x) {
                if (elect_one()) mma_commit(&bars->ring_empty[x % NH]);
                __syncwarp();
            };
            auto wait_p = [&](int t) {
                const bool r = tile_warp_wait(&bars->p_full[t], pc[t] & 1, abort_flag, p, SITE_TILE_P);
                ++pc[t];
                tc_fence_after();
                return r;
            };
            const int n = max(w.n[0], w.n[1]);
            if (w.pair || NS == 1) {
                // Step u: per stream O += P(u-1) V(u-1), then S(u).
                for (int u = 0; u <= n && ok; ++u) {
                    const uint32_t ev = 2 * u - 1, ek = 2 * u;
                    if (u > 0) ok = entry(ev);
                    if (ok && u < n) ok = entry(ek);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int t = 0; t < NS; ++t) {
                        if (u > 0 && u <= w.n[t]) {
                            if (!wait_p(t)) { ok = false; break; }
                            issue_o(t, ev, u > 1, u == w.n[t]);
                        }
                        if (u < w.n[t]) issue_s(t, ek);
                    }
                    if (!ok) break;
                    if (u > 0) release(ev);
                    if (u < n) release(ek);
                }
            } else {
                for (int u = 0; u <= n && ok; ++u) {
#pragma unroll
                    for (int t = 0; t < NS; ++t) {
                        if (!ok) continue;
                        if (u >= 1 && u <= w.n[t]) {
                            ok = entry(e) && wait_p(t);
                            if (!ok) continue;
                            tc_fence_after();
                            issue_o(t, e, u > 1, u == w.n[t]);
                            release(e);
                            ++e;
                        }
                        if (u < w.n[t]) {
                            ok = entry(e);
                            if (!ok) continue;
                            tc_fence_after();
                            issue_s(t, e);
                            release(e);
                            ++e;
                        }
                    }
                }
            }
            // Every MMA issued here has finished before teardown.
            if (elect_one()) {
                mma_commit(&bars->drain);
                const long long t0 = clock64();
                const unsigned long long lim = p.wait_limit > 2000000000ull ? p.wait_limit : 2000000000ull;
                while (!mbar_try_wait(&bars->drain, 0)) {
                    if (static_cast<unsigned long long>(clock64() - t0) > lim) {
                        atomicCAS(p.status, 0, SITE_TILE_DRAIN);
                        break;
                    }
                }
            }
            __syncwarp();
        }
    } else if (warp >= Cfg::LOAD_WARP) {
        regs_decrease<Cfg::LOAD_REGS>();
        // ------------------------------------------------------------ loaders
        const int lt = tid - Cfg::LOAD_WARP * 32;
        const int mask = (1 << p.page_shift) - 1;
        // Q: rows of the segment, zero where there are none.
        {
            const int per = p.Nq * p.G;
            const int tiles = w.pair ? 2 : 1;
            for (int x = lt; x < tiles * BM * (D / 8); x += 128) {
                const int c = x % (D / 8), r = x / (D / 8) % BM, t = x / (D / 8) / BM;
                const int row = w.rt[t] * BM + r;
                const bool in = w.rt[t] >= 0 && row < w.rows;
                long long src = 0;
                if (in) {
                    const int b = w.prefix ? row / per : w.seq, i = (w.prefix ? row % per : row) / p.G;
                    src = ((static_cast<long long>(b) * p.Nq + i) * p.H + w.kvh * p.G + row % p.G) * D + c * 8;
                }
                cp_async16(smem_u32(sQ) + t * Cfg::Q_BYTES + (c >> 3) * (BM * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                           static_cast<const __nv_bfloat16*>(p.q) + src, in);
            }
            cp_async_commit();
            cp_async_wait<0>();
            fence_proxy_async_smem();
            mbar_arrive(&bars->q_full);
        }
        // Cache row of key `key` (its page's row when it is inside the cache),
        // -1 where there is none.
        auto cache_row = [&](int key) -> long long {
            if (key >= w.len) return -1;
            const int page = __ldg(w.table + (key >> p.page_shift));
            if (page < 0 || page >= p.num_pages) {
                atomicCAS(p.status, 0, SITE_PAGED_PAGE);
                return -1;
            }
            return ((static_cast<long long>(page) * p.H_kv + w.kvh) << p.page_shift) + (key & mask);
        };
        constexpr int CPR = D * Cfg::ES / 16;               // 16-byte chunks of a cache row
        constexpr int RPP = 128 / CPR;                      // rows per pass of the 128 threads
        constexpr int PASSES = BN / RPP;
        const int c = lt % CPR, r0 = lt / CPR;
        // The tile's validity bits and (e4m3) scales: at its K entry.
        auto tile_meta = [&](int key0, int slot) {
            const int k = lt;
            long long row = -1;
            if (k < BN) row = cache_row(key0 + k);
            const uint32_t bits = __ballot_sync(0xffffffffu, row >= 0);
            if (k < BN && lane == 0) bars->valid[slot][k >> 5] = bits;
            if constexpr (FP8) {
                if (k < BN) {
                    const uint32_t dst = smem_u32(sScale) + (slot * 2 * BN + k) * 4;
                    const float* ks = p.k_scale + (row < 0 ? 0 : row);
                    const float* vs = p.v_scale + (row < 0 ? 0 : row);
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(ks), "r"(row < 0 ? 0 : 4) : "memory");
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst + BN * 4), "l"(vs), "r"(row < 0 ? 0 : 4) : "memory");
                }
            }
        };
        auto copy_rows = [&](const void* cache, int key0, auto&& dst) {
            const uint8_t* base = static_cast<const uint8_t*>(cache) + c * 16;
#pragma unroll
            for (int i = 0; i < PASSES; ++i) {
                const int r = r0 + i * RPP;
                const long long row = cache_row(key0 + r);
                cp_async16(dst(r, i), base + (row < 0 ? 0 : row * (D * Cfg::ES)), row >= 0);
            }
        };
        const uint32_t ring = smem_u32(sRing), raw = smem_u32(sRaw);
        bool ok = true;
        uint32_t ktile = 0;                                 // key tiles so far (scale slots)
        if constexpr (!FP8) {
            uint32_t e = 0, done = 0;                       // entries issued; signalled
            uint32_t kinds = 0;                             // bit (e & 31): entry e is a V
            int keys[Cfg::AHEAD + 1];
#pragma unroll
            for (int x = 0; x <= Cfg::AHEAD; ++x) keys[x] = 0;
            uint32_t kdone = 0;
            auto signal = [&](uint32_t x, int key0) {
                if ((kinds >> (x & 31)) & 1u) {
                    if (key0 / BN >= diag) {
                        // Non-finite values leave the products of tiles that
                        // only some rows see; the rows that see them learn it
                        // from the poison bits.
                        uint8_t* tile = sRing + (x % NH) * Cfg::HALF_BYTES;
#pragma unroll 1
                        for (int i = 0; i < PASSES; ++i) {
                            const int r = r0 + i * RPP;
                            uint32_t* at = reinterpret_cast<uint32_t*>(tile + tile_offset<Cfg>(r, c));
                            bool any = false;
                            if (key0 + r < diag_key) continue;
#pragma unroll 1
                            for (int y = 0; y < 4; ++y) {
                                uint32_t v = at[y];
                                if ((v & 0x7f80u) == 0x7f80u) { v &= 0xffff0000u; any = true; }
                                if ((v & 0x7f800000u) == 0x7f800000u) { v &= 0xffffu; any = true; }
                                at[y] = v;
                            }
                            if (any) atomicOr(&bars->poison[min(key0 / BN - diag, Cfg::DIAG_TILES - 1)][r >> 5], 1u << (r & 31));
                        }
                    }
                } else {
                    mbar_arrive(&bars->sc_full[kdone++ % Cfg::SLOTS]);
                }
                fence_proxy_async_smem();
                mbar_arrive(&bars->ring_full[x % NH]);
            };
            tile_entries<Cfg>(w, [&](int t, int u, bool is_v) -> bool {
                if (!tile_wait(&bars->ring_empty[e % NH], ((e / NH) & 1) ^ 1, abort_flag, p, SITE_TILE_EMPTY)) {
                    ok = false;
                    return false;
                }
                const int key0 = (w.j0[t] + u) * BN;
                if (!is_v) tile_meta(key0, static_cast<int>(ktile++ % Cfg::SLOTS));
                const uint32_t at = ring + (e % NH) * Cfg::HALF_BYTES;
                copy_rows(is_v ? p.v_cache : p.k_cache, key0, [&](int r, int) { return at + tile_offset<Cfg>(r, c); });
                cp_async_commit();
                kinds = is_v ? kinds | (1u << (e & 31)) : kinds & ~(1u << (e & 31));
#pragma unroll
                for (int x = Cfg::AHEAD; x > 0; --x) keys[x] = keys[x - 1];
                keys[0] = key0;
                ++e;
                if (e > Cfg::AHEAD) {
                    cp_async_wait<Cfg::AHEAD>();
                    signal(done++, keys[Cfg::AHEAD]);
                }
                return true;
            });
            cp_async_wait<0>();
            if (ok) {
#pragma unroll
                for (int x = Cfg::AHEAD - 1; x >= 0; --x)
                    if (static_cast<int>(e) > x) signal(done++, keys[x]);
            }
        } else {
            // The raw queue runs NR - 1 entries ahead of the conversion: a
            // second walk over the same entries.
            uint32_t ei = 0, e = 0, kdone = 0;
            const int total_n = max(w.n[0], w.n[1]);
            const uint32_t total = w.pair || NS == 1 ? 2u * total_n : 2u * (w.n[0] + w.n[1]);
            // Entry x of the walk: stream, tile, K or V.
            int it_u = 0, it_phase = 0;                     // iterator of the issue side
            auto next = [&](int& t, int& u, bool& is_v) {
                // The next ring entry in tile_entries order.
                if (w.pair || NS == 1) {
                    t = 0;
                    u = it_u;
                    is_v = it_phase == 1;
                    if (it_phase == 1) { it_phase = 0; ++it_u; }
                    else it_phase = 1;
                    return;
                }
                while (true) {                              // phases: V of stream 0, K of 0, V of 1, K of 1
                    const int ph = it_phase, uu = it_u;
                    if (++it_phase == 4) { it_phase = 0; ++it_u; }
                    t = ph >> 1;
                    is_v = (ph & 1) == 0;
                    u = is_v ? uu - 1 : uu;
                    if (is_v ? (uu >= 1 && uu <= w.n[t]) : uu < w.n[t]) return;
                    if (uu > total_n) return;
                }
            };
            uint32_t kinds = 0;
            auto issue = [&]() {
                if (ei < total) {
                    int t, u;
                    bool is_v;
                    next(t, u, is_v);
                    const int key0 = (w.j0[t] + u) * BN;
                    if (!is_v) tile_meta(key0, static_cast<int>(ktile++ % Cfg::SLOTS));
                    const uint32_t at = raw + (ei % Cfg::NR) * Cfg::RAW_BYTES + lt * 16;
                    copy_rows(is_v ? p.v_cache : p.k_cache, key0, [&](int, int i) { return at + i * 128 * 16; });
                    kinds = is_v ? kinds | (1u << (ei & 31)) : kinds & ~(1u << (ei & 31));
                    ++ei;
                }
                cp_async_commit();
            };
            for (int x = 0; x < Cfg::NR - 1; ++x) issue();
            for (; e < total; ++e) {
                issue();
                cp_async_wait<Cfg::NR - 1>();
                if (!((kinds >> (e & 31)) & 1u)) mbar_arrive(&bars->sc_full[kdone++ % Cfg::SLOTS]);
                if (!tile_wait(&bars->ring_empty[e % NH], ((e / NH) & 1) ^ 1, abort_flag, p, SITE_TILE_EMPTY)) {
                    ok = false;
                    break;
                }
                const uint8_t* src = sRaw + (e % Cfg::NR) * Cfg::RAW_BYTES + lt * 16;
                uint8_t* dst = sRing + (e % NH) * Cfg::HALF_BYTES;
#pragma unroll 4
                for (int i = 0; i < PASSES; ++i) {
                    const uint4 v = *reinterpret_cast<const uint4*>(src + i * 128 * 16);
                    const int r = r0 + i * RPP;
                    const uint4 lo = make_uint4(e4m3_pair<0x9180>(v.x, 0), e4m3_pair<0xb3a2>(v.x, 0),
                                                e4m3_pair<0x9180>(v.y, 0), e4m3_pair<0xb3a2>(v.y, 0));
                    const uint4 hi = make_uint4(e4m3_pair<0x9180>(v.z, 0), e4m3_pair<0xb3a2>(v.z, 0),
                                                e4m3_pair<0x9180>(v.w, 0), e4m3_pair<0xb3a2>(v.w, 0));
                    *reinterpret_cast<uint4*>(dst + tile_offset<Cfg>(r, 2 * c)) = lo;
                    *reinterpret_cast<uint4*>(dst + tile_offset<Cfg>(r, 2 * c + 1)) = hi;
                }
                fence_proxy_async_smem();
                mbar_arrive(&bars->ring_full[e % NH]);
            }
            cp_async_wait<0>();
        }
        if (ok) mbar_arrive(&bars->loaded);
    } else {
        regs_increase<Cfg::HIGH_REGS>();
        // ------------------------------------------------------------ softmax
        const int t = warp >> 2;
        const int r = (warp & 3) * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_tmem = tmem + lane_off + t * 128, o_tmem = tmem + lane_off + 256 + t * D;
        const int rt = t == 0 ? w.rt[0] : w.rt[1], nt = t == 0 ? w.n[0] : w.n[1];
        const int j0 = t == 0 ? w.j0[0] : w.j0[1], part = t == 0 ? w.part[0] : w.part[1];
        const int row = rt * BM + r;
        const bool in = rt >= 0 && row < w.rows;
        const int per = p.Nq * p.G;
        long long out = 0;
        int lse_at = 0;
        int limit = 0;
        if (in) {
            const int b = w.prefix ? row / per : w.seq, i = (w.prefix ? row % per : row) / p.G;
            const int h = w.kvh * p.G + row % p.G;
            out = (static_cast<long long>(b) * p.Nq + i) * p.H + h;
            lse_at = (b * p.H + h) * p.Nq + i;
            limit = row_limit(p, w, row);
        }
        const bool alt = NS == 2 && !w.pair;
        float m = -INFINITY, l = 0.0f;
        bool ok = true;
        for (int u = 0; u < nt; ++u) {
            // Scale slot of this tile: its position among the K entries.
            int kt = u;
            if (alt) kt = u < min(w.n[0], w.n[1]) ? 2 * u + t : min(w.n[0], w.n[1]) + u;
            const int slot = kt % Cfg::SLOTS;
            bool wt = tile_wait(&bars->sc_full[slot], (kt / Cfg::SLOTS) & 1, abort_flag, p, SITE_TILE_SCALE);
            wt = wt && tile_wait(&bars->s_full[t], u & 1, abort_flag, p, SITE_TILE_S);
            if (!__all_sync(0xffffffffu, wt)) {
                ok = false;
                break;
            }
            tc_fence_after();
            uint32_t sr[BN];
#pragma unroll
            for (int c = 0; c < BN / 32; ++c) tmem_ld32(s_tmem + c * 32, sr + c * 32);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < BN / 32; ++c) reg_fence32(sr + c * 32);
            if constexpr (FP8) {
                const float2* ks = reinterpret_cast<const float2*>(sScale + slot * 2 * BN);
#pragma unroll
                for (int x = 0; x < BN; x += 2) {
                    const float2 v = __fmul2_rn(make_float2(__uint_as_float(sr[x]), __uint_as_float(sr[x + 1])), ks[x / 2]);
                    sr[x] = __float_as_uint(v.x);
                    sr[x + 1] = __float_as_uint(v.y);
                }
            }
            const int key0 = (j0 + u) * BN;
            uint32_t seen[BN / 32];
            uint32_t all = 0xffffffffu;
#pragma unroll
            for (int c = 0; c < BN / 32; ++c) {
                const int n = min(max(limit - key0 - c * 32, 0), 32);
                seen[c] = bars->valid[slot][c] & (n == 32 ? 0xffffffffu : (1u << n) - 1u);
                all &= seen[c];
            }
            const bool masked = __any_sync(0xffffffffu, all != 0xffffffffu);
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
            const float2* vs = reinterpret_cast<const float2*>(sScale + slot * 2 * BN + BN);
#pragma unroll
            for (int c = 0; c < BN / 32; ++c) {
                uint32_t pk[16];
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    const int e = c * 32 + 2 * x;
                    float2 f = __ffma2_rn(make_float2(__uint_as_float(sr[e]), __uint_as_float(sr[e + 1])), mul2, neg2);
                    f.x = ex2_approx(f.x);
                    f.y = ex2_approx(f.y);
                    if (x & 1) acc1 = __fadd2_rn(acc1, f);
                    else acc0 = __fadd2_rn(acc0, f);
                    if constexpr (FP8) {
                        // V's row scale rides on P; l sums the plain weights.
                        const float2 g = __fmul2_rn(f, vs[e / 2]);
                        if (masked) {
                            // 0 times a NaN scale of a key this row does not see
                            f.x = f.x == 0.0f ? 0.0f : g.x;
                            f.y = f.y == 0.0f ? 0.0f : g.y;
                        } else {
                            f = g;
                        }
                    }
                    pk[x] = pack_bf16x2(f.x, f.y);
                }
                tmem_st16(s_tmem + c * 16, pk);
            }
            l = l * alpha + ((acc0.x + acc0.y) + (acc1.x + acc1.y));
            if (u > 0 && __any_sync(0xffffffffu, alpha != 1.0f)) {
                // The commit that signalled S(u) covers O += P(u-1) V(u-1).
#pragma unroll
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
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&bars->p_full[t]);
            m = mn;
        }
        const long long rows_all = static_cast<long long>(p.B) * p.Nq * p.H;
        if (ok && nt > 0) {
            bool wt = tile_wait(&bars->o_full[t], 0, abort_flag, p, SITE_TILE_O);
            if (!FP8 && diag < j0 + nt) wt = wt && tile_wait(&bars->loaded, 0, abort_flag, p, SITE_TILE_LOADED);
            ok = __all_sync(0xffffffffu, wt);
        }
        if (ok) {
            tc_fence_after();
            if (!FP8 && diag < j0 + nt) {
                for (int x = max(diag, j0); x < j0 + nt; ++x) {
#pragma unroll
                    for (int c = 0; c < BN / 32; ++c) {
                        const int n = min(max(limit - x * BN - c * 32, 0), 32);
                        const uint32_t bits = bars->poison[min(x - diag, Cfg::DIAG_TILES - 1)][c];
                        if (bits & (n == 32 ? 0xffffffffu : (1u << n) - 1u)) l = __uint_as_float(0x7fc00000u);
                    }
                }
            }
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            const float lse2 = l == 0.0f ? -INFINITY : m + __log2f(l);
            const bool some = nt > 0;
            if constexpr (DIRECT) {
                if (in) p.lse[lse_at] = lse2 * 0.69314718055994530942f;
            } else {
                if (in) p.part_lse[part * rows_all + out] = lse2;
            }
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                if (some) {
                    tmem_ld32(o_tmem + c * 32, o);
                    tmem_wait_ld();
                    reg_fence32(o);
                }
                __syncwarp();
                if constexpr (DIRECT) {
                    if (in) {
                    uint32_t pk[16];
#pragma unroll
                    for (int x = 0; x < 16; ++x)
                        pk[x] = some ? pack_bf16x2(__uint_as_float(o[2 * x]) * inv, __uint_as_float(o[2 * x + 1]) * inv) : 0u;
                    uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + out * D + c * 32);
#pragma unroll
                    for (int x = 0; x < 4; ++x) dst[x] = make_uint4(pk[4 * x], pk[4 * x + 1], pk[4 * x + 2], pk[4 * x + 3]);
                    }
                } else if (in && l != 0.0f) {
                    float4* dst = reinterpret_cast<float4*>(p.part_o + (part * rows_all + out) * D + c * 32);
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        dst[x] = make_float4(__uint_as_float(o[4 * x]) * inv, __uint_as_float(o[4 * x + 1]) * inv,
                                             __uint_as_float(o[4 * x + 2]) * inv, __uint_as_float(o[4 * x + 3]) * inv);
                }
                __syncwarp();
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace attn
