// Plans of the paged attention and the join of its partial results.
//
//     lse = log2 sum_p 2^lse_p,   O = sum_p 2^(lse_p - lse) O_p
//
// over the parts of a row (ranges of the shared prefix and of the sequence's
// own tokens), in the order of the parts: the result does not depend on which
// CTA finished first.  Bound by memory, and for few rows by latency: 32768 rows of
// 128 in two parts, 33.5 MB read, 8 us behind the tile kernel.
#include <cuda_bf16.h>

#include <algorithm>

#include "paged.cuh"
#include "sm103_bulk.cuh"

namespace attn {

namespace {

long long up(long long a, long long b) { return (a + b - 1) / b; }

// Times of the tile kernel, measured, in microseconds: a step of a CTA (d = 64 and
// 128: a key tile against two row tiles, or two key tiles against one: 1.4 with a
// bf16 cache, 1.8 with an e4m3 one; d = 256: one key tile), and what a CTA costs besides (launch, query rows, first copies,
// epilogue).
constexpr double kTileFixedUs = 7.0;
double tile_step_us(int d) { return d == 256 ? 1.3 : 1.6; }

// CTAs that share a row tile's keys (tile kernel, one CTA an SM).  By itself the
// kernel is fastest with as few waves x steps as possible.  The streaming kernel
// starts beside it on the SMs that it leaves free, and is bound by memory where
// the tile kernel is bound by the tensor cores: with `other` SM-microseconds of
// streaming work the total is what counts, and fewer, longer CTAs may serve it
// better (128 sequences x 4 query heads a key/value head, d = 128, behind a bf16
// prefix of 16384 with up to 512 tokens of their own: 9 CTAs for each of the 16
// units of the prefix, and the own tokens after them, 75 us; 6, with the own tokens
// beside them, 62).  That work is an estimate (the lengths are not known here), so
// the tile kernel itself may become at most half as slow again by it.  More CTAs
// have to be 2 % better: each writes a partial result that is read again.
int tile_ctas(int d, long long units, long long steps, double other) {
    const auto alone = [&](long long s) {
        return static_cast<double>(up(units * s, kPlanSms)) * (static_cast<double>(up(steps, s)) * tile_step_us(d) + kTileFixedUs);
    };
    const long long most = std::min<long long>(kPlanSms, steps);
    double least = alone(1);
    for (long long s = 2; s <= most; ++s) least = std::min(least, alone(s));
    int best = 1;
    double best_total = -1.0;
    for (long long s = 1; s <= most; ++s) {
        const double t = alone(s);
        if (t > 1.5 * least) continue;
        const double free_sms = units * s < kPlanSms ? static_cast<double>(kPlanSms - units * s) : 0.0;
        const double rest = other - free_sms * t;
        const double total = rest > 0.0 ? t + rest / kPlanSms : std::max(t, free_sms > 0.0 ? other / free_sms : t);
        if (best_total < 0.0 || total < 0.98 * best_total) {
            best = static_cast<int>(s);
            best_total = total;
        }
    }
    return best;
}

}  // namespace

PagedPlan paged_plan(int B, int Nq, int H, int H_kv, int d, int prefix_len, int max_pages, int page_size) {
    PagedPlan plan;
    const long long rows = static_cast<long long>(Nq) * (H / H_kv);      // of one sequence and key/value head
    const long long own = static_cast<long long>(max_pages) * page_size;
    const int bn = d == 256 ? 64 : 128;
    const long long all = B * rows;                                      // the prefix's rows of a key/value head
    const bool own_stream = rows <= stream_rows(d);
    plan.prefix_stream = prefix_len > 0 && all <= stream_rows(d);
    // (one launch for both, so one kind of CTA)
    plan.stream_tile = (own_stream ? rows : 0) > 8 || (plan.prefix_stream && all > 8) ? 16 : 8;
    // Streaming kernel.  A CTA's time is its keys plus a fixed cost (page table,
    // first loads, join) worth about 300; beyond one wave CTAs replace one
    // another as they finish, half a CTA's time is lost at the end, and sequences
    // are seldom all as long as their tables (16 x 32768 tokens, 8 heads of 128,
    // e4m3: 121 us in 16 parts against 133 in 3, which fit one wave).
    // (d = 256: the CTAs of an e4m3 cache.  A bf16 one has one on an SM, but with 152
    // for both, 10 x 4096 tokens, 8 heads, take 47.0 us instead of 43.6 in bf16 and
    // 28.1 instead of 26.9 in e4m3, 64 x 1000, 2 heads, 21.5 instead of 27.6 and 21.0
    // instead of 17.2, 2 x 30000 23.2 instead of 29.8 and 20.9 instead of 17.9.)
    const double slots = kPlanSms * (d == 64 ? 4.0 : d == 128 || plan.stream_tile == 8 ? 3.0 : 2.0);
    const auto stream_parts = [&](long long keys, long long units) {
        int best = 1;
        double best_cost = -1.0;
        for (int s = 1; s <= kMaxParts && (s == 1 || s * static_cast<long long>(own_chunk(d)) < keys + own_chunk(d)); ++s) {
            const double waves = static_cast<double>(units) * s / slots, cta = static_cast<double>(up(keys, s)) + kStreamFixed;
            const double cost = waves <= 1.0 ? cta : (0.8 * waves + 0.5) * cta;
            if (best_cost < 0.0 || cost < best_cost) {
                best = s;
                best_cost = cost;
            }
        }
        return best;
    };
    // Steps of a CTA over `keys`: two streams halve the tiles of a single row tile.
    const auto steps_of = [&](long long keys, long long tiles) { return up(keys, bn * (d != 256 && tiles == 1 ? 2 : 1)); };
    double streaming = 0.0;                                              // SM-microseconds
    long long tile_items = 0, stream_blocks = 0;
    if (!own_stream) {
        const long long tiles = up(rows, 128), groups = d == 256 ? tiles : up(tiles, 2);
        plan.own_ctas = tile_ctas(d, B * static_cast<long long>(H_kv) * groups, steps_of(own, tiles), 0.0);
        tile_items = B * static_cast<long long>(H_kv) * groups * plan.own_ctas;
        plan.own_items = static_cast<int>(tile_items);
        plan.own_parts = plan.own_ctas;
    } else {
        const long long units = B * static_cast<long long>(H_kv) * up(rows, plan.stream_tile);
        plan.own_parts = stream_parts(own, units);
        stream_blocks = units * plan.own_parts;
        // (sequences fill three quarters of their tables, say; a key of one head
        // takes an SM 0.08 d nanoseconds)
        streaming = 0.75 * static_cast<double>(units) * static_cast<double>(own) * 0.08e-3 * d;
    }
    if (prefix_len > 0) {
        if (!plan.prefix_stream) {
            const long long tiles = up(all, 128), groups = d == 256 ? tiles : up(tiles, 2);
            plan.prefix_ctas = tile_ctas(d, H_kv * groups, steps_of(prefix_len, tiles), streaming);
            plan.prefix_items = static_cast<int>(H_kv * groups * plan.prefix_ctas);
            tile_items += H_kv * groups * plan.prefix_ctas;
            plan.prefix_parts = plan.prefix_ctas;
        } else {
            const long long units = H_kv * up(all, plan.stream_tile);
            plan.prefix_parts = stream_parts(prefix_len, units);
            stream_blocks += units * plan.prefix_parts;
        }
    }
    plan.blocks = std::max(tile_items, stream_blocks);
    const int parts = plan.prefix_parts + plan.own_parts;
    plan.direct = parts == 1;
    if (!plan.direct) {
        const size_t r = static_cast<size_t>(parts) * B * Nq * H;
        plan.part_o_bytes = (r * d * 4 + 255) / 256 * 256;
        plan.bytes = plan.part_o_bytes + (r * 4 + 255) / 256 * 256;
    }
    return plan;
}

void paged_divisors(PagedParams& p) {
    const unsigned per = static_cast<unsigned>(p.Nq * p.G), all = static_cast<unsigned>(p.B) * per;
    p.by_G = FastDiv(p.G);
    p.by_per = FastDiv(per);
    p.by_heads = FastDiv(p.H_kv);
    p.by_prefix_parts = FastDiv(std::max(p.prefix_parts, 1));
    p.by_own_parts = FastDiv(p.own_parts);
    const auto stream = [&](unsigned rows) { return FastDiv((rows + p.stream_tile - 1) / p.stream_tile); };
    p.by_prefix_rows = stream(all);
    p.by_own_rows = stream(per);
    // (one row tile, d < 256: two streams halve a CTA's keys; more: a CTA takes two)
    const auto tiles = [&](unsigned rows, int ctas, FastDiv& groups, FastDiv& shares) {
        const unsigned n = (rows + 127) / 128;
        groups = FastDiv(p.d == 256 ? n : (n + 1) / 2);
        shares = FastDiv(static_cast<unsigned>(std::max(ctas, 1)) * (p.d != 256 && n == 1 ? 2 : 1));
    };
    tiles(all, p.prefix_ctas, p.by_prefix_groups, p.by_prefix_shares);
    tiles(per, p.own_ctas, p.by_own_groups, p.by_own_shares);
}

namespace {

// W warps per row, D / 32 columns a lane; lane x of a warp has the weight of part
// 32 k + x; the warp sums the parts x = w, w + W, .., four at a time (independent
// loads), and the warps' sums meet in shared memory.
template <int D, int W>
__global__ void __launch_bounds__(128) paged_merge_kernel(const __grid_constant__ PagedParams p) {
    constexpr int V = D / 32;
    __shared__ float joined[4][D];
    const long long rows = static_cast<long long>(p.B) * p.Nq * p.H;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long row = static_cast<long long>(blockIdx.x) * (4 / W) + warp / W;
    const int w = warp % W;
    const int parts = p.prefix_parts + p.own_parts;
    const bool in = row < rows;
    wait_prerequisites();
    float sum = 0.0f, ref = 0.0f, acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.0f;
    if (in) {
        // The first 128 parts' weights stay in registers; there are seldom more.
        auto part_lse = [&](int k) {
            const int x = 32 * k + lane;
            return x < parts ? p.part_lse[x * rows + row] : -INFINITY;
        };
        float l2[4], mm = -INFINITY;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            l2[k] = part_lse(k);
            mm = fmaxf(mm, l2[k]);
        }
        for (int k = 4; 32 * k < parts; ++k) mm = fmaxf(mm, part_lse(k));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
        ref = mm == -INFINITY ? 0.0f : mm;
        auto add = [&](int k, float lse2) {
            const float wt = lse2 == -INFINITY ? 0.0f : ex2_approx(lse2 - ref);
            sum += wt;
            const int n = min(32, parts - 32 * k);
            for (int x = w; x < n; x += 4 * W) {
                float f[4][V], g[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int at = x + y * W;
                    g[y] = __shfl_sync(0xffffffffu, wt, at & 31);
                    if (at >= n) g[y] = 0.0f;
                    // an empty part's O was not written: it is not read
                    const float* src = p.part_o + (static_cast<long long>(32 * k + at) * rows + row) * D + lane * V;
#pragma unroll
                    for (int v = 0; v < V; ++v) f[y][v] = 0.0f;
                    if (g[y] != 0.0f) {
                        if constexpr (V == 2) {
                            const float2 q = *reinterpret_cast<const float2*>(src);
                            f[y][0] = q.x;
                            f[y][1] = q.y;
                        } else {
#pragma unroll
                            for (int v = 0; v < V; v += 4) {
                                const float4 q = *reinterpret_cast<const float4*>(src + v);
                                f[y][v] = q.x;
                                f[y][v + 1] = q.y;
                                f[y][v + 2] = q.z;
                                f[y][v + 3] = q.w;
                            }
                        }
                    }
                }
#pragma unroll
                for (int y = 0; y < 4; ++y)
#pragma unroll
                    for (int v = 0; v < V; ++v) acc[v] += g[y] * f[y][v];
            }
        };
        add(0, l2[0]);
        if (parts > 32) add(1, l2[1]);
        if (parts > 64) add(2, l2[2]);
        if (parts > 96) add(3, l2[3]);
        for (int k = 4; 32 * k < parts; ++k) add(k, part_lse(k));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if constexpr (W > 1) {
#pragma unroll
        for (int v = 0; v < V; ++v) joined[warp][lane * V + v] = acc[v];
        __syncthreads();
        if (w != 0) return;
#pragma unroll
        for (int x = 1; x < W; ++x)
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v] += joined[warp + x][lane * V + v];
    }
    if (!in) return;
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.o) + row * D + lane * V);
#pragma unroll
    for (int v = 0; v < V; v += 2) dst[v / 2] = pack_bf16x2(acc[v] * inv, acc[v + 1] * inv);
    if (lane == 0) {
        const unsigned r = static_cast<unsigned>(row);
        const unsigned h = r % p.H, bi = r / p.H, i = bi % p.Nq, b = bi / p.Nq;
        p.lse[(b * p.H + h) * p.Nq + i] = sum == 0.0f ? -INFINITY : (ref + __log2f(sum)) * 0.69314718055994530942f;
    }
}

template <int D>
cudaError_t merge_d(const PagedParams& p, cudaStream_t stream) {
    const long long rows = static_cast<long long>(p.B) * p.Nq * p.H;
    // A warp sums 8 parts in two rounds of loads; with more, four warps share
    // a row (16 rows of 28 parts: 25.5 us against 28.1 for the whole call; 32768
    // rows of 2 parts: 169 us with four warps, 149 with one).
    if (p.prefix_parts + p.own_parts > 8)
        return launch_kernel(paged_merge_kernel<D, 4>, static_cast<unsigned>(rows), 128, 0, true, stream, p);
    return launch_kernel(paged_merge_kernel<D, 1>, static_cast<unsigned>((rows + 3) / 4), 128, 0, true, stream, p);
}

}  // namespace

cudaError_t run_paged_merge(const PagedParams& p, cudaStream_t stream) {
    return p.d == 64 ? merge_d<64>(p, stream) : p.d == 128 ? merge_d<128>(p, stream) : merge_d<256>(p, stream);
}

}  // namespace attn
