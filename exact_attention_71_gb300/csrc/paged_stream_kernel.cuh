// Attention of a few query rows against a key range of the paged cache: the
// memory-bound side of the paged attention (decoding steps).
//
//     m = max_j s_j,  l = sum_j exp2(s_j - m),  O = sum_j exp2(s_j - m) v_j / l
//     s_j = scale * log2(e) * q . k_j        (times k's row scale: e4m3 cache)
//
// taken in one pass over the keys with a running m, l and O.
//
// A CTA serves 8 or 16 query rows of one key/value head (the group's heads of
// one sequence, or rows of several sequences over the prefix they share) and one
// key range; its four warps take the range's 16-key steps in turn, each with
// its own m, l and O, joined once at the end.  Every key row is read once per
// CTA, so the bound is the cache's bytes: at 8 rows a step does 8 FLOP per
// byte of K and V (bf16), a thirtieth of what the tensor cores could do per
// byte of HBM bandwidth.  The products therefore use the warp-level m16n8k16
// MMA with operands in registers: tcgen05 would leave 120 of its 128 tile rows
// empty and need the tile to be assembled in shared memory first.
//
// The keys and the value columns are the 16 rows of the products, the queries
// the 8 columns: S^T = K Q^T, O^T = V^T P^T.  (The other way round 4 query rows
// of a group would fill a quarter of 16 and every product cost twice as much.)
//
// Way in: 16 rows of one head of one page are contiguous, so a warp's step is a
// few TMA boxes of 16 rows (bf16: 64 columns, e4m3: up to 128), written with the
// 128-byte swizzle (64 for 64-byte rows) into the warp's own ring and awaited on
// the warp's own barriers: nothing crosses warps, no thread computes addresses.
// (Copying 16 bytes a thread with cp.async moved 1.5 times the bytes through the
// L2 and kept the load/store pipe busy: one sequence of 16384 tokens, 16 heads of
// 128, bf16, took 36 us instead of 27.)
//
// Measured at d = 128: that sequence now 24.7 us, 5.4 TB/s; 8 heads with 4 query
// heads each, 16 sequences of 23551 tokens on average, bf16 216 us, 7.2 TB/s, e4m3
// 122 us, 6.5 TB/s; 32 sequences of 3143, bf16 66 us, 6.3 TB/s, e4m3 43 us, 5.0
// TB/s.  Long ranges are bound by HBM; e4m3 also by its instructions (500 a step of
// 32 keys, 128 of which convert codes), short ranges by a CTA's latency (page
// table, first copy, join).
// The MMA's k index may be permuted freely (both operands alike), and so may O's
// columns and the keys, so each thread takes whole 16-byte chunks from the rows
// that its fragments need, chosen so that the 8 threads of a shared-memory phase
// meet 8 different chunk columns of the swizzle:
//   S^T = K Q^T      thread (g, t) = (lane / 4, lane % 4) reads key rows pi(g) and
//                    8 + pi(g), 16-byte chunks 4c + t;  pi(g) = g / 2 + 4 (g % 2)
//   O^T += V^T P^T   value rows t, t + 4, t + 8, t + 12 (the keys pi(2t), pi(2t + 1),
//                    ..), chunks 8c + pi(g); pairs of rows are interleaved by byte
//                    permutes, and P^T is S^T's 8 x 8 blocks transposed
//
// Trees (attn_fwd_paged_tree): the mask of a row is a limit, the tokens before the
// drafts, and a word of bits, its node's path: up to 32 rows have up to 32 nodes.  Every
// warp finds the paths by itself, a node a lane, by doubling, while its first copies are
// on their way; steps before the drafts are not masked, so a tree costs what a chain of as
// many drafts does (27 drafts x 16 heads of 64 for each of 7 sequences of up to 2333
// tokens 19.9 us, a chain 19.3).
#pragma once

#include <cuda_bf16.h>

#include "paged.cuh"
#include "sm103_bulk.cuh"
#include "sm103_ptx.cuh"

namespace attn {

// 16 bytes global -> shared; nothing is read and zeros are written when `valid`
// is false.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// D (16 x 8, fp32) += A (16 x 16) B (16 x 8), fp16 or bf16 operands.
template <bool F16>
__device__ __forceinline__ void mma_m16n8k16(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1) {
    if constexpr (F16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transposes an 8 x 8 matrix of 16-bit elements (thread (g, t): row g, columns 2t
// and 2t + 1).
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t a) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
    return r;
}

// An e4m3 cache is multiplied in fp16.  e4m3 values are fp16 values, and one
// instruction converts two codes (to bf16 it takes four, which bounded the
// kernels: 3.5 TB/s).  The other operands are brought into fp16's range by exact
// powers of two:
//   q    per row, so that its largest element lies in [2^14, 2^15): every bf16
//        element down to 2^-31 of the largest is then exact
//   P    times V's row scale / vref, a power of two that follows the scales and
//        keeps the product below 2^15; rounded once to fp16 (2^-11; below 2^-14,
//        2^-25 absolute, 2^-29 of the largest scale)
// (The warp-level e4m3 products, which would take K as it is, are slower here: 32
// sequences of 3143 tokens, d = 128, 45 us against 43, with 16 rows 71 against 52.)
__device__ __forceinline__ uint32_t f16x2_of_lo(uint32_t codes) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(codes));
    return r;
}
__device__ __forceinline__ uint32_t f16x2_of_hi(uint32_t codes) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(codes));
    return r;
}

// 2^n as a float, n in [-126, 127].
__device__ __forceinline__ float pow2f(int n) { return __uint_as_float(static_cast<uint32_t>(n + 127) << 23); }

// The power of two that brings a row of largest magnitude `bits` (bf16 bits) into
// [2^to, 2^(to + 1)), as its exponent: 0 for rows of zeros or with an infinity or a
// NaN (which stay what they are).
__device__ __forceinline__ int q_shift(uint32_t bits, int to) {
    const int e = static_cast<int>(bits >> 7);
    if (e == 255 || bits == 0) return 0;
    return max(-126, min(126, 127 + to - max(e, 1)));
}

// Eight bf16 times a power of two that brings them below 2^8 -> two e4m3 parts of
// each, x = q1 + q2.  x 2^-8 as an fp16 number has e4m3's exponent, its subnormal
// ones included, so its leading bits are the code: q1 has the first four of x's
// eight significant bits, q2 the rest, exact for |x| >= 2^-2 (2^-9 of the row's
// largest at most); below that q2 is rounded to e4m3's 2^-9.  A factor of NaN makes
// q1 NaN.
__device__ __forceinline__ uint32_t e4m3_of_bits(uint32_t a, uint32_t b) {
    const uint32_t x = a << 1 | (a & 0x80008000u), y = b << 1 | (b & 0x80008000u);
    return __byte_perm(x, y, 0x7531);
}
__device__ __forceinline__ void q_split(const uint4& v, float factor, uint2& q1, uint2& q2) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    const float f = factor * 0x1p-8f;
    uint32_t a[4], b[4];
#pragma unroll
    for (int y = 0; y < 4; ++y) {
        const uint32_t x = pack_f16x2(__uint_as_float(w[y] << 16) * f, __uint_as_float(w[y] & 0xffff0000u) * f);
        a[y] = x & 0xff80ff80u;
        b[y] = sub_f16x2(x, a[y]) + 0x00400040u;       // (half of the last bit that is kept)
    }
    q1 = make_uint2(e4m3_of_bits(a[0], a[1]), e4m3_of_bits(a[2], a[3]));
    q2 = make_uint2(e4m3_of_bits(b[0], b[1]), e4m3_of_bits(b[2], b[3]));
}

// sum + four bf16 times four e4m3 codes.
__device__ __forceinline__ float dot4(const uint2& q, uint32_t codes, float sum) {
    const float2 lo = f16x2_to_float2(f16x2_of_lo(codes)), hi = f16x2_to_float2(f16x2_of_hi(codes));
    sum = fmaf(__uint_as_float(q.x << 16), lo.x, sum);
    sum = fmaf(__uint_as_float(q.x & 0xffff0000u), lo.y, sum);
    sum = fmaf(__uint_as_float(q.y << 16), hi.x, sum);
    return fmaf(__uint_as_float(q.y & 0xffff0000u), hi.y, sum);
}

// Eight bf16 times a power of two -> eight fp16.
__device__ __forceinline__ uint4 q_to_f16(const uint4& v, float factor) {
    uint4 r;
    const uint32_t* in = &v.x;
    uint32_t* out = &r.x;
#pragma unroll
    for (int y = 0; y < 4; ++y)
        out[y] = pack_f16x2(__uint_as_float(in[y] << 16) * factor, __uint_as_float(in[y] & 0xffff0000u) * factor);
    return r;
}

// The largest magnitude of eight bf16, as bf16 bits (unsigned comparison orders
// finite < inf < NaN).
__device__ __forceinline__ uint32_t bf16x8_amax(const uint4& v) {
    constexpr uint32_t kAbs = 0x7fff7fffu;
    const uint32_t m = __vmaxu2(__vmaxu2(v.x & kAbs, v.y & kAbs), __vmaxu2(v.z & kAbs, v.w & kAbs));
    return max(m & 0xffffu, m >> 16);
}

// vref for a largest V scale vm: 2^4 below it, so that P vs / vref is at most
// 2^8 * 2^5 until a scale is more than 2^2 above it (then vref moves).
__device__ __forceinline__ float vref_of(float vm) {
    const int e = static_cast<int>(__float_as_uint(vm) >> 23) - 127;
    return pow2f(max(-126, min(120, e - 4)));
}

template <int D_, bool FP8_, int R_>
struct StreamCfg {
    static constexpr int D = D_;
    static constexpr bool FP8 = FP8_;
    static constexpr int R = R_, ROWS = 8 * R;                     // query rows: R tiles of 8
    static constexpr int ES = FP8 ? 1 : 2;
    static constexpr int ROW = D * ES;                             // bytes of a row
    static constexpr int SW = ROW >= 128 ? 128 : 64;               // swizzle span: bytes of a box row
    static constexpr int NB = ROW / SW;                            // boxes of 16 rows
    static constexpr int E = 16 / ES;                              // elements of a K chunk
    static constexpr int KC = D / (4 * E);                         // K chunks per row and thread
    static constexpr int VB = ROW / 8 >= 16 ? 16 : 8;              // bytes of a V chunk
    static constexpr int VE = VB / ES;
    static constexpr int VC = D / (8 * VE);                        // V chunks per row and thread
    static constexpr int WARPS = 4;
    static constexpr int THREADS = WARPS * 32;
    // 16-key blocks of a warp's step.  e4m3 steps are bound by instructions: two
    // blocks share the waits, the copies' issue and the running maximum (d = 64:
    // 30 us against 38).  bf16 steps are bound by bytes, and small steps fill the
    // ring more evenly (d = 128: 66 us against 68); so are e4m3 steps at d = 256 (81
    // against 83, and 51 against 68 where sequences are short).
    static constexpr int H = FP8 && D <= 128 ? 2 : 1;
    static constexpr int STEP = 16 * H;
    static constexpr int TILE = 16 * ROW;                          // a block's K or V rows
    static constexpr int SCALES = FP8 ? 128 : 0;                   // its 16 K and 16 V scales
    static constexpr int CTAS = D == 64 ? 4 : D == 128 ? 3 : FP8 ? (R == 1 ? 3 : 2) : 1;     // per SM
    static constexpr int STAGES = D == 64 ? 3 : D == 128 ? 2 : FP8 ? (R == 1 ? 2 : 3) : 3;
    static constexpr int STAGE_BYTES = H * 2 * TILE;               // (block, K / V, TILE)
    static constexpr int WARP_BYTES = STAGES * STAGE_BYTES;
    static constexpr int RING_BYTES = WARPS * WARP_BYTES;
    static constexpr int JD = D + 4;                               // row stride of the join (banks)
    static constexpr int JOIN_BYTES = WARPS * ROWS * (JD + 2) * 4;
    static constexpr int MAIN_BYTES = RING_BYTES > JOIN_BYTES ? RING_BYTES : JOIN_BYTES;
    static constexpr int SCALE_BYTES = WARPS * STAGES * H * SCALES;
    static constexpr int Q_BYTES = FP8 ? ROWS * D * 2 : 0;
    static constexpr int SMEM_BYTES = 1024 + MAIN_BYTES + SCALE_BYTES + Q_BYTES + WARPS * STAGES * 8;
    static constexpr int NT = D / 16;                              // O's column tiles
    // Chains of products that S is summed in (d = 256, bf16: 137 us with two, 140 with
    // one; at d = 128 their registers cost more: 16 rows 72 us with one, 77 with two).
    static constexpr int CH = D == 256 && !FP8 ? 2 : 1;
    // e4m3: Q's fragments are read from shared memory where registers are short.
    static constexpr bool QREG = !FP8 || R * D <= 128;
    static_assert(CTAS * (SMEM_BYTES + 1024) <= 228 * 1024, "shared memory");
};

enum : int { SITE_STREAM_FULL = 0xb1, SITE_STREAM_DRAIN = 0xb2 };

// Bounded wait of a whole warp.
__device__ __forceinline__ bool stream_wait(uint64_t* bar, uint32_t parity, unsigned long long limit, int* status,
                                            int site) {
    bool ok = mbar_try_wait(bar, parity);
    if (!__all_sync(0xffffffffu, ok)) {
        const long long t0 = clock64();
        while (!ok) {
            ok = mbar_try_wait(bar, parity);
            if (!ok && static_cast<unsigned long long>(clock64() - t0) > limit) {
                atomicCAS(status, 0, site);
                break;
            }
        }
        ok = __all_sync(0xffffffffu, ok);
    }
    return ok;
}

// Byte offset of the 16-byte chunk c of row r in a step's tile.
template <class Cfg>
__device__ __forceinline__ uint32_t stream_chunk(int r, int c) {
    constexpr int PER = Cfg::SW / 16;
    const int x = Cfg::SW == 128 ? (c % PER) ^ (r & 7) : (c % PER) ^ ((r >> 1) & 3);
    return static_cast<uint32_t>((c / PER) * (16 * Cfg::SW) + r * Cfg::SW + (x << 4));
}

// One warp's pass over a step's V rows: those from n on become 0 (stale),
// infinities and NaN in those from `diag` on become 0; bit r of the result: row r
// had one.
template <class Cfg>
__device__ __noinline__ uint32_t fix_v_step(uint8_t* tile, int n, int diag, int lane) {
    constexpr int CPR = Cfg::ROW / 16;
    uint32_t hit = 0;
    for (int x = lane; x < 16 * CPR; x += 32) {
        const int r = x / CPR;
        if (r < n && r < diag) continue;
        uint4* at = reinterpret_cast<uint4*>(tile + stream_chunk<Cfg>(r, x % CPR));
        uint4 v = r < n ? *at : make_uint4(0, 0, 0, 0);
        uint32_t* w = &v.x;
        bool bad = false;
        for (int y = 0; y < 4; ++y) {
            if constexpr (Cfg::FP8) {
                const uint32_t nan = __vcmpeq4(w[y] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                w[y] &= ~nan;
                bad |= nan != 0;
            } else {
                if ((w[y] & 0x7f80u) == 0x7f80u) { w[y] &= 0xffff0000u; bad = true; }
                if ((w[y] & 0x7f800000u) == 0x7f800000u) { w[y] &= 0xffffu; bad = true; }
            }
        }
        *at = v;
        if (bad) hit |= 1u << r;
    }
    fence_proxy_async_smem();              // the ring slot's next copy comes after these writes
    __syncwarp();
    return __reduce_or_sync(0xffffffffu, hit);
}

// The paths of a tree of up to 32 nodes: lane j has node j's parent (past them: -2); the result is
// lane j's nodes (its ancestors and itself; bit: node), 0 where j is no node.  Whole
// warp.  A path that leaves the tree, meets no node or runs in a circle is reported.
__device__ __forceinline__ uint32_t tree_paths32(const PagedParams& p, int parent, int lane, bool tell) {
    // After r rounds: the first 2^r nodes of the path, and the one that follows.
    uint32_t path = 1u << lane;
    int at = parent < p.Nq ? parent : -2;
    for (int span = 1; span < p.Nq; span <<= 1) {
        const uint32_t more = __shfl_sync(0xffffffffu, path, at & 31);
        const int next = __shfl_sync(0xffffffffu, at, at & 31);
        if (at >= 0) {
            path |= more;
            at = next;
        }
    }
    if (at != -1 && parent >= -1 && tell) atomicCAS(p.status, 0, SITE_TREE_PARENT);
    return at == -1 ? path : 0;
}

// DIRECT: the own tokens are one part and there is no prefix: o and lse are
// written; otherwise partial results.  Blocks below prefix_blocks have the
// prefix and all sequences' rows, the others one sequence's own tokens.
// TREE: the last Nq own tokens are nodes of a tree: a row sees those of its path.
template <class Cfg, bool DIRECT, bool TREE>
__global__ void __launch_bounds__(Cfg::THREADS, Cfg::CTAS)
    paged_stream_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                        const __grid_constant__ PagedParams p, const unsigned prefix_blocks) {
    constexpr int D = Cfg::D, KC = Cfg::KC, VC = Cfg::VC, NT = Cfg::NT, STAGES = Cfg::STAGES, R = Cfg::R;
    constexpr bool FP8 = Cfg::FP8;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    // Permutations of the swizzled layout (see above); 64-byte rows need none.
    constexpr bool PI = Cfg::SW == 128;
    const int pig = PI ? (g >> 1) | ((g & 1) << 2) : g;            // K row (key of S^T row g), V chunk
    const int ka = PI ? t : 2 * t, kb = PI ? t + 4 : 2 * t + 1;    // keys of P^T rows 2t, 2t + 1

    launch_dependents();
    unsigned x0 = blockIdx.x;
    const bool prefix = !DIRECT && x0 < prefix_blocks;
    if (!prefix) x0 -= prefix_blocks;
    const int rows = (prefix ? p.B : 1) * p.Nq * p.G;
    const FastDiv by_tiles = prefix ? p.by_prefix_rows : p.by_own_rows, by_parts = prefix ? p.by_prefix_parts : p.by_own_parts;
    const int parts = by_parts.d;
    // Row tiles and heads of the same pages run next to one another.
    unsigned y0 = by_tiles.div(x0);
    const int tile = x0 - y0 * by_tiles.d;
    x0 = p.by_heads.div(y0);
    const int kvh = y0 - x0 * p.H_kv;
    y0 = by_parts.div(x0);
    const int part = x0 - y0 * parts;
    const int seq = prefix ? 0 : y0;

    // The key range.
    int len = prefix ? p.prefix_len : __ldg(p.seq_lens + seq);
    if (!prefix) {
        const long long room = static_cast<long long>(p.max_pages) << p.page_shift;
        if (len > room) {
            if (tid == 0) atomicCAS(p.status, 0, SITE_PAGED_LENGTH);
            len = static_cast<int>(room);
        }
        len = max(len, 0);
    }
    const int chunk = max((static_cast<int>(by_parts.div(len + parts - 1)) + 63) / 64 * 64, own_chunk(D));
    const int k0 = static_cast<int>(min(static_cast<long long>(part) * chunk, static_cast<long long>(len)));
    const int k1 = min(k0 + chunk, len);
    const int* table = prefix ? p.prefix_table : p.table + seq * p.table_stride;

    constexpr int H = Cfg::H, STEP = Cfg::STEP, STRIDE = STEP * Cfg::WARPS;
    const int first = k0 + warp * STEP;                    // this warp's steps: keys first, first + STRIDE, ...
    const int end = k0 < k1 ? k1 : 0;                      // (an empty range ends at len, inside a step)
    uint8_t* ring = smem + warp * Cfg::WARP_BYTES;
    float* scales = reinterpret_cast<float*>(smem + Cfg::MAIN_BYTES + warp * STAGES * H * Cfg::SCALES);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + Cfg::MAIN_BYTES + Cfg::SCALE_BYTES + Cfg::Q_BYTES) + warp * STAGES;
    if (lane == 0) {
        for (int s = 0; s < STAGES; ++s) mbar_init(full + s, 1);
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    __syncwarp();

    // Lane 2h + v (v: V instead of K) looks up the page of a step's block h and
    // copies its rows.
    const int my_block = lane >> 1;
    const bool my_v = lane & 1;
    const uint64_t policy = l2_policy_evict_first();
    const CUtensorMap* my_map = my_v ? &tmap_v : &tmap_k;
    uint32_t gone = 0;                                     // bit H * (round & 7) + h: the block's page is refused
    auto page_of = [&](int key) -> int {
        const int at = key + my_block * 16;
        return my_block < H && at < end ? __ldg(table + (at >> p.page_shift)) : -1;
    };
    auto issue = [&](int key, int stage, int round, int page) {
        if (key >= end) return;
        const int at = key + my_block * 16;
        const bool want = my_block < H && at < end;
        const bool have = want && page >= 0 && page < p.num_pages;
        const uint32_t copies = __ballot_sync(0xffffffffu, have), wanted = __ballot_sync(0xffffffffu, want);
        if (copies != wanted) {
            if (lane == 0) atomicCAS(p.status, 0, SITE_PAGED_PAGE);
        }
        uint32_t bits = 0;
#pragma unroll
        for (int h = 0; h < H; ++h) bits |= (copies >> (2 * h)) & 1u ? 0u : 1u << h;
        const int sh = H * (round & 7);
        gone = (gone & ~(((1u << H) - 1u) << sh)) | (bits << sh);
        if (lane == 0) mbar_arrive_expect_tx(full + stage, __popc(copies) * (Cfg::TILE + Cfg::SCALES / 2));
        __syncwarp();
        if (have) {
            const int row = at & ((1 << p.page_shift) - 1);
            uint8_t* dst = ring + stage * Cfg::STAGE_BYTES + lane * Cfg::TILE;
            if constexpr (FP8) {
                const long long r = ((static_cast<long long>(page) * p.H_kv + kvh) << p.page_shift) + row;
                bulk_load(scales + (stage * H * 2 + lane) * 16, (my_v ? p.v_scale : p.k_scale) + r, 64, full + stage);
            }
#pragma unroll
            for (int b = 0; b < Cfg::NB; ++b)
                tma_load_4d(dst + b * 16 * Cfg::SW, my_map, full + stage, b * (Cfg::SW / Cfg::ES), row, kvh, page, policy);
        }
    };
    {
        // The first steps' pages together, then their copies.
        int pages[STAGES];
#pragma unroll
        for (int s = 0; s < STAGES; ++s) pages[s] = page_of(first + STRIDE * s);
#pragma unroll
        for (int s = 0; s < STAGES; ++s) issue(first + STRIDE * s, s, s, pages[s]);
    }
    int next_page = page_of(first + STRIDE * STAGES);

    // Query row r of the tile: its index in q and o, and the keys it sees.
    const int per = p.Nq * p.G;
    const int live = min(Cfg::ROWS, rows - tile * Cfg::ROWS);            // rows of this tile
    auto row_of = [&](int r, long long& out, int& lse_at) -> int {
        const int x = tile * Cfg::ROWS + r;
        const int y = prefix ? p.by_per.div(x) : 0, z = x - y * per;               // row z of its sequence
        const int b = prefix ? y : seq, i = p.by_G.div(z), h = kvh * p.G + z - i * p.G;
        out = (static_cast<long long>(b) * p.Nq + i) * p.H + h;
        lse_at = (b * p.H + h) * p.Nq + i;
        return i;
    };
    int limit[R][2];               // keys that rows 8n + 2t and 8n + 2t + 1 see
    // TREE: and of the keys from `nodes` on (< 0: the first nodes are not there) those of
    // these bits.
    const int nodes = len - p.Nq, start = TREE && !prefix ? max(nodes, 0) : len;
    uint32_t path[TREE ? R : 1][2];
    __shared__ uint32_t row_path[TREE ? Cfg::ROWS : 1];
    if constexpr (TREE) {
        const int parent = !prefix && lane < p.Nq ? __ldg(p.parents + seq * p.parents_stride + lane) : -2;
        const uint32_t paths = prefix ? 0 : tree_paths32(p, parent, lane, warp == 0);
#pragma unroll
        for (int n = 0; n < R; ++n)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                const int r = 8 * n + 2 * t + z;
                long long out;
                int at, i = 0;
                if (!prefix && r < live) i = row_of(r, out, at);
                path[n][z] = __shfl_sync(0xffffffffu, paths, i & 31);
                if (r >= live) path[n][z] = 0;
                if (warp == 0 && g == 0) row_path[r] = path[n][z];
            }
    }
    float to_log2[R][2];           // raw score -> log2 units
    uint32_t qb[R][Cfg::QREG ? D / 8 : 1];         // row 8n + g: chunk c of the k permutation, elements [c * 4E + t * E, + E)
    uint4* sq = reinterpret_cast<uint4*>(smem + Cfg::MAIN_BYTES + Cfg::SCALE_BYTES);
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q);
    auto row_at = [&](int r) -> const uint4* {
        if (r >= live) return nullptr;
        long long out;
        int at;
        row_of(r, out, at);
        return reinterpret_cast<const uint4*>(q + out * D);
    };
#pragma unroll
    for (int n = 0; n < R; ++n) {
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            const int r = 8 * n + 2 * t + z;
            long long out;
            int at, i = 0;
            if (r < live) i = row_of(r, out, at);
            if constexpr (TREE) limit[n][z] = r >= live || (!prefix && path[n][z] == 0) ? 0 : min(start, k1);
            else limit[n][z] = r >= live ? 0 : min(prefix || !p.causal ? len : max(0, len - p.Nq + 1 + i), k1);
            to_log2[n][z] = p.scale_log2;
        }
        if constexpr (!FP8) {
            const uint4* src = row_at(8 * n + g);
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                const uint4 v = src ? __ldg(src + c * 4 + t) : make_uint4(0, 0, 0, 0);
                qb[n][c * 4] = v.x;
                qb[n][c * 4 + 1] = v.y;
                qb[n][c * 4 + 2] = v.z;
                qb[n][c * 4 + 3] = v.w;
            }
        }
    }
    // Whether row 8n + 2t + z sees a key of the range.
    const auto visible = [&](int key, int n, int z) {
        if constexpr (TREE)
            return key < limit[n][z] || (key >= start && key < k1 && ((path[n][z] >> ((key - nodes) & 31)) & 1u));
        else
            return key < limit[n][z];
    };
    __shared__ uint32_t loud;              // e4m3: keys from diag on (32 at most) whose values are added at the end
    if constexpr (FP8) {
        // To fp16, once per CTA: a warp takes 2R rows, eight lanes a row, and
        // writes them as fragments (chunk half, row tile, lane).
        __shared__ float row_log2[Cfg::ROWS];
        if (tid == 0) loud = 0;
        const int r = warp * (2 * R) + (lane >> 3);
        const bool mine = (lane >> 3) < 2 * R;
        uint4 v[D / 64];
        uint32_t top = 0;
        const uint4* src = mine ? row_at(r) : nullptr;
#pragma unroll
        for (int y = 0; y < D / 64; ++y) {
            v[y] = src ? __ldg(src + y * 8 + (lane & 7)) : make_uint4(0, 0, 0, 0);
            top = max(top, bf16x8_amax(v[y]));
        }
#pragma unroll
        for (int y = 1; y < 8; y <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, y));
        const int shift = q_shift(top, 14);
        if (mine) {
            // (not 0: -inf, the masked score, stays -inf when multiplied)
            if ((lane & 7) == 0) row_log2[r] = fmaxf(p.scale_log2 * pow2f(-shift), 0x1p-126f);
#pragma unroll
            for (int y = 0; y < D / 64; ++y) {
                const int i8 = y * 8 + (lane & 7);         // eight elements: chunk i8 / 8, thread (i8 / 2) % 4, half i8 % 2
                const int at = (i8 >> 3) * 2 + (i8 & 1);
                sq[(at * R + (r >> 3)) * 32 + (r & 7) * 4 + ((i8 >> 1) & 3)] = q_to_f16(v[y], pow2f(shift));
            }
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < R; ++n) {
            to_log2[n][0] = row_log2[8 * n + 2 * t];
            to_log2[n][1] = row_log2[8 * n + 2 * t + 1];
            if constexpr (Cfg::QREG) {
#pragma unroll
                for (int c = 0; c < 2 * KC; ++c) {
                    const uint4 v = sq[(c * R + n) * 32 + lane];
                    qb[n][c * 4] = v.x;
                    qb[n][c * 4 + 1] = v.y;
                    qb[n][c * 4 + 2] = v.z;
                    qb[n][c * 4 + 3] = v.w;
                }
            }
        }
    }
    // From this key on some query of the sequence does not see what another does
    // (of the sequence, not of the tile: which rows become NaN beside a value that is
    // not finite must not depend on the tiles).
    const int diag = TREE ? start : !prefix && p.causal ? max(0, len - p.Nq + 1) : len;
    // Steps that reach it (or the range's end) are masked key by key.
    const int plain_end = min(diag, k1);

    // O^T: o[j][n][z] and o[j][n][2 + z] are the elements 2j and 2j + 1 (of VE a
    // chunk) of query row 8n + 2t + z.
    float o[NT][R][4], m[R][2], l[R][2];
#pragma unroll
    for (int n = 0; n < R; ++n) {
#pragma unroll
        for (int j = 0; j < NT; ++j) o[j][n][0] = o[j][n][1] = o[j][n][2] = o[j][n][3] = 0.0f;
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.0f;
    }
    float vref = FP8 ? 0.0f : 1.0f;

    // Shared-memory offsets of this thread's chunks (SW = 128: the chunk's column
    // is xor-ed with the row, so the next four columns, and the rows four below,
    // are one xor of 64 away).
    uint32_t koff[2], voff[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        koff[x] = stream_chunk<Cfg>(pig, 4 * x + t) % (16 * Cfg::SW);
        const int r = x ? kb : ka;
        voff[x] = Cfg::VB == 16 ? stream_chunk<Cfg>(r, pig) : stream_chunk<Cfg>(r, g >> 1) + (g & 1) * 8;
    }

    int stage = 0, round = 0;
    uint32_t parity = 0;
    bool ok = true;
    int key0 = first;
    for (; key0 < end; key0 += STRIDE, ++round) {
        const int page = next_page;
        next_page = page_of(key0 + STRIDE * (STAGES + 1));
        if (!(ok = stream_wait(full + stage, parity, p.wait_limit, p.status, SITE_STREAM_FULL))) break;
        uint8_t* st = ring + stage * Cfg::STAGE_BYTES;

        // -------------------------------------------------------- S^T = K Q^T
        // s[h][n][z]: key 16h + pi(g), query row 8n + 2t + z; s[h][n][2 + z]: key 8 on.
        float s[H][R][4], s1[Cfg::CH == 2 ? H : 1][R][4];
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
            for (int n = 0; n < R; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[h][n][i] = 0.0f;
                    if constexpr (Cfg::CH == 2) s1[h][n][i] = 0.0f;
                }
#pragma unroll
        for (int c = 0; c < KC; ++c) {
            const uint32_t col = Cfg::SW == 128 ? koff[c & 1] + (c >> 1) * (16 * Cfg::SW) : koff[0];
            constexpr int W = FP8 ? 8 : 4;                 // Q's words of a chunk
            uint32_t qw[R][W];
#pragma unroll
            for (int n = 0; n < R; ++n)
#pragma unroll
                for (int y = 0; y < W / 4; ++y) {
                    if constexpr (Cfg::QREG) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) qw[n][4 * y + i] = qb[n][c * W + 4 * y + i];
                    } else {
                        const uint4 v = sq[((c * 2 + y) * R + n) * 32 + lane];
                        qw[n][4 * y] = v.x;
                        qw[n][4 * y + 1] = v.y;
                        qw[n][4 * y + 2] = v.z;
                        qw[n][4 * y + 3] = v.w;
                    }
                }
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const uint8_t* at = st + h * 2 * Cfg::TILE + col;
                const uint4 ka4 = *reinterpret_cast<const uint4*>(at);
                const uint4 kb4 = *reinterpret_cast<const uint4*>(at + 8 * Cfg::SW);
                const uint32_t a[4] = {ka4.x, ka4.y, ka4.z, ka4.w}, b[4] = {kb4.x, kb4.y, kb4.z, kb4.w};
#pragma unroll
                for (int y = 0; y < W / 2; ++y) {
#pragma unroll
                    for (int n = 0; n < R; ++n) {
                        float* d = Cfg::CH == 2 && (y & 1) ? s1[Cfg::CH == 2 ? h : 0][n] : s[h][n];
                        if constexpr (FP8)
                            mma_m16n8k16<true>(d, f16x2_of_lo(a[y]), f16x2_of_lo(b[y]), f16x2_of_hi(a[y]), f16x2_of_hi(b[y]),
                                               qw[n][2 * y], qw[n][2 * y + 1]);
                        else
                            mma_m16n8k16<false>(d, a[2 * y], b[2 * y], a[2 * y + 1], b[2 * y + 1], qw[n][2 * y],
                                                qw[n][2 * y + 1]);
                    }
                }
            }
        }
        const uint32_t miss = (gone >> (H * (round & 7))) & ((1u << H) - 1u);
        const bool special = miss != 0 || key0 + STEP > plain_end;
        float vscale[H][2];
#pragma unroll
        for (int h = 0; h < H; ++h) {
            float mul[2] = {1.0f, 1.0f};
            if constexpr (FP8) {
                const float* at = scales + (stage * H + h) * 32 + pig;
                mul[0] = at[0];
                mul[1] = at[8];
                vscale[h][0] = at[16];
                vscale[h][1] = at[24];
            }
#pragma unroll
            for (int n = 0; n < R; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (Cfg::CH == 2) s[h][n][i] += s1[h][n][i];
                    if constexpr (FP8) s[h][n][i] *= mul[i >> 1];
                }
        }
        if (special) {
            // A masked score is -inf whatever was read for it.
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const bool skip = (miss >> h) & 1u;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int key = key0 + 16 * h + 8 * x + pig;
#pragma unroll
                    for (int n = 0; n < R; ++n)
#pragma unroll
                        for (int z = 0; z < 2; ++z)
                            if (skip || !visible(key, n, z)) s[h][n][2 * x + z] = -INFINITY;
                    // (scales of rows that are not there)
                    if (FP8 && (skip || key >= k1)) vscale[h][x] = 0.0f;
                }
            }
            if (FP8 && key0 + STEP > diag && diag < len) {
                // vref must not follow a scale that some row does not see.  Every row
                // that sees a key of this warp sees the warp's first one, and those
                // before diag: these are what it starts from and follows.
                // (TREE: no node is seen by all that see another.  Where there are only
                // nodes, the smallest of their scales: no row's own are below it.)
                const int both = TREE ? diag : max(diag, first + 1);
                if (vref == 0.0f) {
                    float top = 0.0f;
#pragma unroll
                    for (int h = 0; h < H; ++h)
#pragma unroll
                        for (int x = 0; x < 2; ++x)
                            if (key0 + 16 * h + 8 * x + pig < both && vscale[h][x] < INFINITY) top = fmaxf(top, vscale[h][x]);
                    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
                    if (TREE && top == 0.0f) {
                        uint32_t low = 0x7f800000u;
#pragma unroll
                        for (int h = 0; h < H; ++h)
#pragma unroll
                            for (int x = 0; x < 2; ++x)
                                if (vscale[h][x] > 0.0f) low = min(low, __float_as_uint(vscale[h][x]));
                        low = __reduce_min_sync(0xffffffffu, low);
                        if (low < 0x7f800000u) top = __uint_as_float(low);
                    }
                    if (top > 0.0f) vref = vref_of(top);
                }
#pragma unroll
                for (int h = 0; h < H; ++h)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        // A scale far above vref: left out here, added at the end.  One
                        // that is not finite makes the rows that see it NaN as a whole,
                        // as a code that is NaN does (below).
                        const int key = key0 + 16 * h + 8 * x + pig;
                        if (key < diag || vscale[h][x] <= 64.0f * vref) continue;
                        if (vscale[h][x] < INFINITY) {
                            atomicOr(&loud, 1u << (key - diag));
                        } else {
#pragma unroll
                            for (int n = 0; n < R; ++n)
#pragma unroll
                                for (int z = 0; z < 2; ++z)
                                    if (visible(key, n, z)) l[n][z] = __uint_as_float(0x7fc00000u);
                        }
                        vscale[h][x] = 0.0f;
                    }
            }
        }
        // ------------------------------------------------------ running maximum
        // A row's reference moves only when a score of the row exceeds it by
        // more than 8 (log2 units), so that the shuffles and O's rescaling are
        // rare; O and l share the reference, so the result does not depend on it.
        float mx[R][2];
        bool move = false;
#pragma unroll
        for (int n = 0; n < R; ++n)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                mx[n][z] = fmaxf(s[0][n][z], s[0][n][2 + z]);
#pragma unroll
                for (int h = 1; h < H; ++h) mx[n][z] = fmax3(mx[n][z], s[h][n][z], s[h][n][2 + z]);
                mx[n][z] *= to_log2[n][z];
                move = move || mx[n][z] > m[n][z] + 8.0f;
            }
        float vm = 0.0f;
        if constexpr (FP8) {
#pragma unroll
            for (int h = 0; h < H; ++h) vm = fmax3(vm, vscale[h][0], vscale[h][1]);
            move = move || vm > 64.0f * vref;
        }
        if (__any_sync(0xffffffffu, move)) {
            float vfall = 1.0f;
            if constexpr (FP8) {
                // V scales are never negative: their bits order them.
                vm = __uint_as_float(__reduce_max_sync(0xffffffffu, vm > 0.0f ? __float_as_uint(vm) : 0u));
                if (vm > 64.0f * vref) {
                    const float to = vref_of(vm);
                    vfall = vref * (1.0f / to);                // (O is 0 while vref is)
                    vref = to;
                }
            }
#pragma unroll
            for (int n = 0; n < R; ++n)
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    float x = mx[n][z];
#pragma unroll
                    for (int y = 4; y < 32; y <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, y));
                    // (per row: a row's result does not depend on its neighbours)
                    const float was = m[n][z], mn = x > was + 8.0f ? x : was;
                    const float a = mn == was ? 1.0f : ex2_approx(was - mn);
                    m[n][z] = mn;
                    l[n][z] *= a;
                    const float ao = FP8 ? a * vfall : a;
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        o[j][n][z] *= ao;
                        o[j][n][2 + z] *= ao;
                    }
                }
        }
        const float iv = FP8 ? (vref == 0.0f ? 0.0f : 1.0f / vref) : 1.0f;         // a power of two
        uint32_t pb[H][R][2];          // P^T as the B operand of each block
#pragma unroll
        for (int n = 0; n < R; ++n) {
            const float n0 = m[n][0] == -INFINITY ? 0.0f : -m[n][0], n1 = m[n][1] == -INFINITY ? 0.0f : -m[n][1];
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float e0 = ex2_approx(fmaf(s[h][n][2 * x], to_log2[n][0], n0));
                    float e1 = ex2_approx(fmaf(s[h][n][2 * x + 1], to_log2[n][1], n1));
                    l[n][0] += e0;
                    l[n][1] += e1;
                    if constexpr (FP8) {
                        // V's row scale rides on P; l sums the plain weights.  A
                        // weight of 0 stays 0 beside a NaN scale: a row that does
                        // not see the key must not notice it.
                        const float vs = vscale[h][x] * iv;
                        if (special) {
                            e0 = e0 == 0.0f ? 0.0f : e0 * vs;
                            e1 = e1 == 0.0f ? 0.0f : e1 * vs;
                        } else {
                            e0 *= vs;
                            e1 *= vs;
                        }
                    }
                    // P is rounded for the product: to fp16 (see above), or to
                    // bf16 (2^-8 per weight, as in the dense forward); l keeps
                    // the unrounded values.
                    pb[h][n][x] = transpose_8x8(FP8 ? pack_f16x2(e0, e1) : pack_bf16x2(e0, e1));
                }
        }
        // ---------------------------------------------------------- O^T += V^T P^T
        if (special) {
            // 0 * NaN is NaN: stale rows become 0, and where rows of the tile see
            // different keys a non-finite value is taken out of the product and
            // the rows that do see its key become NaN as a whole.
#pragma unroll 1
            for (int h = 0; h < H; ++h) {
                const int at = key0 + h * 16;
                const uint32_t hit = fix_v_step<Cfg>(st + (2 * h + 1) * Cfg::TILE, (miss >> h) & 1u ? 0 : k1 - at, diag - at, lane);
#pragma unroll
                for (int n = 0; n < R; ++n)
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const int seen = min(max(limit[n][z] - at, 0), 16);
                        uint32_t sees = (1u << seen) - 1u;
                        if constexpr (TREE) {
                            // (key at + x is node at - nodes + x)
                            const int y = at - nodes;
                            if (!prefix) sees |= y >= 0 ? (y < 32 ? path[n][z] >> y : 0u) : (y > -16 ? path[n][z] << -y : 0u);
                        }
                        if (hit & sees) l[n][z] = __uint_as_float(0x7fc00000u);
                    }
            }
        }
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const uint8_t* sv = st + (2 * h + 1) * Cfg::TILE;
#pragma unroll
            for (int c = 0; c < VC; ++c) {
                uint32_t w[4][Cfg::VB / 4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    // value rows ka, kb, 8 + ka, 8 + kb
                    const uint8_t* at = sv + voff[x & 1] + (x >> 1) * 8 * Cfg::SW + c * 16 * Cfg::SW;
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
                    auto* oo = &o[(c * Cfg::VE + y * (4 / Cfg::ES)) / 2];
                    if constexpr (FP8) {
                        // codes of two rows, interleaved: elements 0, 1 and 2, 3
                        const uint32_t ab01 = __byte_perm(w[0][y], w[1][y], 0x5140), ab23 = __byte_perm(w[0][y], w[1][y], 0x7362);
                        const uint32_t cd01 = __byte_perm(w[2][y], w[3][y], 0x5140), cd23 = __byte_perm(w[2][y], w[3][y], 0x7362);
#pragma unroll
                        for (int n = 0; n < R; ++n) {
                            mma_m16n8k16<true>(oo[0][n], f16x2_of_lo(ab01), f16x2_of_hi(ab01), f16x2_of_lo(cd01),
                                               f16x2_of_hi(cd01), pb[h][n][0], pb[h][n][1]);
                            mma_m16n8k16<true>(oo[1][n], f16x2_of_lo(ab23), f16x2_of_hi(ab23), f16x2_of_lo(cd23),
                                               f16x2_of_hi(cd23), pb[h][n][0], pb[h][n][1]);
                        }
                    } else {
                        const uint32_t a0 = __byte_perm(w[0][y], w[1][y], 0x5410), a1 = __byte_perm(w[0][y], w[1][y], 0x7632);
                        const uint32_t a2 = __byte_perm(w[2][y], w[3][y], 0x5410), a3 = __byte_perm(w[2][y], w[3][y], 0x7632);
#pragma unroll
                        for (int n = 0; n < R; ++n) mma_m16n8k16<false>(oo[0][n], a0, a1, a2, a3, pb[h][n][0], pb[h][n][1]);
                    }
                }
            }
        }
        __syncwarp();
        issue(key0 + STRIDE * STAGES, stage, round + STAGES, page);
        if (++stage == STAGES) {
            stage = 0;
            parity ^= 1;
        }
    }
    if (!ok) {
        // A wait ran out: whatever copy is in flight lands before the CTA leaves.
        for (int s = 0; s < STAGES && key0 + STRIDE * s < end; ++s)
            stream_wait(full + (stage + s) % STAGES, parity ^ (stage + s >= STAGES ? 1u : 0u), 2000000000ull, p.status,
                        SITE_STREAM_DRAIN);
    }

    // ------------------------------------------------------------ join the warps
#pragma unroll
    for (int n = 0; n < R; ++n)
#pragma unroll
        for (int z = 0; z < 2; ++z) {
#pragma unroll
            for (int y = 4; y < 32; y <<= 1) l[n][z] += __shfl_xor_sync(0xffffffffu, l[n][z], y);
        }
    __syncthreads();                       // every warp is done with the ring
    constexpr int JD = Cfg::JD;
    float* js = reinterpret_cast<float*>(smem);                        // (warp, ROWS, JD)
    float* jm = js + Cfg::WARPS * Cfg::ROWS * JD;                      // (warp, ROWS)
    float* jl = jm + Cfg::WARPS * Cfg::ROWS;
#pragma unroll
    for (int n = 0; n < R; ++n)
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            const int r = 8 * n + 2 * t + z;
            if (r >= live) continue;
            float* dst = js + (warp * Cfg::ROWS + r) * JD;
#pragma unroll
            for (int c = 0; c < VC; ++c)
#pragma unroll
                for (int e = 0; e < Cfg::VE; e += 4) {
                    const int j = (c * Cfg::VE + e) / 2;
                    *reinterpret_cast<float4*>(dst + (c * 8 + pig) * Cfg::VE + e) =
                        make_float4(o[j][n][z] * vref, o[j][n][2 + z] * vref, o[j + 1][n][z] * vref, o[j + 1][n][2 + z] * vref);
                }
            if (g == 0) {
                jm[warp * Cfg::ROWS + r] = m[n][z];
                jl[warp * Cfg::ROWS + r] = l[n][z];
            }
        }
    __syncthreads();
    // A thread takes 4 columns of a row at a time; D / 4 threads a row.
    for (int x = tid; x < live * (D / 4); x += Cfg::THREADS) {
        const int rr = x / (D / 4), c4 = x % (D / 4);
        long long out;
        int lse_at;
        const int i = row_of(rr, out, lse_at);
        float mm = jm[rr];
#pragma unroll
        for (int w = 1; w < Cfg::WARPS; ++w) mm = fmaxf(mm, jm[w * Cfg::ROWS + rr]);
        const float ref = mm == -INFINITY ? 0.0f : mm;
        float ll = 0.0f;
        float4 acc = make_float4(0, 0, 0, 0);
#pragma unroll
        for (int w = 0; w < Cfg::WARPS; ++w) {
            const float a = ex2_approx(jm[w * Cfg::ROWS + rr] - ref);
            const float4 v = *reinterpret_cast<const float4*>(js + (w * Cfg::ROWS + rr) * JD + c4 * 4);
            ll += a * jl[w * Cfg::ROWS + rr];
            acc.x += a * v.x;
            acc.y += a * v.y;
            acc.z += a * v.z;
            acc.w += a * v.w;
        }
        if (FP8 && !prefix) {
            // (rare) Values whose scale is far above those that other rows of the tile
            // see; l has their weights.
#pragma unroll 1
            for (uint32_t bits = loud; bits; bits &= bits - 1) {
                const int key = diag + __ffs(bits) - 1;
                if constexpr (TREE) {
                    if (!((row_path[rr] >> ((key - nodes) & 31)) & 1u)) continue;
                } else if (key >= max(0, len - p.Nq + 1 + i)) {
                    break;
                }
                const long long at = ((static_cast<long long>(__ldg(table + (key >> p.page_shift))) * p.H_kv + kvh) << p.page_shift) +
                                     (key & ((1 << p.page_shift) - 1));
                const uint8_t* kc = static_cast<const uint8_t*>(p.k_cache) + at * D;
                float dot = 0.0f;
#pragma unroll 1
                for (int y = 0; y < D; y += 4)
                    dot = dot4(__ldg(reinterpret_cast<const uint2*>(q + out * D + y)), __ldg(reinterpret_cast<const uint32_t*>(kc + y)), dot);
                const float e = ex2_approx(dot * __ldg(p.k_scale + at) * p.scale_log2 - ref) * __ldg(p.v_scale + at);
                const uint32_t codes = __ldg(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(p.v_cache) + at * D + c4 * 4));
                const float2 lo = f16x2_to_float2(f16x2_of_lo(codes)), hi = f16x2_to_float2(f16x2_of_hi(codes));
                acc.x = fmaf(e, lo.x, acc.x);
                acc.y = fmaf(e, lo.y, acc.y);
                acc.z = fmaf(e, hi.x, acc.z);
                acc.w = fmaf(e, hi.y, acc.w);
            }
        }
        // TREE: a row that is no node has taken part in the steps before the drafts, which
        // are not masked.
        const bool none = TREE && !prefix && row_path[rr] == 0;
        if (none) {
            ll = 0.0f;
            acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
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
            if (c4 == 0) p.lse[lse_at] = lse2 * 0.69314718055994530942f;
        } else {
            const long long pr = static_cast<long long>(prefix ? part : p.prefix_parts + part) *
                                     (static_cast<long long>(p.B) * p.Nq * p.H) + out;
            // An empty part's O is not read by the join.
            if (lse2 != -INFINITY) reinterpret_cast<float4*>(p.part_o + pr * D)[c4] = acc;
            if (c4 == 0) p.part_lse[pr] = none ? kNoNode : lse2;
        }
    }
    // The join is launched after this kernel and waits for it alone, so this
    // kernel does not end before the one before it (the tile kernel) has.
    if (!DIRECT && blockIdx.x == gridDim.x - 1) wait_prerequisites();
}

}  // namespace attn
