// Plans of the paged attention and the join of its partial results.
//
//     lse = log2 sum_p 2^lse_p,   O = sum_p 2^(lse_p - lse) O_p
//
// over the parts of a row (ranges of the shared prefix and of the sequence's
// own tokens), in the order of the parts: the result does not depend on which
// CTA finished first.
#include <cuda_bf16.h>

#include <algorithm>

#include "paged.cuh"
#include "sm103_ptx.cuh"

namespace attn {

PagedPlan paged_plan(int B, int Nq, int H, int H_kv, int d, int prefix_len, int max_pages, int page_size) {
    PagedPlan plan;
    const long long rows = static_cast<long long>(Nq) * (H / H_kv);
    const auto up = [](long long a, long long b) { return (a + b - 1) / b; };
    // About four waves of two CTAs an SM, in ranges of kOwnChunk keys or more.
    const long long target = 8LL * kPlanSms;
    const long long own = static_cast<long long>(max_pages) * page_size;
    const long long own_units = B * static_cast<long long>(H_kv) * up(rows, 16);
    plan.own_parts = static_cast<int>(std::max(1LL, std::min({up(own, kOwnChunk), up(target, own_units), 128LL})));
    if (prefix_len > 0) {
        const long long units = static_cast<long long>(H_kv) * up(B * rows, 16);
        plan.prefix_parts = static_cast<int>(std::max(1LL, std::min({up(prefix_len, kOwnChunk), up(target, units), 128LL})));
    }
    const int parts = plan.prefix_parts + plan.own_parts;
    plan.direct = parts == 1;
    if (!plan.direct) {
        const size_t r = static_cast<size_t>(parts) * B * Nq * H;
        plan.part_o_bytes = (r * d * 4 + 255) / 256 * 256;
        plan.bytes = plan.part_o_bytes + (r * 4 + 255) / 256 * 256;
    }
    return plan;
}

namespace {

// One warp per row; D / 32 columns a lane.
template <int D>
__global__ void __launch_bounds__(128) paged_merge_kernel(const PagedParams p) {
    constexpr int V = D / 32;
    const long long rows = static_cast<long long>(p.B) * p.Nq * p.H;
    const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= rows) return;
    const int parts = p.prefix_parts + p.own_parts;
    float mm = -INFINITY;
    for (int x = lane; x < parts; x += 32) mm = fmaxf(mm, p.part_lse[x * rows + row]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
    const float ref = mm == -INFINITY ? 0.0f : mm;
    float sum = 0.0f, acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.0f;
    for (int x = 0; x < parts; ++x) {
        const float l2 = p.part_lse[x * rows + row];
        if (l2 == -INFINITY) continue;                 // an empty part: its O was not written
        const float w = ex2_approx(l2 - ref);
        sum += w;
        const float* src = p.part_o + (x * rows + row) * D + lane * V;
        if constexpr (V == 2) {
            const float2 f = *reinterpret_cast<const float2*>(src);
            acc[0] += w * f.x;
            acc[1] += w * f.y;
        } else {
#pragma unroll
            for (int v = 0; v < V; v += 4) {
                const float4 f = *reinterpret_cast<const float4*>(src + v);
                acc[v] += w * f.x;
                acc[v + 1] += w * f.y;
                acc[v + 2] += w * f.z;
                acc[v + 3] += w * f.w;
            }
        }
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.o) + row * D + lane * V);
#pragma unroll
    for (int v = 0; v < V; v += 2) dst[v / 2] = pack_bf16x2(acc[v] * inv, acc[v + 1] * inv);
    if (lane == 0) {
        const int h = static_cast<int>(row % p.H);
        const long long bi = row / p.H;
        const int i = static_cast<int>(bi % p.Nq), b = static_cast<int>(bi / p.Nq);
        p.lse[(static_cast<long long>(b) * p.H + h) * p.Nq + i] =
            sum == 0.0f ? -INFINITY : (ref + __log2f(sum)) * 0.69314718055994530942f;
    }
}

}  // namespace

cudaError_t run_paged_merge(const PagedParams& p, cudaStream_t stream) {
    const long long rows = static_cast<long long>(p.B) * p.Nq * p.H;
    const unsigned grid = static_cast<unsigned>((rows + 3) / 4);
    if (p.d == 64) paged_merge_kernel<64><<<grid, 128, 0, stream>>>(p);
    else if (p.d == 128) paged_merge_kernel<128><<<grid, 128, 0, stream>>>(p);
    else paged_merge_kernel<256><<<grid, 128, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace attn
