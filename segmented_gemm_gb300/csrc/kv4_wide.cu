// The wide requests of a step over the 4-bit cache (lora_kv4_attn): chunks of
// prompts, whose many rows share each key, so that the tensor cores bound them and
// not the cache's bytes.  Their keys are unpacked to bf16 and their values to fp16 once (exactly), and the attention over a
// bf16 cache (attn.cu) runs over that, with p in fp16 as in the kernel for the other requests: 8 chunks of 64 tokens over
// 1000 to 8000 take 113 us so and 224 by blocks of 8 columns, one of 512 over 8000 102 to 104 us (about 88 of them that
// kernel, 9 its list, 4 the plan).
#include <cuda_runtime.h>

#include "block_scan.cuh"
#include "kv4.cuh"
#include "kv4_request.cuh"
#include "kv_ops.h"
#include "internal.h"
#include "ptx.cuh"

namespace lora {

namespace {

constexpr int kPlanThreads = 512;
constexpr int kUnpackThreads = 256;
constexpr int kPageTiles = kKv4WidePage / 16;

// One CTA: which requests are wide, and where each goes.  In request order as long as there
// is room for their keys.  What the attention is given are the wide requests and, in
// between, everything else as requests without keys, whose rows it writes as zeros
// and the kernel for the other requests (after it) as they are.
__global__ void __launch_bounds__(kPlanThreads) kv4_wide_plan_kernel(const Kv4WideParams w, const Kv4AttnParams p)
{
    pdl_launch_dependents();
    __shared__ int64_t scan[32];
    const int tid = threadIdx.x;
    const int run = (p.R + kPlanThreads - 1) / kPlanThreads, r0 = min(p.R, tid * run), r1 = min(p.R, r0 + run);
    pdl_wait();
    int bad = 0;
    // pages in the low half (one more than there are for what cannot fit, so that they add up), requests in the high one
    auto need = [&](const Kv4Request &q) {
        const bool wide = static_cast<int64_t>(q.n) * p.group > kv4_wide_rows(p.head_dim) && q.keys > 0;
        const int pages = min(w.pages + 1, (q.keys - 1) / kKv4WidePage + 1);
        return wide ? (int64_t(1) << 32) + pages : int64_t(0);
    };
    int64_t sum = 0, total;
    for (int r = r0; r < r1; ++r) sum += need(kv4_request(p, r, &bad));
    int64_t at = block_scan_i64(sum, scan, &total);
    int64_t served = 0;
    for (int r = r0; r < r1; ++r) {
        const Kv4Request q = kv4_request(p, r, &bad);
        const int64_t n = need(q);
        const int pages = static_cast<int>(n), first = static_cast<int>(at & 0xFFFFFFFF), i = static_cast<int>(at >> 32);
        const bool wide = n != 0 && static_cast<int64_t>(first) + pages <= w.pages && i < w.max_wide;
        w.wide[r] = wide;
        if (wide) {
            served += n;
            w.cu[2 * i + 1] = q.tok0;
            w.cu[2 * i + 2] = q.tok0 + q.n;
            w.kv_len[2 * i] = 0;
            w.kv_len[2 * i + 1] = q.keys;
            for (int j = 0; j < pages; ++j) {   // what the unpacking takes, and what the attention sees
                w.pages_of[first + j] = make_int4(r, j, q.keys, 0);
                w.table[(2 * i + 1) * static_cast<int64_t>(w.pages) + j] = first + j;
            }
        }
        at += n;
    }
    // the served ones are the first: n and the pages of all of them
    block_scan_i64(served, scan, &total);
    const int count = static_cast<int>(total >> 32);
    // rows of no request, in front and behind, stay out
    const int begin = max(0, min(p.cu[0], p.T)), end = max(begin, min(p.cu[p.R], p.T));
    if (tid == 0) {
        w.cu[0] = begin;
        w.kv_len[2 * count] = 0;
        *w.used = static_cast<int>(total & 0xFFFFFFFF);
    }
    for (int i = 2 * count + 1 + tid; i <= 2 * w.max_wide + 1; i += kPlanThreads) {
        w.cu[i] = end;
        if (i <= 2 * w.max_wide) w.kv_len[i] = 0;
    }
}

// A warp a tile, as a lane takes it in the attention.  Memory bounds it: 8512 tokens of 8 heads of 128 are 45 MB.
// It runs beside the attention's list of work (one CTA, 9 us), the launch ahead of it, which lets others start only when
// the plan is done: so it takes the plan's results at once and waits for the list at its end.
template <int DP>
__global__ void __launch_bounds__(kUnpackThreads) kv4_unpack_kernel(const Kv4WideParams w, const Kv4AttnParams p)
{
    pdl_launch_dependents();
    using Tile = Kv4Tile<DP>;
    constexpr int W = DP / 32;
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int in_page = p.page_shift - 4;
    const bool sectors = p.head_dim % 16 == 0;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kUnpackThreads / 32);
    const int per_page = kPageTiles * p.kv_heads;
    const int64_t tiles = static_cast<int64_t>(__ldcg(w.used)) * per_page;
    for (int64_t u = (static_cast<int64_t>(blockIdx.x) * kUnpackThreads + threadIdx.x) >> 5; u < tiles; u += warps) {
        const int page = static_cast<int>(u / per_page), rest = static_cast<int>(u - static_cast<int64_t>(page) * per_page);
        const int h = rest / kPageTiles, in = rest % kPageTiles;
        const int4 whose = __ldcg(w.pages_of + page);   // request, page of the request, its keys
        const int t = whose.y * kPageTiles + in;
        if (t * 16 >= whose.z) continue;
        const int from = p.table[whose.x * p.table_stride + (t >> in_page)];
        const uint8_t *tile = p.zeros;
        if (from >= 0 && from < p.num_pages)
            tile = p.data + from * p.page_stride + h * p.head_stride + (t & ((1 << in_page) - 1)) * static_cast<int64_t>(Tile::kBytes);
        else if (lane == 0)
            atomicOr(p.counters, LORA_DEV_BAD_PAGE);
        uint32_t k[2][W], v[2][W], ks[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint8_t *at = tile + e * (4 * DP) + lane * (4 * W);
            if (W == 4) {
                *reinterpret_cast<uint4 *>(k[e]) = *reinterpret_cast<const uint4 *>(at);
                *reinterpret_cast<uint4 *>(v[e]) = *reinterpret_cast<const uint4 *>(at + Tile::kValues);
            } else {
                *reinterpret_cast<uint2 *>(k[e]) = *reinterpret_cast<const uint2 *>(at);
                *reinterpret_cast<uint2 *>(v[e]) = *reinterpret_cast<const uint2 *>(at + Tile::kValues);
            }
            at = tile + Tile::kKeyScales + (8 * e + g) * Tile::kGroups + c * (W / 2);
            ks[e] = W == 4 ? *reinterpret_cast<const uint16_t *>(at) : *at;
        }
        const uint32_t vs = *reinterpret_cast<const uint32_t *>(tile + Tile::kValueScales + ((DP == 128 ? g : g / 2) * 4 + c) * 4);
        const int64_t row = ((static_cast<int64_t>(page) * p.kv_heads + h) * kKv4WidePage + in * 16) * p.head_dim;
#pragma unroll
        for (int e = 0; e < 2; ++e) {   // keys g and g + 8, elements from c * DP / 4 on: a scale for two words
            uint16_t *to = w.k + row + (8 * e + g) * p.head_dim + c * (DP / 4);
#pragma unroll
            for (int j = 0; j < W; j += 2) {
                const int d = c * (DP / 4) + 8 * j;
                const uint32_t scale = ks[e] >> (4 * j) & 0xFF;
                const uint4 lo = kv4_values(k[e][j], scale), hi = kv4_values(k[e][j + 1], scale);
                if (sectors) {
                    if (d < p.head_dim) store32(to + 8 * j, lo, hi);
                } else {
                    if (d < p.head_dim) *reinterpret_cast<uint4 *>(to + 8 * j) = lo;
                    if (d + 8 < p.head_dim) *reinterpret_cast<uint4 *>(to + 8 * j + 8) = hi;
                }
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)     // keys 2c, 2c + 1 and 8 more, elements from g * DP / 8 on
#pragma unroll
            for (int o = 0; o < 2; ++o) {
                const int d = g * (DP / 8);
                const uint32_t scale = vs >> (8 * (2 * e + o)) & 0xFF;
                uint16_t *to = w.v + row + (8 * e + 2 * c + o) * p.head_dim + d;
                const uint4 lo = kv4_values_f16(v[e][o], scale);
                if (DP == 64) {
                    if (d < p.head_dim) *reinterpret_cast<uint4 *>(to) = lo;
                    continue;
                }
                const uint4 hi = kv4_values_f16(v[e][DP == 64 ? o : o + 2], scale);
                if (sectors) {
                    if (d < p.head_dim) store32(to, lo, hi);
                } else {
                    if (d < p.head_dim) *reinterpret_cast<uint4 *>(to) = lo;
                    if (d + 8 < p.head_dim) *reinterpret_cast<uint4 *>(to + 8) = hi;
                }
            }
    }
    pdl_wait();   // the list: the attention waits for this kernel alone
}

}  // namespace

cudaError_t launch_kv4_wide_plan(const Kv4WideParams &w, const Kv4AttnParams &p, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    pdl_attribute(cfg, at);
    return cudaLaunchKernelEx(&cfg, kv4_wide_plan_kernel, w, p);
}

cudaError_t launch_kv4_unpack(const Kv4WideParams &w, const Kv4AttnParams &p, cudaStream_t stream)
{
    const int64_t most = static_cast<int64_t>(w.pages) * kPageTiles * p.kv_heads / (kUnpackThreads / 32) + 1;
    const int64_t cap = 8ll * num_sms_current_device();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(most < cap ? most : cap));
    cfg.blockDim = dim3(kUnpackThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    pdl_attribute(cfg, at);
    return cudaLaunchKernelEx(&cfg, p.head_dim <= 64 ? kv4_unpack_kernel<64> : kv4_unpack_kernel<128>, w, p);
}

}  // namespace lora
