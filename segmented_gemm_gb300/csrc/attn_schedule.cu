// The attention's work list, from the requests' lengths (lora_attn_schedule).
//
// A request's n query rows are cut into blocks of 2 tq tokens (two query tiles
// of 128 rows: tq tokens times the group's heads each).  A block's cost is the
// key tiles of 128 that its last token reaches, max(1, ceil(keys / 128)), once
// for every kv head.
//
// The persistent attention kernel takes units from the list in one of two ways,
// chosen here by which ends sooner:
//   whole   a unit is one (block, head), longest blocks first, taken as CTAs
//           come free: nothing is split, the end is ragged by about half of the
//           longest unit
//   cut     the tiles of all (block, head) pairs laid end to end, cut into one
//           equal piece a CTA: ends together, but a pair that spans pieces is
//           written as partial results and joined
// One CTA, one pass over the requests and two over the blocks; once a step.
#include <cuda_runtime.h>

#include "attn.h"
#include "block_scan.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace lora {

constexpr int kSchedThreads = 1024;
constexpr int kSchedBuckets = 1024;          // block costs told apart by the sort
constexpr int kMinPiece = 2;                 // key tiles of a piece, at least
constexpr int kJoinSingle = 2, kJoinPair = 6; // what joining partial results costs, in key tiles
constexpr int64_t kSectionBytes = 64 << 20;  // keys and values of the heads that run together (L2 holds 126 MB)

__global__ void __launch_bounds__(kSchedThreads) attn_schedule_kernel(const AttnSchedParams p)
{
    pdl_launch_dependents();
    extern __shared__ int32_t blk_start[];   // [R + 1] first block of each request
    __shared__ int64_t wsum[32];
    __shared__ int32_t hist[kSchedBuckets];
    __shared__ int32_t s_max, s_pair;
    const int tid = threadIdx.x;
    const int R = p.R, tb = 2 * p.tq;
    if (tid == 0) {
        s_max = 0;
        s_pair = 0;
    }
    hist[tid] = 0;
    pdl_wait();
    // a call whose waits gave up may have left counters behind
    for (int i = tid; i < ACNT_WORDS; i += kSchedThreads)
        if (i != CNT_STATUS) p.counters[i] = 0;

    // query rows and keys of request r, clamped
    int bad = 0;
    auto rows_of = [&](int r, int32_t *start) {
        const int32_t c0 = p.cu[r], c1 = p.cu[r + 1];
        const int64_t s = c0 < 0 ? 0 : c0 > p.T ? p.T : c0;
        const int64_t e = c1 < s ? s : c1 > p.T ? p.T : c1;
        bad |= (s != c0) | (e != c1);
        *start = static_cast<int32_t>(s);
        return static_cast<int32_t>(e - s);
    };
    auto keys_of = [&](int r, int32_t n) {
        const int32_t l = p.kv_len ? p.kv_len[r] : n;
        const int64_t c = l < 0 ? 0 : l > p.max_kv ? p.max_kv : l;
        bad |= c != l;
        return static_cast<int32_t>(c);
    };

    int64_t carry = 0, keys = 0;
    for (int r0 = 0; r0 < R; r0 += kSchedThreads) {
        const int r = r0 + tid;
        int64_t nb = 0;
        if (r < R) {
            int32_t start;
            const int32_t n = rows_of(r, &start);
            nb = (static_cast<int64_t>(n) + tb - 1) / tb;
            if (n > 0) keys += keys_of(r, n);
        }
        int64_t total;
        const int64_t ex = carry + block_scan_i64(nb, wsum, &total);
        if (r < R) blk_start[r] = static_cast<int32_t>(ex < p.max_blocks ? ex : p.max_blocks);
        carry += total;
    }
    // offsets that overlap could ask for more blocks than the rows have
    bad |= carry > p.max_blocks;
    const int nb = static_cast<int>(carry < p.max_blocks ? carry : p.max_blocks);
    if (tid == 0) blk_start[R] = nb;
    int64_t all_keys;
    block_scan_i64(keys, wsum, &all_keys);   // also makes blk_start visible

    carry = 0;
    int my_max = 0, my_pair = 0;
    for (int b0 = 0; b0 < nb; b0 += kSchedThreads) {
        const int b = b0 + tid;
        AttnBlock k = {};
        if (b < nb) {
            const int r = last_le(blk_start, R, b);
            int32_t start;
            const int32_t n = rows_of(r, &start), len = keys_of(r, n);
            const int32_t local = (b - blk_start[r]) * tb;
            k.req = r;
            k.tok0 = start + local;
            k.ntok = min(tb, n - local);
            k.qpos0 = len - n + local;
            k.kv_len = len;
            const int32_t seen = max(0, k.qpos0 + k.ntok);   // <= len
            k.tiles = max(1, (seen + kAttnTileK - 1) / kAttnTileK);
            my_max = max(my_max, k.tiles);
            my_pair |= k.ntok > p.tq;
            atomicAdd(&hist[kSchedBuckets - min(k.tiles, kSchedBuckets)], 1);
        }
        int64_t total;
        k.pre = carry + block_scan_i64(k.tiles, wsum, &total);
        if (b < nb) p.blocks[b] = k;
        carry += total;
    }
    if (my_max) atomicMax(&s_max, my_max);
    if (my_pair) atomicOr(&s_pair, 1);
    if (bad) atomicOr(p.counters + CNT_STATUS, LORA_DEV_BAD_LENGTH);
    __syncthreads();

    // longest blocks first (ties in any order: they are whole either way)
    {
        int64_t total;
        const int32_t h = hist[tid];
        const int64_t ex = block_scan_i64(h, wsum, &total);
        hist[tid] = static_cast<int32_t>(ex);
        __syncthreads();
        for (int b = tid; b < nb; b += kSchedThreads) {
            const int at = atomicAdd(&hist[kSchedBuckets - min(p.blocks[b].tiles, kSchedBuckets)], 1);
            p.order[at] = b;
        }
    }
    if (tid == 0) {
        const int64_t W = carry * p.kv_heads;
        AttnHdr h;
        h.nblocks = nb;
        h.tiles = W;
        // key tiles a CTA runs, on average, and what each way adds to that
        const int64_t each = (W + p.ctas - 1) / p.ctas;
        const int64_t whole = max(each + (s_max + 1) / 2, static_cast<int64_t>(s_max));
        const int64_t piece = max(each, static_cast<int64_t>(kMinPiece)) + (s_pair ? kJoinPair : kJoinSingle);
        h.cut = piece < whole;
        h.unit_tiles = max(each, static_cast<int64_t>(kMinPiece));
        h.units = static_cast<int32_t>(h.cut ? (W + h.unit_tiles - 1) / h.unit_tiles
                                             : min(static_cast<int64_t>(nb) * p.kv_heads, static_cast<int64_t>(INT32_MAX)));
        const int64_t head_bytes = max(static_cast<int64_t>(1), all_keys * p.head_dim * 4);
        h.sec_heads = static_cast<int32_t>(max(static_cast<int64_t>(1), min(static_cast<int64_t>(p.kv_heads), kSectionBytes / head_bytes)));
        *p.hdr = h;
    }
}

cudaError_t launch_attn_schedule(const AttnSchedParams &p, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kSchedThreads);
    cfg.dynamicSmemBytes = (static_cast<size_t>(p.R) + 1) * 4;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    pdl_attribute(cfg, at);
    return cudaLaunchKernelEx(&cfg, attn_schedule_kernel, p);
}

}  // namespace lora
