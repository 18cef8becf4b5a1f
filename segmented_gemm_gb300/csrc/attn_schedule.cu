// The attention's work list, from the requests' lengths (lora_attn_schedule).
//
// A request's n query rows are cut into blocks of 2 tq tokens (two query tiles
// of 128 rows: tq tokens times the group's heads each).  A group is a block and
// a kv head; it costs the key tiles of 128 that the block's last token reaches,
// and kAttnItemCost more for starting and ending it.
//
// The persistent attention kernel takes units from the list in one of two ways,
// chosen here by which ends sooner:
//   whole   a unit is one group, longest first, taken as CTAs come free: nothing
//           is split, the end is ragged by about a third of the units that run last
//   cut     all groups laid end to end and cut into one equal piece a CTA: they
//           end together, but a group that spans pieces is written as partial
//           results and joined
// One token over 1000 takes 8.9 us cut and 12.3 whole, 32 requests of one token over up
// to 8000 98 and 121; a 16384-token prompt 1409 cut and 1347 whole (1 head of 128: 78 and
// 177), one of 2048 tokens 56 and 30 (1 head: 72 and 27).
// Whole groups run by sections of heads whose keys and values L2 holds together (a
// 65536-token prompt of 8 kv heads: 21.1 ms, 22.4 with all heads at once).
// One CTA, once a step.
#include <cuda_runtime.h>

#include "attn.h"
#include "attn_piece.cuh"
#include "block_scan.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace lora {

constexpr int kSchedThreads = 1024;
constexpr int kSchedBuckets = 1024;          // block costs told apart by the sort
constexpr int kMinPiece = 2;                 // key tiles of a piece, at least (one token over 1000: 8.9 us, 9.2 with 1, 10.8 with 4)
// What cutting costs, in a cut list's units.  A fixed part for writing and counting
// partial results, less where their few rows are joined in place and CTAs are to spare.
// And the join, which reads every piece's rows, one piece after another: kJoinElems
// elements in the time of a unit.  256 tokens of one head over 4096, 36 pieces of 256 rows
// of 128, take 126 us cut and 54 whole, one prompt of 2048 72 and 27; a fixed part alone (2
// and 16) had both cut.  Both lists of 855 steps were timed, prompts, chunks, single tokens
// and mixtures, heads 40 to 1 over 1 to 8, dimensions 64 to 128: this rule's choice takes
// 0.3 % longer than the better list on average and 21 % at most, the fixed part alone 8 %
// and 180 %.
constexpr int kCutFew = 4, kCutSingle = 6, kCutPair = 24;
constexpr int kFewElems = 1024;
constexpr float kJoinElems = 8192.f;
constexpr int64_t kSectionBytes = 64 << 20;  // keys and values of the heads that run together (L2 holds 126 MB)

__global__ void __launch_bounds__(kSchedThreads) attn_schedule_kernel(const AttnSchedParams p)
{
    extern __shared__ int32_t blk_start[];   // [R + 1] first block of each request
    __shared__ int64_t wsum[32];
    __shared__ int32_t hist[kSchedBuckets];
    __shared__ int32_t unit_blk[kAttnMaxCtas];
    __shared__ int32_t s_max, s_tail, s_ntok, s_join;
    __shared__ unsigned long long s_shares;
    const int tid = threadIdx.x;
    const int R = p.R, tb = 2 * p.tq;
    if (tid == 0) {
        s_max = 0;
        s_tail = 1;
        s_ntok = 0;
        s_join = 0;
        s_shares = 0;
    }
    hist[tid] = 0;
    pdl_wait();
    pdl_launch_dependents();   // not before: a kernel behind this one may count on what lies ahead of it (kv4_wide.cu)
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

    // block b: two query tiles at most, and what its last row reaches
    auto block_of = [&](int b) {
        AttnBlock k = {};
        const int r = last_le(blk_start, R, b);
        int32_t start;
        const int32_t n = rows_of(r, &start), len = keys_of(r, n);
        const int32_t local = (b - blk_start[r]) * tb;
        k.base = p.kv_len ? r : start;   // (not tok0 - qpos0: a clamped prompt's differs)
        k.tok0 = start + local;
        k.ntok = min(tb, n - local);
        k.qpos0 = len - n + local;
        k.kv_len = len;
        const int32_t seen = max(0, k.qpos0 + k.ntok);   // <= len
        k.tiles = max(1, (seen + kAttnTileK - 1) / kAttnTileK);
        return k;
    };
    auto bucket = [](int tiles) { return kSchedBuckets - min(tiles, kSchedBuckets); };
    int64_t tiles = 0, shares = 0;   // shares: in a list with pairs
    int my_max = 0, my_ntok = 0, my_join = 0;   // my_join: most tokens times share
    for (int b = tid; b < nb; b += kSchedThreads) {
        const AttnBlock k = block_of(b);
        tiles += k.tiles;
        const int32_t share = attn_share(k.tiles, k.ntok > p.tq, 2);
        shares += share;
        my_join = max(my_join, static_cast<int>(min(static_cast<int64_t>(share) * k.ntok, static_cast<int64_t>(INT32_MAX))));
        my_max = max(my_max, k.tiles);
        my_ntok = max(my_ntok, k.ntok);
        atomicAdd(&hist[bucket(k.tiles)], 1);
    }
    if (my_max) atomicMax(&s_max, my_max);
    if (my_ntok) {
        atomicMax(&s_ntok, my_ntok);
        atomicMax(&s_join, my_join);
    }
    if (bad) atomicOr(p.counters + CNT_STATUS, LORA_DEV_BAD_LENGTH);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) shares += __shfl_xor_sync(0xffffffffu, shares, d);
    if ((tid & 31) == 0 && shares) atomicAdd(&s_shares, static_cast<unsigned long long>(shares));
    int64_t all_tiles, total;
    block_scan_i64(tiles, wsum, &all_tiles);   // also makes hist and the shared maxima and sums visible
    const int32_t here = hist[tid];
    const int32_t before = static_cast<int32_t>(block_scan_i64(here, wsum, &total));
    hist[tid] = before;   // first place of each cost in the longest-first order
    // the cost of the units that run last when whole: those that start when about
    // every CTA has one left
    const int last = max(0, nb - (p.ctas + p.kv_heads - 1) / p.kv_heads);
    if (here > 0 && before <= last && last < before + here) s_tail = kSchedBuckets - tid;
    __syncthreads();

    const int64_t groups = static_cast<int64_t>(nb) * p.kv_heads;
    const bool pairs = s_ntok > p.tq;
    const int weight = pairs ? 2 : 1;
    const int64_t cost = (pairs ? static_cast<int64_t>(s_shares) : all_tiles + static_cast<int64_t>(nb) * kAttnItemCost) * p.kv_heads;
    const int64_t even = (cost + p.ctas - 1) / p.ctas;
    const int64_t each = max((even + weight - 1) & -static_cast<int64_t>(weight), static_cast<int64_t>(kMinPiece));
    const int64_t whole = weight * max(groups >= p.ctas ? each / weight + s_tail * 3 / 8 : 0, static_cast<int64_t>(s_max + kAttnItemCost));
    // a group's rows are joined as often as it has pieces, share / each and a first
    const int elems = p.group * p.head_dim;   // of a token
    const int fixed = pairs ? kCutPair : each == kMinPiece && s_ntok * elems <= kFewElems ? kCutFew : kCutSingle;
    const float n = static_cast<float>(each), join = (static_cast<float>(s_join) + s_ntok * n) * elems;   // times n
    // (a list too long for 32-bit positions is never short of units)
    const bool cut = join < static_cast<float>(whole - each - fixed) * n * kJoinElems && cost + each < INT32_MAX;
    AttnHdr h = {};
    h.stamp = p.stamp;
    h.nblocks = nb;
    h.cut = cut ? weight : 0;
    h.cost = cut ? static_cast<int32_t>(cost) : 0;
    // whole groups of few rows: two heads at once, a stream each, while that leaves a few for every CTA
    const int two = !cut && p.two && s_ntok * p.group <= kAttnFewRows && groups >= 4 * p.ctas;
    h.unit_cost = cut ? static_cast<int32_t>(each) : two;
    h.units = static_cast<int32_t>(cut ? (cost + each - 1) / each : min(groups >> two, static_cast<int64_t>(INT32_MAX)));
    const int64_t head_bytes = max(static_cast<int64_t>(1), all_keys * p.head_dim * 4);
    h.sec_heads = static_cast<int32_t>(
        max(static_cast<int64_t>(1), min(static_cast<int64_t>(p.kv_heads >> two), kSectionBytes / (head_bytes << two))));
    if (tid == 0) *p.hdr = h;
    // the blocks in their order, and (cut) the block that each unit starts in
    if (!cut) {
        // ties in any order: the results do not depend on it
        for (int b = tid; b < nb; b += kSchedThreads) {
            const AttnBlock k = block_of(b);
            p.blocks[atomicAdd(&hist[bucket(k.tiles)], 1)] = k;
        }
    } else {
        carry = 0;
        for (int b0 = 0; b0 < nb; b0 += kSchedThreads) {
            const int b = b0 + tid;
            AttnBlock k = {};
            if (b < nb) k = block_of(b);
            const int32_t own = b < nb ? attn_share(k.tiles, k.ntok > p.tq, weight) : 0;
            k.pre = static_cast<int32_t>(carry + block_scan_i64(own, wsum, &total));
            if (b < nb) {
                p.blocks[b] = k;
                const int64_t from = static_cast<int64_t>(k.pre) * p.kv_heads, to = from + static_cast<int64_t>(own) * p.kv_heads;
                for (int64_t u = (from + each - 1) / each; u * each < to && u < h.units; ++u) unit_blk[u] = b;
            }
            carry += total;
        }
    }
    __syncthreads();
    // each CTA's first piece, so that it need not look for it
    if (tid < p.ctas) {
        AttnItem w = {};
        if (tid < h.units) {
            int blk, kvh;
            if (!cut) {
                whole_unit(h, p.kv_heads, tid, &blk, &kvh);
                w = item_of(p.blocks[blk], blk, kvh, p.tq);
                w.valid += two;
            } else {
                blk = unit_blk[tid];
                const AttnBlock b = p.blocks[blk];
                int pos = tid * h.unit_cost;
                kvh = (pos - b.pre * p.kv_heads) / attn_share(b.tiles, b.ntok > p.tq, weight);
                w = cut_piece(h, b, blk, kvh, p.kv_heads, p.tq, tid, min(pos + h.unit_cost, h.cost), &pos);
            }
        }
        p.first[tid] = w;
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
