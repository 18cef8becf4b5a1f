// Attention over packed rows or a paged cache (include/lora_attn.h):
//   o_i = sum_j p_ij v_j / l_i,   p_ij = 2^(c q_i.k_j - c m_i),   l_i = sum_j p_ij,   c = scale log2(e)
// over the keys j that row i sees, m_i a reference score of the row.
//
// A query tile is 128 rows: tq tokens times the group's query heads, which
// share the key/value head, so a key tile is loaded once for the group.  A
// CTA works on two score streams at once, so that one's softmax runs under the
// other's matrix products:
//   pair     two query tiles against the same key tiles (long chunks, prompts)
//   single   one query tile, the key tiles dealt to the streams in turn
//            (decode and short chunks, where the cache's bytes bound the call)
//   two      single tokens (or a few) of large batches: two kv heads of a request, a
//            stream each, so that contexts of a tile or two keep both busy
// Per stream and key tile of 128 keys, all on the tensor cores:
//   S = Q K^T   both from shared memory, S [128 x 128] fp32 in tensor memory
//   softmax     a thread per row: S to registers, p = 2^(..), P as bf16 back
//               over S's cells (half of them)
//   O += P V    P from tensor memory, V from shared memory as it was loaded
//               (its head dimension contiguous: an N-major operand)
// With up to 16 rows (a decoded token, or a few) a thread per row would leave all
// but a few lanes idle over 128 keys each: there the four lanes of a quad share
// a row (tensor memory loads of 16 lanes x 256 bits), 32 keys each: one token over
// 1000 takes 8.9 us so and 11.3 by a thread per row, 32 requests of one token over up
// to 8000 97 and 103.
// O stays in tensor memory.  Any m_i near the scores is as good as their maximum: p, l
// and O are floating point (bf16 has fp32's range), so a larger p costs no precision,
// and the division by l_i takes m_i out again.  It costs range: over all keys p may sum
// to 2^66 (2^25 half tiles of 2^40, twice that where quads share rows), so O is finite for
// |v| up to 2^60.  So m_i is the first score that the row
// sees, and its own p = 1 keeps l_i from vanishing; it moves, to the maximum of the
// half tile, only when half a tile's p sum to more than 2^40, and the softmax threads
// rescale O then.  Otherwise no maximum is computed (with the first half tile's
// maximum to start from, a prompt of 77 tokens took 8.9 us instead of 8.2).
//
// Roles (384 threads): warps 0..3 and 4..7 the softmax and the results of
// stream 0 and 1; warp 8 takes the work and loads keys, 11 loads queries and
// values (TMA); 9 and 10 issue the matrix products of stream 0 and 1.
// Shared memory: two query tiles and a ring of key and value tiles.
// Persistent, one CTA per SM; work comes from the schedule (attn_schedule.cu).
// A group (block, kv head) cut into pieces leaves partial (O, m, l) in the
// workspace; the piece that finishes last joins them in their order, so
// results do not depend on timing.  Every wait is bounded.
//
// What bounds it, and what it measured (32 query and 8 kv heads of 128 unless said;
// peaks: a 6690 GB/s copy, 1867 TFLOP/s bf16):
//   decode        the cache's bytes.  128 requests of 1000 to 16000 tokens, 4.14 GB:
//                 608 to 621 us, 6.7 to 6.8 TB/s; 32 requests of up to 8000, 579 MB:
//                 97 to 98 us, 5.9 to 6.0 TB/s (the start, 4 us, and the last pieces' join show)
//   long prompts  16384 tokens, 2.2 TFLOP: 1260 to 1310 us (1.68 to 1.74 PFLOP/s, the
//                 tensor cores busy for 76 % of the cycles), 1320 to 1400 back to back,
//                 where the power cap bounds it (a plain product then has 1710 TFLOP/s)
//   head dim 64   the softmax threads: the products take half as long for the same
//                 exponentials.  Chunks of up to 700 over 9000 tokens, 94 GFLOP: 132 us,
//                 the special function units busy for 33 % of it and each warp
//                 waiting mostly on its own chain of loads, exponentials and stores
//   single calls  latency: one token over 1000 8.9 us, a prompt of 77 8.2 us
#include <cuda_runtime.h>

#include "attn.h"
#include "attn_piece.cuh"
#include "attn_ptx.cuh"
#include "internal.h"

namespace lora {

constexpr int kAttnThreads = 384;
constexpr int kItems = 4;             // work items in flight between the loader and the others
constexpr float kMostP = 0x1p40f;     // half a tile whose p sum to more than this moves m_i
// Values of a 4-bit cache (kv4_wide.cu; kF16): fp16 has them exactly, and p with three bits more than bf16: the outputs are 0.0017
// of their norm off fp64, 0.0023 with p in bf16.  What it lacks is bf16's range: p is 2^kLiftF16 where the score is m_i, at most
// kMostPF16, and has all its bits down to 2^-21, some to 2^-31, of what it is at m_i (kv4_attn.cu has the same
// range).  So that m_i need not move soon it starts as the largest of eight scores: chunks of up to 700 over 9000
// take 152 us so, 154 with the first one, 157 with the largest of 64; 150 with p in bf16.
constexpr float kMostPF16 = 65504.f, kLiftF16 = 7.f;

// tensor memory columns (512 in all): S of stream s at s * 128, O at 256 + s * DP.
// With a head dimension of 128 that is all of them, and P lies over S's first 64:
// the next scores wait for its product.  With 64 there is room for P of its own,
// and they only wait until S has been read: softmax and products overlap within a
// stream.
constexpr uint32_t kColS = 128, kColO = 256, kColP = 384;

template <int DP>
struct AttnSmem {
    static constexpr int kHalves = DP / 64;                    // 128-byte column blocks of a tile
    static constexpr int kTile = 128 * DP * 2;                 // bytes of a query, key or value tile
    static constexpr int kStages = 5 * 128 / DP + (DP == 64 ? 2 : 0);
    static constexpr int kStats = 2 * kTile + kStages * kTile; // offsets
    static constexpr int kItem = kStats + 128 * 8;
    static constexpr int kBars = kItem + kItems * static_cast<int>(sizeof(AttnItem));
    static constexpr bool kOwnP = DP == 64;                    // P does not share S's cells
    static constexpr int kNumBars = 2 * kStages + 2 * kItems + 2 + 1 + 2 + 2 + 2 + 2 + 2 + 2 + 2 + 2;
    static constexpr int kEnd = kBars + kNumBars * 8 + 4 * (3 + kStages + 2);
    static constexpr int kBytes = kEnd + 1024;                 // room to align the base
    static_assert(kBytes <= 232448, "fits the opt-in shared memory of a CTA");
};

// 32 bytes of the lane's own row; dst a multiple of 32.
__device__ __forceinline__ void store32(uint8_t *dst, const uint32_t *v)
{
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
                 "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// A piece's 2 n loads, in the order in which the products need them:
//   pair    K0 V0 K1 V1 ...
//   single  K0 K1 V0 K2 V1 K3 ... V(n-2) V(n-1)   (n = 1: K0 V0)
__device__ __forceinline__ uint32_t load_of_key(int pair, int t) { return pair ? 2 * t : t < 2 ? t : 2 * t - 1; }
__device__ __forceinline__ uint32_t load_of_value(int pair, int t, int n) { return pair ? 2 * t + 1 : min(2 * t + 2, n + t); }

// The work list of a few prompts, made by the warp that uses it: at most 32
// requests, one a lane, and no more groups than two a CTA.  Whole groups, the last
// blocks of the last request first: a prompt's own longest first, but unequal prompts
// in the order they came (20 of 300 to 500 tokens of 8 heads on 1: 19.8 us; 15.9 by a
// list that exists already).  Where it is used, and what it saves: makes_own_list.
struct ShortList {
    int start, rows, first, nb;   // the lane's request: its rows, its first block; all blocks
    __device__ __forceinline__ void load(const AttnParams &p, int lane)
    {
        start = rows = 0;
        if (lane < p.requests) {
            start = p.cu[lane];
            rows = p.cu[lane + 1];   // the end, until header() has seen it
        }
    }
    __device__ __forceinline__ AttnHdr header(const AttnParams &p, int32_t *status, int lane)
    {
        if (lane < p.requests) {
            const int32_t c0 = start, c1 = rows, T = static_cast<int32_t>(p.T);
            start = max(0, min(c0, T));
            const int e = max(start, min(c1, T));
            rows = e - start;
            if (start != c0 || e != c1) atomicOr(status, LORA_DEV_BAD_LENGTH);
        }
        const int mine = (rows + 2 * p.tq - 1) / (2 * p.tq);
        first = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, first, d);
            if (lane >= d) first += y;
        }
        // offsets that overlap could ask for more blocks than the rows have
        nb = static_cast<int>(min(static_cast<int64_t>(__shfl_sync(0xffffffffu, first, 31)), p.max_blocks));
        first -= mine;
        AttnHdr h = {};
        h.nblocks = nb;
        h.units = nb * p.kv_heads;
        h.sec_heads = p.kv_heads;
        return h;
    }
    // block i, from the last one (the longest of its request) on
    __device__ __forceinline__ AttnBlock block(const AttnParams &p, int i)
    {
        i = nb - 1 - i;
        const int r = 31 - __clz(__ballot_sync(0xffffffffu, first <= i && rows > 0));
        const int n = __shfl_sync(0xffffffffu, rows, r);
        const int local = (i - __shfl_sync(0xffffffffu, first, r)) * 2 * p.tq;
        AttnBlock b = {};
        b.base = __shfl_sync(0xffffffffu, start, r);
        b.tok0 = b.base + local;
        b.ntok = min(2 * p.tq, n - local);
        b.qpos0 = local;
        b.kv_len = n;
        b.tiles = (local + b.ntok + kAttnTileK - 1) / kAttnTileK;
        return b;
    }
};

struct AttnMaps {
    CUtensorMap q, k, v;
};

// mbar_wait with a 32-bit clock and without the status bit (set once, at the
// end): it stands in the kernel many times.
__device__ __forceinline__ bool attn_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag, uint32_t limit)
{
    if (mbar_try_wait(bar, parity)) return true;
    const uint32_t t0 = static_cast<uint32_t>(clock());
    while (!mbar_try_wait(bar, parity)) {
        const uint32_t most = *abort_flag ? min(limit, static_cast<uint32_t>(kWaitShort)) : limit;
        if (static_cast<uint32_t>(clock()) - t0 > most) {
            *abort_flag = 1;
            return false;
        }
    }
    return true;
}

// The same with its loop out of line, for the roles that only issue work.  What
// they run per piece and the softmax do not fit the instruction cache together, so code
// that only waits is kept out of it: 12 prompts of 500 to 700 tokens take 59.5 us
// instead of 62.5, chunks of up to 700 over 9000 133 instead of 135.
__device__ __noinline__ bool attn_wait_loop(uint32_t bar, uint32_t parity, volatile int *abort_flag, uint32_t limit)
{
    return attn_wait(bar, parity, abort_flag, limit);
}
__device__ __forceinline__ bool attn_wait_far(uint32_t bar, uint32_t parity, volatile int *abort_flag, uint32_t limit)
{
    return mbar_try_wait(bar, parity) || attn_wait_loop(bar, parity, abort_flag, limit);
}

// Bounded wait until *count > n (shared memory; what it counts is ordered by the
// barrier that is waited on next).
__device__ __noinline__ bool attn_wait_count_loop(const int *count, int n, volatile int *abort_flag, uint32_t limit)
{
    const uint32_t t0 = static_cast<uint32_t>(clock());
    while (ld_volatile_shared(count) <= n) {
        const uint32_t most = *abort_flag ? min(limit, static_cast<uint32_t>(kWaitShort)) : limit;
        if (static_cast<uint32_t>(clock()) - t0 > most) {
            *abort_flag = 1;
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool attn_wait_count(const int *count, int n, volatile int *abort_flag, uint32_t limit)
{
    return ld_volatile_shared(count) > n || attn_wait_count_loop(count, n, abort_flag, limit);
}

// log2 of a sum of p, as if p were 1 where the score is m_i
template <bool kF16>
__device__ __forceinline__ float log2_sum(float l)
{
    return kF16 ? log2f(l) - kLiftF16 : log2f(l);
}

// First row of the partial results of a group's piece k, of the group that starts in
// unit unit0: the last piece of that unit, then the first of the units after it.
__device__ __forceinline__ int64_t join_slot(const AttnParams &p, int unit0, int k)
{
    return static_cast<int64_t>(k == 0 ? 2 * unit0 + 1 : 2 * (unit0 + k)) * p.part_rows;
}

// The pieces of a group, joined by the 256 softmax threads in the pieces' order:
//   m = max m_k,  l = sum l_k 2^(c (m_k - m)),  o = sum O_k 2^(c (m_k - m)) / l.
// Latency bounds it (a piece's rows lie in L2), so a thread has four elements of a
// piece in flight: with one, chunks of up to 700 tokens over 9000 cached took 148 us
// instead of 141, up to five new tokens a request 61.4 instead of 59.3.  A function of
// its own: inlined it costs the softmax loop registers.  A few rows (at most one
// element a thread, often of many pieces) are joined where it is called instead, with
// four pieces in flight: one decoded token takes 9.0 us so, 10.6 through this function.
template <bool kF16>
__device__ __noinline__ void join_pieces(const AttnParams &p, int ntok, int tok0, int kvh, int parts, int unit0, float c)
{
    const int G = p.group, D = p.head_dim, rows = ntok * G, d4 = D / 4;
    constexpr int kJoin = 4;   // elements of four columns at once
    const int all = rows * d4;
#pragma unroll 1
    for (int u0 = threadIdx.x; u0 < all; u0 += 256 * kJoin) {
        float mm[kJoin], ll[kJoin], a[kJoin][4];
        int64_t at[kJoin];   // my elements' rows of a slot, and their columns
        int col[kJoin];
#pragma unroll
        for (int j = 0; j < kJoin; ++j) {
            const int u = min(u0 + 256 * j, all - 1), rr = u / d4;
            at[j] = rr;
            col[j] = (u - rr * d4) * 4;
            mm[j] = -INFINITY;
            ll[j] = a[j][0] = a[j][1] = a[j][2] = a[j][3] = 0.f;
        }
#pragma unroll 1
        for (int k = 0; k < parts; ++k) {
            const int64_t slot = join_slot(p, unit0, k);
            float2 ml[kJoin];
            float4 v[kJoin];
#pragma unroll
            for (int j = 0; j < kJoin; ++j) {
                ml[j] = __ldcg(p.part_ml + slot + at[j]);
                v[j] = __ldcg(reinterpret_cast<const float4 *>(p.part + (slot + at[j]) * D + col[j]));
            }
#pragma unroll
            for (int j = 0; j < kJoin; ++j) {
                const float mn = fmaxf(mm[j], ml[j].x);
                const float f = ml[j].y == 0.f ? 0.f : ex2((ml[j].x - mn) * c);
                const float g = ll[j] == 0.f ? 0.f : ex2((mm[j] - mn) * c);
                mm[j] = mn;
                ll[j] = ll[j] * g + f * ml[j].y;
                a[j][0] = a[j][0] * g + f * v[j].x;
                a[j][1] = a[j][1] * g + f * v[j].y;
                a[j][2] = a[j][2] * g + f * v[j].z;
                a[j][3] = a[j][3] * g + f * v[j].w;
            }
        }
#pragma unroll
        for (int j = 0; j < kJoin; ++j) {
            if (u0 + 256 * j >= all) continue;
            const float inv = ll[j] == 0.f ? 0.f : 1.f / ll[j];
            const int rr = static_cast<int>(at[j]), tk = rr / G, hd = kvh * G + (rr - tk * G);
            const int64_t row = static_cast<int64_t>(tok0) + tk;
            *reinterpret_cast<uint2 *>(p.o + row * p.o_tok + hd * p.o_head + col[j]) =
                make_uint2(pack_bf16x2(a[j][0] * inv, a[j][1] * inv), pack_bf16x2(a[j][2] * inv, a[j][3] * inv));
            if (p.lse && col[j] == 0)
                p.lse[row * p.heads + hd] = ll[j] == 0.f ? -INFINITY : (mm[j] * c + log2_sum<kF16>(ll[j])) * 0.6931471805599453f;
        }
    }
}

// kTwo: lists whose units are two heads of few rows are run too.  kF16: p and the values are fp16
template <int DP, bool kPaged, bool kTwo, bool kF16>
__global__ void __launch_bounds__(kAttnThreads, 1)
    attn_kernel(const __grid_constant__ AttnMaps maps, const __grid_constant__ AttnParams p)
{
    using Sm = AttnSmem<DP>;
    constexpr int kStages = Sm::kStages, kTile = Sm::kTile, kHalves = Sm::kHalves;
    constexpr bool kOwnP = Sm::kOwnP;
    constexpr float kMost = kF16 ? kMostPF16 : kMostP;
    auto pack_p = [](float a, float b) { return kF16 ? pack_f16x2(a, b) : pack_bf16x2(a, b); };
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *qbuf = smem, *ring = smem + 2 * kTile;
    // single items: stream 1's (m, l) by row; narrow ones: stream 0's too, from entry 64 on
    float2 *stats = reinterpret_cast<float2 *>(smem + Sm::kStats);
    AttnItem *items = reinterpret_cast<AttnItem *>(smem + Sm::kItem);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + Sm::kBars), *empty = full + kStages;
    uint64_t *item_full = empty + kStages, *item_empty = item_full + kItems;
    uint64_t *q_full = item_empty + kItems;   // [2]
    uint64_t *q_empty = q_full + 2;
    uint64_t *s_full = q_empty + 1;           // [2]
    uint64_t *p_half = s_full + 2;            // [2] P of the tile's first 64 keys is in place
    uint64_t *p_full = p_half + 2;            // [2]
    uint64_t *pv_half = p_full + 2;           // [2] the products of the first 64 keys are done
    uint64_t *pv_done = pv_half + 2;          // [2] all of a tile's are (P of its own)
    uint64_t *o_full = pv_done + 2;           // [2]
    uint64_t *turn = o_full + 2;              // [2] the other stream's exponentials are through (in turns, see below)
    uint64_t *xbar = turn + 2;                // the 256 softmax threads meet here
    uint64_t *end_bar = xbar + 1;             // all matrix products are done
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(end_bar + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *join_flag = reinterpret_cast<int *>(tmem_slot + 2);
    // Loads issued into each ring stage and query buffer.  No loader and (single)
    // no stream sees every phase of a stage's barriers, and a parity tells only
    // neighbouring phases apart: a barrier is waited on once this says that it is
    // in that phase or the one before.
    int *issued = join_flag + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int32_t *status = p.counters + CNT_STATUS;
    // Bounded wait, called by whole warps; the answer is the same for all lanes,
    // so a wait that gives up takes its warp out together.
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        return __all_sync(0xffffffffu, attn_wait(smem_u32(bar), parity, abort_flag, p.wait_cycles)) != 0;
    };
    auto wait_far = [&](uint64_t *bar, uint32_t parity) {
        return __all_sync(0xffffffffu, attn_wait_far(smem_u32(bar), parity, abort_flag, p.wait_cycles)) != 0;
    };
    // The same without agreement: lanes go on together whatever it says, and
    // agree at the end of their loop's round.
    auto wait_each = [&](uint64_t *bar, uint32_t parity) {
        return attn_wait_far(smem_u32(bar), parity, abort_flag, p.wait_cycles);
    };
    // load number f of stage s (from 0) has been issued
    auto wait_issued = [&](uint32_t s, uint32_t f) {
        return __all_sync(0xffffffffu, attn_wait_count(&issued[s], static_cast<int>(f), abort_flag, p.wait_cycles)) != 0;
    };
    pdl_launch_dependents();

    // The work list is on its way while the rest is set up.  (The wait is for the
    // kernels ahead, once for all threads: nobody touches memory before the barrier.)
    AttnHdr hdr = {};
    ShortList list;
    int word = 0;
    if (warp == 8) {
        pdl_wait();
        if (p.short_list) {
            list.load(p, lane);
        } else {
            hdr = *p.hdr;
            if (lane < 16) word = reinterpret_cast<const int32_t *>(p.first + blockIdx.x)[lane];
        }
    } else if (threadIdx.x < Sm::kNumBars) {
        uint64_t *bar = full + threadIdx.x;
        const int n = bar < empty ? 1
                      : bar < item_full ? 2      // empty: one arrival a stream (two from the only one that uses the stage)
                      : bar < item_empty ? 1
                      : bar < q_full ? 11        // item_empty: 8 softmax warps, 2 MMA warps, the value loader
                      : bar < q_empty ? 1
                      : bar == q_empty ? 2
                      : bar >= p_half && bar < pv_half ? 4   // p_half, p_full: a stream's warps
                      : bar == turn || bar == turn + 1 ? 4
                      : bar == xbar ? 8
                      : bar == end_bar ? 2 : 1;
        mbar_init(bar, n);
        fence_mbarrier_init();
    } else if (threadIdx.x < Sm::kNumBars + kStages + 2) {
        issued[threadIdx.x - Sm::kNumBars] = 0;
    } else if (threadIdx.x == Sm::kNumBars + kStages + 2) {
        *abort_flag = 0;
    }
    if (warp == 11 && lane == 0) {
        tma_prefetch_map(&maps.q);
        tma_prefetch_map(&maps.k);
        tma_prefetch_map(&maps.v);
    }
    if (warp == 9) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    // A tile of 128 keys in boxes of box_rows keys (a page, or 128 keys of a
    // larger one; 32 or 128 packed rows), each 64 columns wide: one lane per box.
    const int box = p.box_rows, box_shift = __ffs(box) - 1, per_tile = kAttnTileK >> box_shift;
    const int mybox = lane / kHalves, myhalf = lane % kHalves;
    // paged: lane l holds the page of box l % per_tile of tile l / per_tile of a
    // window of 32 / per_tile tiles; the next window's pages are on their way
    // while a window is used
    const int win_shift = box_shift - 2, in_win = (1 << win_shift) - 1;
    auto pages_of = [&](const int32_t *table, int tile, int seen) {
        const int64_t key = (static_cast<int64_t>(tile) << 7) + (static_cast<int64_t>(lane) << box_shift);
        const int64_t col = key >> p.page_shift;
        return key < seen && col < p.table_width ? table[col] : -1;
    };
    // load i of the CTA <- a key or value tile; false after a wait gave up
    auto load_tile = [&](const CUtensorMap *map, uint32_t i, int tile, int page, int seen, int kvh, int row0) {
        const int key = tile * kAttnTileK + mybox * box;
        const int boxes = (max(0, min(kAttnTileK, seen - tile * kAttnTileK)) + box - 1) >> box_shift;
        const uint32_t s = i % kStages, f = i / kStages;
        // the stage's previous load has been issued (perhaps by the other loader), and is used up
        if (f > 0 && !(wait_issued(s, f - 1) && wait_far(&empty[s], (f - 1) & 1))) return false;
        if (lane == 0) {
            st_release_shared(&issued[s], static_cast<int>(f) + 1);
            mbar_expect_tx(&full[s], boxes * box * 128 * kHalves);
        }
        __syncwarp();
        if (mybox < boxes) {
            const uint32_t dst = smem_u32(ring) + s * kTile + myhalf * (kAttnTileK * 128) + mybox * box * 128;
            if (kPaged) {
                if (page < 0 || page >= p.num_pages) {
                    atomicOr(status, LORA_DEV_BAD_PAGE);
                    page = p.num_pages;   // outside the map: reads as zeros
                }
                tma_load_4d_if(1, dst, map, smem_u32(&full[s]), myhalf * 64, key & ((1 << p.page_shift) - 1), kvh, page);
            } else {
                tma_load_3d_if(1, dst, map, smem_u32(&full[s]), myhalf * 64, kvh, row0 + key);
            }
        }
        return true;
    };

    if (warp == 8) {
        // ===================== work and keys ==================================
        if (p.short_list) {
            hdr = list.header(p, status, lane);
        } else if (hdr.stamp != p.stamp) {   // a list of other sizes, or none: nothing is run
            if (lane == 0) atomicOr(status, LORA_DEV_CHECK);
            hdr = {};
            word = 0;
        }
        uint32_t it = 0, nitem = 0;
        const bool cut = hdr.cut != 0;
        int unit = blockIdx.x;
        // cut: my unit [pos, end) of the list
        const int end = cut ? min((unit + 1) * hdr.unit_cost, hdr.cost) : 0;
        int pos = 0;
        AttnBlock b = {};
        bool have_b = false, ok = true, more = true;
        while (more) {
            // the next piece, handed to the other roles
            const int is = nitem % kItems;
            if (nitem >= kItems && !wait_far(&item_empty[is], (nitem / kItems - 1) & 1)) ok = false;
            if (nitem == 0 && !p.short_list) {
                if (lane < 16) reinterpret_cast<int32_t *>(&items[is])[lane] = word;   // laid out by the schedule
                __syncwarp();
            } else {
                AttnItem w = {};
                if (!cut && ok && unit < hdr.units) {
                    int blk, kvh;
                    whole_unit(hdr, p.kv_heads, unit, &blk, &kvh);
                    w = item_of(p.short_list ? list.block(p, blk) : p.blocks[blk], blk, kvh, p.tq);
                    if (kTwo) w.valid += hdr.unit_cost;
                } else if (cut && ok) {
                    const AttnItem &last = items[(nitem - 1) % kItems];
                    int blk = last.blk, kvh = last.kvh + 1;
                    if (kvh == p.kv_heads) {
                        kvh = 0;
                        if (++blk < hdr.nblocks) b = p.blocks[blk];
                    }
                    if (blk < hdr.nblocks) w = cut_piece(hdr, b, blk, kvh, p.kv_heads, p.tq, unit, end, &pos);
                }
                if (lane == 0) items[is] = w;
                __syncwarp();
            }
            const AttnItem &w = items[is];
            const int two = kTwo ? w.valid >> 1 : 0;   // two heads: their tiles take turns, 2 t + stream
            const int pair = w.pair, t0 = w.t0, n = (w.t1 - t0) << two, seen = w.seen, kvh = w.kvh, row0 = w.base;
            const int32_t *table = p.block_table + w.base * p.table_stride;
            more = w.valid;
            if (lane == 0) mbar_arrive(&item_full[is]);
            ++nitem;
            if (!more) break;
            if (cut && !have_b) {   // of the first piece's group, for what comes after it
                b = p.blocks[w.blk];
                pos = group_start(hdr, b, kvh, p.kv_heads, pair) + (w.t1 << (pair ? hdr.cut - 1 : 0));
                have_b = true;
            }
            int next = 0, cur = -1, nxt = -1;
#pragma unroll 1
            for (int t = 0; t < n; ++t) {
                const int tile = t >> two, head = kvh + (t & two);
                if (kPaged && (tile & in_win) == 0 && tile << two == t) {
                    cur = t == 0 ? pages_of(table, t0, seen) : nxt;
                    nxt = pages_of(table, t0 + tile + in_win + 1, seen);
                }
                const int page = kPaged ? __shfl_sync(0xffffffffu, cur, (tile & in_win) * per_tile + mybox) : 0;
                // whole: the next unit is claimed late, so that the last ones go to the CTAs
                // that come free first, and under the wait for the last tile's stage
                if (!cut && t == n - 1 && lane == 0) next = atomicAdd(p.counters + ACNT_NEXT, 1);
                ok = load_tile(&maps.k, it + load_of_key(pair, t), t0 + tile, page, seen, head, row0);
                if (!ok) break;
            }
            it += 2 * n;
            if (!cut) unit = static_cast<int>(gridDim.x) + __shfl_sync(0xffffffffu, next, 0);
        }
        // no CTA claims a unit any more once all have come here: the counters go back to zero
        if (lane == 0 && !cut && atom_acq_rel_gpu_add(p.counters + ACNT_DONE, 1) == static_cast<int>(gridDim.x) - 1) {
            p.counters[ACNT_NEXT] = 0;
            p.counters[ACNT_DONE] = 0;
        }
    } else if (warp == 11) {
        // ===================== queries and values =============================
        uint32_t it = 0, nitem = 0;
        bool ok = true;
        while (ok) {
            const int is = nitem % kItems;
            if (!wait_far(&item_full[is], (nitem / kItems) & 1)) break;
            const AttnItem &wi = items[is];
            const int valid = wi.valid, two = kTwo ? valid >> 1 : 0;
            const int pair = wi.pair, t0 = wi.t0, n = (wi.t1 - t0) << two, seen = wi.seen, kvh = wi.kvh;
            const int tok0 = wi.tok0, row0 = wi.base;
            const int32_t *table = p.block_table + wi.base * p.table_stride;
            __syncwarp();
            if (lane == 0) mbar_arrive(&item_empty[is]);
            ++nitem;
            if (!valid) break;
            int cur = -1, nxt = kPaged ? pages_of(table, t0, seen) : -1;
            // the queries, once the previous piece's products have read theirs
            if (nitem > 1 && !wait_far(q_empty, (nitem - 2) & 1)) break;
#pragma unroll 1
            for (int s = 0; s <= (pair | two); ++s) {
                if (lane == 0) {
                    ++issued[kStages + s];
                    mbar_expect_tx(&q_full[s], p.tq * p.group * 128 * kHalves);
                }
                __syncwarp();
                if (lane < kHalves)
                    tma_load_3d_if(1, smem_u32(qbuf) + s * kTile + lane * (kAttnTileQ * 128), &maps.q, smem_u32(&q_full[s]),
                                   lane * 64, (kvh + (s & two)) * p.group, tok0 + (two ? 0 : s * p.tq));
            }
#pragma unroll 1
            for (int t = 0; t < n && ok; ++t) {
                const int tile = t >> two, head = kvh + (t & two);
                if (kPaged && (tile & in_win) == 0 && tile << two == t) {
                    cur = nxt;
                    nxt = pages_of(table, t0 + tile + in_win + 1, seen);
                }
                const int page = kPaged ? __shfl_sync(0xffffffffu, cur, (tile & in_win) * per_tile + mybox) : 0;
                ok = load_tile(&maps.v, it + load_of_value(pair, t, n), t0 + tile, page, seen, head, row0);
            }
            it += 2 * n;
        }
    } else if (warp >= 9) {
        // ===================== MMA issuers ====================================
        // Warp 9 + s issues stream s's products: a product executes in 64 cycles
        // and issuing one takes 35 (66 with a branch around it), so one warp for
        // both streams would be as busy as the tensor cores.  All lanes run the
        // same code and the elected one's instructions take effect.
        const int s = uniform(warp - 9);
        const uint32_t tmem_u = uniform(static_cast<int>(tmem));
        uint32_t it = 0, nitem = 0, nq0 = 0, nq1 = 0, np = 0;
        const uint32_t qlo = umma_lo(smem_u32(qbuf), 16);
        const uint32_t klo = umma_lo(smem_u32(ring), 16), vlo = umma_lo(smem_u32(ring), kAttnTileK * 128);
        const int dsteps = (p.head_dim + 15) / 16;
        const uint32_t idesc_pv = kF16 ? umma_idesc_f16_bn(kAttnTileQ, dsteps * 16) : umma_idesc_bf16_bn(kAttnTileQ, dsteps * 16);
        const uint32_t s_cells = tmem_u + s * kColS, o_cells = tmem_u + kColO + s * DP;
        const uint32_t p_cells = kOwnP ? tmem_u + kColP + s * 64 : s_cells;
        auto commit = [&](uint64_t *bar) { umma_commit_if(elect_one(), bar); };
        bool ok = true;
        while (ok) {
            const int is = nitem % kItems;
            if (!wait_far(&item_full[is], (nitem / kItems) & 1)) break;
            const AttnItem &wi = items[is];
            const int valid = uniform(wi.valid), pair = uniform(wi.pair), t0 = uniform(wi.t0);
            const int two = kTwo ? valid >> 1 : 0, n = (uniform(wi.t1) - t0) << two;
            const int seen = uniform(wi.seen) - t0 * kAttnTileK;   // keys that any row sees, from t0
            // pair: both streams go through all tiles, stream 0 uses its first `mine`;
            // single: stream s uses tiles s, s + 2, ...
            const int mine = pair ? (s ? n : max(0, min(n, uniform(wi.end0) - t0))) : (n - s + 1) >> 1;
            const int all = pair ? n : mine;
            __syncwarp();
            if (lane == 0) mbar_arrive(&item_empty[is]);
            ++nitem;
            if (!valid) break;
            // load i of the CTA has landed
            auto wait_load = [&](uint32_t i) {
                const uint32_t st = i % kStages, f = i / kStages;
                ok &= attn_wait_count(&issued[st], static_cast<int>(f), abort_flag, p.wait_cycles);
                ok &= wait_each(&full[st], f & 1);
            };
            auto release = [&](uint32_t st) {
                const uint32_t lead = elect_one();
                umma_commit_if(lead, &empty[st]);
                if (!pair) umma_commit_if(lead, &empty[st]);
            };
            ok &= wait_each(&q_full[0], nq0++ & 1);
            if (pair | two) ok &= wait_each(&q_full[1], nq1++ & 1);
            if (all == 0) commit(q_empty);
            // Round k: tile k's values, then the keys of tile k + 1, whose scores go over
            // the P just read (round -1: only keys).  What can be waited for ahead of P
            // is, and the stages go back last: from P to the next scores nothing is in
            // the way of the tensor cores.
#pragma unroll 1
            for (int k = -1; k < all; ++k) {
                const int tv = pair ? k : s + 2 * k, tk = pair ? k + 1 : s + 2 * k + 2;
                const uint32_t iv = it + load_of_value(pair, tv, n), ik = it + load_of_key(pair, tk);
                const uint32_t stv = iv % kStages, stk = ik % kStages;
                const bool more = k + 1 < all;
                if (k >= 0) wait_load(iv);
                if (more) wait_load(ik);
                auto scores = [&] {   // of tile k + 1
                    if (k + 1 >= mine) return;
                    tc_fence_after();
                    const int keys = min(kAttnTileK, seen - (tk >> two) * kAttnTileK);
                    const uint32_t idesc = umma_idesc_bf16(kAttnTileQ, max(16, (keys + 15) & ~15));
                    const uint32_t qd = qlo + ((pair | two) && s ? kTile >> 4 : 0), kd = klo + stk * (kTile >> 4);
                    const uint32_t lead = elect_one();
                    auto step = [&](int kk) {
                        const uint32_t o = (kk >> 2) * ((kAttnTileK * 128) >> 4) + (kk & 3) * 2;
                        umma_ss_if(lead, s_cells, qd + o, kd + o, idesc, kk > 0);
                    };
                    if (dsteps == DP / 16) {
#pragma unroll
                        for (int kk = 0; kk < DP / 16; ++kk) step(kk);
                    } else {
#pragma unroll 1
                        for (int kk = 0; kk < dsteps; ++kk) step(kk);
                    }
                    umma_commit_if(lead, &s_full[s]);
                };
                const bool values = k >= 0 && k < mine;
                const int keys = values ? min(kAttnTileK, seen - (tv >> two) * kAttnTileK) : 0;
                const uint32_t vd = vlo + stv * (kTile >> 4), par = np & 1;
                auto step = [&](uint32_t lead, int kk) {
                    umma_ts_if(lead, o_cells, p_cells + kk * 8, vd + kk * (2048 >> 4), idesc_pv, kk > 0 ? 1 : k > 0);
                };
                if (values) {
                    // keys past the last one that a row sees: their p is 0, but 0 times
                    // what the tile holds there (another request's rows, stale pages)
                    // may be NaN
                    const int up = (keys + 15) & ~15;
                    if (keys > 0 && keys != up) {
                        uint8_t *v = ring + stv * kTile;
                        for (int e = lane; e < (up - keys) * 8 * kHalves; e += 32) {
                            const int r = keys + e / (8 * kHalves), c = e % (8 * kHalves);
                            *reinterpret_cast<uint4 *>(v + (c >> 3) * (kAttnTileK * 128) + r * 128 + (c & 7) * 16) =
                                make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    ++np;
                    ok &= wait_each(&p_half[s], par);   // the first half of P is in place, and S has been read
                    tc_fence_after();
                    const uint32_t lead = elect_one();
                    if (keys == kAttnTileK) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) step(lead, kk);
                    } else {
#pragma unroll 1
                        for (int kk = 0; kk < 4 && kk * 16 < keys; ++kk) step(lead, kk);
                    }
                    umma_commit_if(lead, &pv_half[s]);
                }
                if (kOwnP) scores();
                if (values) {
                    ok &= wait_each(&p_full[s], par);
                    tc_fence_after();
                    const uint32_t lead = elect_one();
                    if (keys == kAttnTileK) {
#pragma unroll
                        for (int kk = 4; kk < 8; ++kk) step(lead, kk);
                    } else {
#pragma unroll 1
                        for (int kk = 4; kk * 16 < keys; ++kk) step(lead, kk);
                    }
                    if (kOwnP) umma_commit_if(lead, &pv_done[s]);
                    if (k == mine - 1) umma_commit_if(lead, &o_full[s]);
                }
                if (!kOwnP) scores();
                if (k >= 0) release(stv);
                if (more) release(stk);
                if (k + 2 == all) commit(q_empty);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
            }
            it += 2 * n;
        }
        // nothing issued here is in flight when the block ends
        commit(end_bar);
        attn_wait(smem_u32(end_bar), 0, abort_flag, max(p.wait_cycles, static_cast<uint32_t>(kWaitShort)));
    } else {
        // ===================== softmax and results ============================
        const int s = warp >> 2, quad = warp & 3;
        const int r = quad * 32 + lane;   // my row of the query tile
        const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t t_s = tmem + lanes + s * kColS, t_o = tmem + lanes + kColO + s * DP;
        const uint32_t t_p = kOwnP ? tmem + lanes + kColP + s * 64 : t_s;
        const int G = p.group, D = p.head_dim;
        const float c = p.scale * 1.4426950408889634f;
        auto offset = [&](float m) {   // p = 2^(c x + offset(m))
            if (kF16) return m == -INFINITY ? 0.f : fmaf(-m, c, kLiftF16);
            return m == -INFINITY ? 0.f : -m * c;
        };
        uint32_t nitem = 0, ns = 0, no = 0, nx = 0, nt = 0;
        auto meet = [&] {   // all 256 threads
            __syncwarp();
            if (lane == 0) mbar_arrive(xbar);
            wait(xbar, nx++ & 1);
        };
        while (true) {
            const int is = nitem % kItems;
            if (!wait(&item_full[is], (nitem / kItems) & 1)) break;
            const AttnItem w = items[is];
            __syncwarp();
            if (lane == 0) mbar_arrive(&item_empty[is]);
            ++nitem;
            if (!w.valid) break;
            const int n = w.t1 - w.t0;
            const bool own = kTwo && w.valid == 2;   // a head of its own for each stream
            // key tiles of the two streams
            const int cnt0 = w.pair ? max(0, min(w.t1, w.end0) - w.t0) : own ? n : (n + 1) / 2, cnt1 = w.pair || own ? n : n / 2;
            const int mine_n = s ? cnt1 : cnt0;
            const int i = r / G, tok = (w.pair && s ? p.tq : 0) + i;   // my token of the block
            const bool row_ok = i < p.tq && tok < w.ntok;
            const int limit = row_ok ? max(0, min(w.kv_len, w.qpos0 + tok + 1)) : 0;
            const bool live = __any_sync(0xffffffffu, limit > 0);
            const bool narrow = kPaged && !w.pair && w.ntok * G <= kAttnFewRows, two = w.ntok * G > 8;   // two: rows past the eighth
            // Where P shares S's cells a stream's softmax and products alternate; left alone the
            // two streams fall into step, both in their exponentials and then both waiting for
            // the tensor cores.  With two query tiles they take turns instead: stream 1's
            // exponentials of a tile follow stream 0's, which follow stream 1's of the tile
            // before.  A 16384-token prompt took 1280 us so, 1600 without; over one to three
            // tiles waiting for the turn costs more than it gives (77 tokens: 8.5 us without,
            // 9.3 with).
            const bool in_turns = !kOwnP && w.pair && n >= 4;
            const int both = min(cnt0, cnt1);
            float m = -INFINITY, l = 0.f;
            // narrow: rows lane / 4 and 8 more, of which this lane has keys 8 j + 2 (lane % 4) and the next
            float nm[2] = {-INFINITY, -INFINITY}, nl[2] = {0.f, 0.f}, nf[2][2];
            bool nu[2][2];
            int nlim[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int t = ((lane >> 2) + 8 * h) / G;
                nlim[h] = t < w.ntok ? max(0, min(w.kv_len, w.qpos0 + t + 1)) : 0;
            }
            for (int k = 0; k < mine_n; ++k) {
                const int tile = w.pair || own ? w.t0 + k : w.t0 + s + 2 * k;
                const int rem = limit - tile * kAttnTileK;   // my visible columns of this tile
                if (!wait(&s_full[s], ns++ & 1)) break;
                tc_fence_after();
                // The previous tile's products are done: O holds them, P may be overwritten, and
                // all warps of the stream have handed theirs over (none may be counted twice in
                // one phase of p_full).  Sharing S's cells, these scores could not be here otherwise.
                auto products_done = [&] {
                    if (kOwnP && k > 0) {
                        wait(&pv_done[s], (ns - 2) & 1);
                        tc_fence_after();
                    }
                };
                if (narrow && live) {
                    const uint64_t c2 = pack_f2(c, c);
                    const int first = 2 * (lane & 3);
                    int see[2];   // visible columns, from my first on
#pragma unroll
                    for (int h = 0; h < 2; ++h) see[h] = nlim[h] - tile * kAttnTileK - first;
                    float x[64];   // x[4 j + 2 h + e]: row 8 h + lane / 4, key 8 j + first + e
                    tmem_ld_16x256(t_s, x);
                    tmem_ld_wait();
                    tmem_use32(x);
                    tmem_use32(x + 32);
                    if (__any_sync(0xffffffffu, see[0] + first < kAttnTileK || (two && see[1] + first < kAttnTileK))) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (h == 1 && !two) continue;
#pragma unroll
                            for (int j = 0; j < 16; ++j)
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    x[4 * j + 2 * h + e] = 8 * j + e < see[h] ? x[4 * j + 2 * h + e] : -INFINITY;
                        }
                    }
                    uint32_t pk[32];
                    bool move = (nm[0] == -INFINITY && see[0] + first > 0) || (two && nm[1] == -INFINITY && see[1] + first > 0);
                    for (int round = 0;; ++round) {
                        if (__any_sync(0xffffffffu, move)) {
                            products_done();
                            float f[2];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                f[h] = 1.f;
                                if (h == 1 && !two) continue;
                                float mn = nm[h];
#pragma unroll
                                for (int j = 0; j < 16; ++j) mn = fmaxf(fmaxf(mn, x[4 * j + 2 * h]), x[4 * j + 2 * h + 1]);
                                mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, 1));
                                mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, 2));
                                f[h] = mn == nm[h] ? 1.f : ex2((nm[h] - mn) * c);
                                nm[h] = mn;
                                nl[h] *= f[h];
                            }
#pragma unroll 1
                            for (int q = 0; q < (k > 0 ? DP / 64 : 0); ++q) {
                                float y[32];
                                tmem_ld_16x256_half(t_o + 64 * q, y);
                                tmem_ld_wait();
                                tmem_use32(y);
#pragma unroll
                                for (int e = 0; e < 32; ++e) y[e] *= f[(e >> 1) & 1];
                                tmem_st_16x256_half(t_o + 64 * q, y);
                            }
                        }
                        float part[2];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            part[h] = 0.f;
                            if (h == 1 && !two) {
#pragma unroll
                                for (int j = 0; j < 16; ++j) pk[2 * j + 1] = 0;
                                continue;
                            }
                            const float off = offset(nm[h]);
                            const uint64_t off2 = pack_f2(off, off);
                            uint64_t sum[2] = {0, 0};
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                float a, b;
                                unpack_f2(fma_f2(pack_f2(x[4 * j + 2 * h], x[4 * j + 2 * h + 1]), c2, off2), a, b);
                                a = ex2(a);
                                b = ex2(b);
                                sum[j & 1] = add_f2(sum[j & 1], pack_f2(a, b));
                                pk[2 * j + h] = pack_p(a, b);
                            }
                            float a, b;
                            unpack_f2(add_f2(sum[0], sum[1]), a, b);
                            part[h] = a + b;
                        }
                        move = part[0] > kMost || part[1] > kMost;
                        if (round == 1 || !__any_sync(0xffffffffu, move)) {
                            nl[0] += part[0];
                            nl[1] += part[1];
                            break;
                        }
                    }
                    products_done();
                    tmem_st_16x128(t_p, pk);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_half[s]);
                } else if (live) {
                    const uint64_t c2 = pack_f2(c, c);
                    // two halves of 64 keys, so that the first one's products start early
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t cells = t_s + 64 * h;
                        const int seen = rem - 64 * h;   // my visible columns of this half
                        float x[64];
                        tmem_ld32(cells, x);
                        tmem_ld32(cells + 32, x + 32);
                        if (h == 1) tmem_st_wait();      // the first half's P is in place
                        tmem_ld_wait();
                        if (h == 0 && in_turns && k < both) {   // stream 0's first has none before it
                            if (s == 1 || nt > 0) wait(&turn[s], (nt - (s == 0)) & 1);
                            ++nt;
                        }
                        tmem_use32(x);
                        tmem_use32(x + 32);
                        if (h == 1) {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&p_half[s]);
                        }
                        if (__any_sync(0xffffffffu, seen < 64)) {
#pragma unroll
                            for (int e = 0; e < 64; ++e) x[e] = e < seen ? x[e] : -INFINITY;
                        }
                        if (h == 0) {   // the first score (-infinity if it is not seen), or the largest of the first few
                            float first = x[0];
                            if (kF16 && k == 0) {
#pragma unroll
                                for (int e = 1; e < 8; ++e) first = fmaxf(first, x[e]);
                            }
                            m = m == -INFINITY ? first : m;
                        }
                        uint32_t pk[32];
                        float total;
                        auto exps = [&] {
                            const float off = offset(m);
                            const uint64_t off2 = pack_f2(off, off);
                            uint64_t sum[2] = {0, 0};
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                float a, b;
                                unpack_f2(fma_f2(pack_f2(x[2 * e], x[2 * e + 1]), c2, off2), a, b);
                                a = ex2(a);
                                b = ex2(b);
                                sum[e & 1] = add_f2(sum[e & 1], pack_f2(a, b));
                                pk[e] = pack_p(a, b);
                            }
                            float a, b;
                            unpack_f2(add_f2(sum[0], sum[1]), a, b);
                            total = a + b;
                        };
                        exps();
                        if (__any_sync(0xffffffffu, total > kMost || (m == -INFINITY && seen > 0))) {
                            if (h == 0) {
                                products_done();
                            } else {
                                wait(&pv_half[s], (ns - 1) & 1);
                                tc_fence_after();
                            }
                            float mn = m, y[32];
                            if (kOwnP && h == 1) {   // S may be gone
#pragma unroll
                                for (int e = 0; e < 64; e += 2) mn = fmaxf(fmaxf(mn, x[e]), x[e + 1]);
                            } else {
#pragma unroll 1
                                for (int q = 0; q < 2; ++q) {
                                    tmem_ld32(cells + 32 * q, y);
                                    tmem_ld_wait();
                                    tmem_use32(y);
#pragma unroll
                                    for (int e = 0; e < 32; ++e) mn = fmaxf(mn, e < seen - 32 * q ? y[e] : -INFINITY);
                                }
                            }
                            const float f = mn == m ? 1.f : ex2((m - mn) * c);   // 0 from -infinity
                            m = mn;
                            l *= f;
#pragma unroll 1
                            for (int q = 0; q < (k + h > 0 ? DP / 32 : 0); ++q) {
                                tmem_ld32(t_o + 32 * q, y);
                                tmem_ld_wait();
                                tmem_use32(y);
#pragma unroll
                                for (int e = 0; e < 32; ++e) y[e] *= f;
                                tmem_st32(t_o + 32 * q, y);
                            }
                            exps();
                        }
                        l += total;
                        if (h == 1 && in_turns && k < both && lane == 0) mbar_arrive(&turn[1 - s]);
                        if (h == 0) products_done();
                        tmem_st16(t_p + 32 * h, pk);
                        tmem_st16(t_p + 32 * h + 16, pk + 16);
                    }
                    tmem_st_wait();
                } else {
                    if (in_turns && k < both) {
                        if (s == 1 || nt > 0) wait(&turn[s], (nt - (s == 0)) & 1);
                        ++nt;
                    }
                    if (in_turns && k < both && lane == 0) mbar_arrive(&turn[1 - s]);
                    products_done();   // not ahead of the stream's other warps
                    if (lane == 0) mbar_arrive(&p_half[s]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[s]);
            }

            // ---- results ----------------------------------------------------
            const int g = r - i * G;
            // factors of the two streams' sums (single); a stream without keys for the
            // row has nothing defined in O
            float f0 = 1.f, f1 = 0.f;
            bool use0 = l != 0.f, use1 = false;
            if (mine_n > 0) wait(&o_full[s], no++ & 1);
            if (!w.pair) {
                // both streams worked on the same rows: stream 0's threads join them
                if (narrow) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        nl[h] += __shfl_xor_sync(0xffffffffu, nl[h], 1);
                        nl[h] += __shfl_xor_sync(0xffffffffu, nl[h], 2);
                        if (!own && quad == 0 && (lane & 3) == 0)
                            stats[(s ? 0 : 64) + (lane >> 2) + 8 * h] = make_float2(nm[h], nl[h]);
                    }
                } else if (s == 1) {
                    stats[r] = make_float2(m, l);
                }
                if (!own) meet();
                if (s == 0 && !narrow) {
                    const float2 st = stats[r];
                    const float mm = fmaxf(m, st.x);
                    use1 = st.y != 0.f;
                    f0 = use0 ? ex2((m - mm) * c) : 0.f;
                    f1 = use1 ? ex2((st.x - mm) * c) : 0.f;
                    m = mm;
                    l = l * f0 + st.y * f1;
                }
            }
            tc_fence_after();
            const bool mine = w.pair || s == 0;
            const int rho = tok * G + g;   // my row of the block
            if (narrow) {
                // rows by quads, as in the softmax.  Stream s's first warp joins half of the
                // columns, both streams' O of the row by one load each; or (own) it has all
                // columns of its own rows, a half by each load
                if (quad == 0) {
                    const bool whole = w.parts == 1;
                    constexpr int kCols = DP / 2;   // columns of a stream's warp
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int row = (lane >> 2) + 8 * h;
                        const float2 a = own ? make_float2(nm[h], nl[h]) : stats[64 + row], b = own ? a : stats[row];
                        const float mm = fmaxf(a.x, b.x);
                        const bool u0 = a.y != 0.f, u1 = b.y != 0.f;
                        const float e0 = u0 ? ex2((a.x - mm) * c) : 0.f, e1 = u1 ? ex2((b.x - mm) * c) : 0.f;
                        nm[h] = mm;
                        nl[h] = own ? a.y : a.y * e0 + b.y * e1;
                        const float inv = whole && nl[h] != 0.f ? 1.f / nl[h] : 1.f;
                        nf[h][0] = e0 * inv;
                        nf[h][1] = e1 * inv;
                        nu[h][0] = u0;
                        nu[h][1] = u1;
                    }
                    const uint32_t cells = tmem + kColO + s * (own ? DP : kCols), next = own ? kCols : DP;
                    float y[2][kCols / 2];   // [stream, or half][4 j + 2 h + e]
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        if (DP == 128) tmem_ld_16x256_half(cells + q * next, y[q]);
                        else tmem_ld_16x256_quarter(cells + q * next, y[q]);
                    }
                    tmem_ld_wait();
                    tmem_use<kCols / 2>(y[0]);
                    tmem_use<kCols / 2>(y[1]);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int row = (lane >> 2) + 8 * h, t = row / G, gg = row - t * G;
                        if (t >= w.ntok) continue;
                        const int head = (w.kvh + (own ? s : 0)) * G + gg, c0 = (own ? 0 : s * kCols) + 2 * (lane & 3);
                        const int64_t at = static_cast<int64_t>(w.tok0) + t;
                        uint16_t *out = p.o + at * p.o_tok + head * p.o_head;
                        float *part = p.part + (static_cast<int64_t>(w.slot) * p.part_rows + row) * D;
#pragma unroll
                        for (int j = 0; j < kCols / 8; ++j) {
                            if (own) {
#pragma unroll
                                for (int q = 0; q < 2; ++q)
                                    if (c0 + 8 * j + q * kCols < D)
                                        *reinterpret_cast<uint32_t *>(out + c0 + 8 * j + q * kCols) =
                                            nu[h][0] ? pack_bf16x2(y[q][4 * j + 2 * h] * nf[h][0], y[q][4 * j + 2 * h + 1] * nf[h][0])
                                                     : 0;
                                continue;
                            }
                            float v[2];
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                v[e] = (nu[h][0] ? y[0][4 * j + 2 * h + e] * nf[h][0] : 0.f) +
                                       (nu[h][1] ? y[1][4 * j + 2 * h + e] * nf[h][1] : 0.f);
                            if (c0 + 8 * j >= D) continue;
                            if (whole) *reinterpret_cast<uint32_t *>(out + c0 + 8 * j) = pack_bf16x2(v[0], v[1]);
                            else *reinterpret_cast<float2 *>(part + c0 + 8 * j) = make_float2(v[0], v[1]);
                        }
                        if ((own || s == 0) && (lane & 3) == 0) {
                            if (!whole)
                                p.part_ml[static_cast<int64_t>(w.slot) * p.part_rows + row] = make_float2(nm[h], nl[h]);
                            else if (p.lse)
                                p.lse[at * p.heads + head] =
                                    nl[h] == 0.f ? -INFINITY : (nm[h] * c + log2_sum<kF16>(nl[h])) * 0.6931471805599453f;
                        }
                    }
                }
            } else if (mine && __any_sync(0xffffffffu, row_ok)) {
                const bool whole = w.parts == 1;
                const float inv = whole && l != 0.f ? 1.f / l : 1.f;
                f0 *= inv;
                f1 *= inv;
                const int64_t row = static_cast<int64_t>(w.tok0) + tok;
                const int head = w.kvh * G + g;
                uint8_t *out = whole ? reinterpret_cast<uint8_t *>(p.o + row * p.o_tok + head * p.o_head)
                                     : reinterpret_cast<uint8_t *>(p.part + (static_cast<int64_t>(w.slot) * p.part_rows + rho) * D);
#pragma unroll 1
                for (int q = 0; 32 * q < D; ++q) {
                    float o[32];
                    tmem_ld32(t_o + 32 * q, o);
                    tmem_ld_wait();
                    tmem_use32(o);
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = use0 ? o[e] * f0 : 0.f;
                    if (!w.pair) {
                        float o1[32];
                        tmem_ld32(t_o + DP + 32 * q, o1);
                        tmem_ld_wait();
                        tmem_use32(o1);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] += use1 ? o1[e] * f1 : 0.f;
                    }
                    if (whole) {
                        uint32_t v[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] = pack_bf16x2(o[2 * e], o[2 * e + 1]);
#pragma unroll
                        for (int e = 0; e < 16; e += 8) {
                            // whole sectors where rows allow it: 40 prompts of 100 to 200
                            // tokens take 43 us with 32-byte stores and 49 with 16
                            const int col = 32 * q + 2 * e;
                            if (row_ok && p.o_wide && col + 8 < D) {
                                store32(out + 2 * col, v + e);
                            } else {
                                if (row_ok && col < D)
                                    *reinterpret_cast<uint4 *>(out + 2 * col) = make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                                if (row_ok && col + 8 < D)
                                    *reinterpret_cast<uint4 *>(out + 2 * col + 16) =
                                        make_uint4(v[e + 4], v[e + 5], v[e + 6], v[e + 7]);
                            }
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            if (row_ok && 32 * q + e < D) store32(out + (32 * q + e) * 4, reinterpret_cast<uint32_t *>(o + e));
                    }
                }
                if (row_ok) {
                    if (!whole)
                        p.part_ml[static_cast<int64_t>(w.slot) * p.part_rows + rho] = make_float2(m, l);
                    else if (p.lse)
                        p.lse[row * p.heads + head] = l == 0.f ? -INFINITY : (m * c + log2_sum<kF16>(l)) * 0.6931471805599453f;
                }
            }
            if (w.parts > 1) {
                // the piece that finishes last joins the group's pieces, in their order
                meet();   // with the release below, every thread's writes come before the count
                if (threadIdx.x == 0)
                    *join_flag = atom_acq_rel_gpu_add(p.counters + ACNT_GROUP + w.unit0, 1) == w.parts - 1;
                meet();
                if (*join_flag) {
                    const int d4 = D / 4, all = w.ntok * G * d4;
                    if (all > 256) {
                        join_pieces<kF16>(p, w.ntok, w.tok0, w.kvh, w.parts, w.unit0, c);
                    } else if (threadIdx.x < all) {   // a thread's element, four pieces in flight
                        const int rr = threadIdx.x / d4, col = (threadIdx.x - rr * d4) * 4;
                        float mm = -INFINITY, ll = 0.f, a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
                        for (int k = 0; k < w.parts; ++k) {
                            const float2 ml = __ldcg(p.part_ml + join_slot(p, w.unit0, k) + rr);
                            const float4 v = __ldcg(reinterpret_cast<const float4 *>(p.part + (join_slot(p, w.unit0, k) + rr) * D + col));
                            const float mn = fmaxf(mm, ml.x);
                            const float f = ml.y == 0.f ? 0.f : ex2((ml.x - mn) * c), g = ll == 0.f ? 0.f : ex2((mm - mn) * c);
                            mm = mn;
                            ll = ll * g + f * ml.y;
                            a[0] = a[0] * g + f * v.x;
                            a[1] = a[1] * g + f * v.y;
                            a[2] = a[2] * g + f * v.z;
                            a[3] = a[3] * g + f * v.w;
                        }
                        const float inv = ll == 0.f ? 0.f : 1.f / ll;
                        const int tk = rr / G, hd = w.kvh * G + (rr - tk * G);
                        const int64_t row = static_cast<int64_t>(w.tok0) + tk;
                        *reinterpret_cast<uint2 *>(p.o + row * p.o_tok + hd * p.o_head + col) =
                            make_uint2(pack_bf16x2(a[0] * inv, a[1] * inv), pack_bf16x2(a[2] * inv, a[3] * inv));
                        if (p.lse && col == 0)
                            p.lse[row * p.heads + hd] = ll == 0.f ? -INFINITY : (mm * c + log2_sum<kF16>(ll)) * 0.6931471805599453f;
                    }
                    if (threadIdx.x == 0) p.counters[ACNT_GROUP + w.unit0] = 0;
                }
            } else if (!w.pair && !own) {
                tc_fence_before();
                meet();   // O of stream 1 and its stats have been read
            }
            tc_fence_before();
        }
    }

    // ---- teardown -----------------------------------------------------------
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (*abort_flag) {
        // loads in flight are waited for (bounded) before the shared memory goes
        auto settle = [&](uint64_t *bar, uint32_t parity) {
            attn_wait(smem_u32(bar), parity, abort_flag, static_cast<uint32_t>(kWaitShort));
        };
        if (threadIdx.x == 0) atomicOr(status, LORA_DEV_TIMEOUT);
        if (warp == 8 && lane == 0)
            for (int s = 0; s < kStages; ++s)
                if (issued[s] > 0) settle(&full[s], (issued[s] - 1) & 1);
        if (warp == 11 && lane == 0)
            for (int s = 0; s < 2; ++s)
                if (issued[kStages + s] > 0) settle(&q_full[s], (issued[kStages + s] - 1) & 1);
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    }
    if (warp == 9) tmem_dealloc(tmem, 512);
}

template <int DP, bool kPaged, bool kTwo, bool kF16 = false>
static cudaError_t launch(const AttnMaps &maps, const AttnParams &p, cudaStream_t stream)
{
    static int configured[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
    constexpr int bytes = AttnSmem<DP>::kBytes;
    if (dev >= 64 || !configured[dev]) {
        const cudaError_t e =
            cudaFuncSetAttribute(attn_kernel<DP, kPaged, kTwo, kF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        if (dev < 64) configured[dev] = 1;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.ctas));
    cfg.blockDim = dim3(kAttnThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    pdl_attribute(cfg, at);
    return cudaLaunchKernelEx(&cfg, attn_kernel<DP, kPaged, kTwo, kF16>, maps, p);
}

cudaError_t launch_attn(AttnParams &p, cudaStream_t stream)
{
    AttnMaps m;
    const uint64_t D = p.head_dim, row = D * 2;
    // a stride over an extent of 1 is never used; the map wants a valid one
    auto bytes = [&](int64_t stride, int64_t extent) {
        return extent > 1 ? static_cast<uint64_t>(stride) * 2 : row;
    };
    const uint32_t G = static_cast<uint32_t>(p.group);
    {
        const uint64_t dims[3] = {D, static_cast<uint64_t>(p.heads), static_cast<uint64_t>(p.T)};
        const uint64_t st[2] = {bytes(p.q_head, p.heads), bytes(p.q_tok, p.T)};
        const uint32_t box[3] = {64, G, static_cast<uint32_t>(p.tq)};
        if (!encode_map(&m.q, p.q, 3, dims, st, box, CU_TENSOR_MAP_SWIZZLE_128B)) return cudaErrorInvalidValue;
    }
    if (p.paged) {
        const int page = 1 << p.page_shift;
        p.box_rows = page < kAttnTileK ? page : kAttnTileK;
        const uint64_t dims[4] = {D, static_cast<uint64_t>(page), static_cast<uint64_t>(p.kv_heads),
                                  static_cast<uint64_t>(p.num_pages)};
        const uint64_t st[3] = {bytes(p.slot_stride, page), bytes(p.head_stride, p.kv_heads),
                                bytes(p.page_stride, p.num_pages)};
        const uint32_t box[4] = {64, static_cast<uint32_t>(p.box_rows), 1, 1};
        if (!encode_map(&m.k, p.k, 4, dims, st, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !encode_map(&m.v, p.v, 4, dims, st, box, CU_TENSOR_MAP_SWIZZLE_128B))
            return cudaErrorInvalidValue;
    } else {
        p.box_rows = kAttnTileK;   // (32 rows a box: no faster for prompts of 1 to 400 tokens, 1 % slower for long ones)
        const uint64_t dims[3] = {D, static_cast<uint64_t>(p.kv_heads), static_cast<uint64_t>(p.T)};
        const uint64_t ks[2] = {bytes(p.k_head, p.kv_heads), bytes(p.k_tok, p.T)};
        const uint64_t vs[2] = {bytes(p.v_head, p.kv_heads), bytes(p.v_tok, p.T)};
        const uint32_t box[3] = {64, 1, static_cast<uint32_t>(p.box_rows)};
        if (!encode_map(&m.k, p.k, 3, dims, ks, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !encode_map(&m.v, p.v, 3, dims, vs, box, CU_TENSOR_MAP_SWIZZLE_128B))
            return cudaErrorInvalidValue;
    }
    if (!p.paged) return p.head_dim <= 64 ? launch<64, false, false>(m, p, stream) : launch<128, false, false>(m, p, stream);
    if (p.f16) return p.head_dim <= 64 ? launch<64, true, false, true>(m, p, stream) : launch<128, true, false, true>(m, p, stream);
    if (p.two) return p.head_dim <= 64 ? launch<64, true, true>(m, p, stream) : launch<128, true, true>(m, p, stream);
    return p.head_dim <= 64 ? launch<64, true, false>(m, p, stream) : launch<128, true, false>(m, p, stream);
}

}  // namespace lora
