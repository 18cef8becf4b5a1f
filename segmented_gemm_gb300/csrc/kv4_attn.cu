// lora_kv4_attn (include/lora_kv.h): attention of a step's new tokens over the
// paged cache held in 4 bits.
//
// For column c (a token and a query head of a key head's group) and key j:
//   s_jc = k_j . q_c,  p_jc = exp2(x_jc - m_c) with x = scale log2(e) s,
//   o_c = sum_j p_jc v_j / l_c,  l_c = sum_j p_jc
// over the keys that the column's token sees; m_c is a score that no key's x is
// more than kSlack above, moved (and o, l scaled) when one is.
//
// A quarter of the bytes that bf16 takes, so a decode step is bound by HBM only if
// turning codes into operands costs less than a byte takes to arrive: 16 keys of a
// head (2304 bytes) are 4096 elements, 128 of each lane.  Hence:
//   - keys are the rows of the products (m16n8k16), S^T = K Q^T and O^T = V^T P^T:
//     8 columns fit the 4 to 8 query heads of a group, where 16 would be half empty,
//     and the unpacked codes are the A operand, straight from registers;
//   - a tile lies in memory as its lanes want it: one 16-byte load for each half of
//     the keys, one for each half of the values, the conversion instruction
//     (two codes to a pair of fp16) and one product with the scale pair;
//   - fp16 operands: code times scale is exact, q is scaled by a power of two a
//     column, p of at most 2^kSlack has three bits more than in bf16 (as it has where keys and
//     values are unpacked first, kv4_wide.cu);
//   - a warp is on its own: it takes tiles of 16 keys from its own ring of bulk
//     copies, so nothing but the ends of pieces is synchronised.
//
// The groups (request, key head, block of columns) in a row, with what beginning one
// costs (kGap) ahead of its tiles, are cut evenly over all warps.  Whole groups are
// written by their warp.  The pieces of a cut one meet in shared memory at the end,
// once for a CTA; those of a group that CTAs share in the workspace, where the
// CTA that stores the last of them joins them in order, so that results do not depend
// on timing.
//
// What bounds it, and what it measured (32 query and 8 kv heads of 128 unless said; a copy has 6780 GB/s):
//   128 requests of one token over 1000 to 16000, 1.17 GB: 197 us, 5.9 TB/s; the tiles at
//     6.7 TB/s, then one of an SM's two CTAs ends 15 % before the other, and the joins (7 us)
//   32 over 100 to 8000, 163 MB: 40 us; the tiles take 27, the lists and the first loads 4, the ends of
//     shares and the joins 5 to 9
//   one over 1000: 12 us, all latency (counts, table, tiles, two tiles a warp, two joins)
// The integer pipe is the busiest unit (it converts the codes, 16 lanes a cycle), so whatever could
// went elsewhere: scales become fp16 pairs by a multiplication, masks have a branch of their own, addresses
// are made 32 tiles at a time.  That took the first case from 242 to 197 us.  No gain: two tiles a round
// (235 us where one took 223), three CTAs of 80 registers (259), four or sixteen warps a CTA (207, 196,
// but 15 us for one token), more units for the CTA that runs ahead (200 to 224).
#include <cuda_runtime.h>

#include "attn_ptx.cuh"
#include "block_scan.cuh"
#include "kv4.cuh"
#include "kv4_request.cuh"
#include "kv_ops.h"
#include "internal.h"
#include "ptx.cuh"

namespace lora {

namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kGap = 4;             // what a group costs beside its tiles, in tiles (512 requests over 50 to 300: 38.1 us, 39.1 with 2)
constexpr int kMinShare = 2;        // least share of a warp, in tiles (one token over 1000: 11.9 us, 13.4 with 4, 15.9 with 8)
constexpr int kBatch = 2;           // most tiles of a stage of a warp's ring
constexpr float kLift = 7.f;        // m is this far below the largest score where it is set: fp16 has p down to 2^-31 of the largest
constexpr float kSlack = 15.f;      // log2 of the largest p; m is set again past it
constexpr float kNone = -1e30f;     // m of a column that has seen no key

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t transposed(uint32_t v)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// mbar_try_wait without suspending: whether the phase is over now.
__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Bounded wait, with what it does when the barrier is not there yet out of line.  A try may suspend for longer than the
// load that it waits for takes, whatever the budget: short budgets are waited out without.
__device__ __noinline__ bool wait_loop(uint64_t *bar, uint32_t parity, volatile int *abort, int32_t *status, int64_t budget)
{
    const uint32_t at = smem_u32(bar);
    const long long most = wait_budget(abort, budget), t0 = clock64();
    while (!(budget < kWaitShort ? mbar_test_wait(at, parity) : mbar_try_wait(at, parity))) {
        if (clock64() - t0 > most) {
            *abort = 1;
            atomicOr(status, LORA_DEV_TIMEOUT);
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, volatile int *abort, int32_t *status, int64_t budget)
{
    return mbar_test_wait(smem_u32(bar), parity) || wait_loop(bar, parity, abort, status, budget);
}

// a / b; most quotients here fit 32 bits, where a division takes a quarter of the time.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b)
{
    return ((a | b) >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}

// bulk_load of what is read once: the first to leave L2, before the parts of cut groups, tables and queries (32
// requests over 100 to 8000 40.0 us so, 40.9 without; 512 over 50 to 300 38 and 40; 128 over 1000 to 16000 the same).
__device__ __forceinline__ uint64_t read_once_policy()
{
    uint64_t policy;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    return policy;
}
__device__ __forceinline__ void bulk_load_once(void *dst, const void *src, uint32_t bytes, uint64_t *bar, uint64_t policy)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
                 : "memory");
}

// row / group (the token of a row): exact, as row * group < 2^64, and a division takes several times as long.
__device__ __forceinline__ int token_of(const Kv4AttnParams &p, int row)
{
    return p.group == 1 ? row : static_cast<int>(__umul64hi(static_cast<uint64_t>(row), p.group_inverse));
}

// A request without what the attention over a bf16 cache has done (a wide request).
__device__ __forceinline__ Kv4Request request(const Kv4AttnParams &p, int r, int *bad)
{
    Kv4Request q = kv4_request(p, r, bad);
    if (p.wide && p.wide[r]) q.n = 0;
    return q;
}

// A group, as far as its rows and its place among the units go.
struct Group {
    int64_t start;      // its first unit
    int cost;           // its units: kGap and its tiles
    int tok0, h, first_row, cols;   // first token of the request, key head, first row of the block, rows of the block
};

// The pieces of a warp's share, one after another: tiles [t0, t1) of block b of key head
// h of request r.  A request has kv_heads * blocks groups of kGap + tiles units, and a
// warp begins or ends inside one only behind its gap.
template <int NC>
struct Pieces {
    int r, h, b, t0, t1, tiles, blocks;
    Kv4Request q;
    int64_t at, left;   // place in the group, units left from there

    __device__ __forceinline__ void take(const Kv4AttnParams &p)
    {
        int bad = 0;
        q = request(p, r, &bad);
        blocks = (q.n * p.group + NC - 1) / NC;
        tiles = max(1, (q.keys + 15) >> 4);
    }
    // the first piece of a share of `units` that begins at unit u of request r_; false if there is none
    __device__ __forceinline__ bool start(const Kv4AttnParams &p, int r_, int64_t u, int64_t units)
    {
        r = r_;
        take(p);
        const int64_t g = quotient(u, tiles + kGap);
        at = u - g * (tiles + kGap);
        h = static_cast<int>(blocks == 1 ? g : quotient(g, blocks));
        b = static_cast<int>(g - static_cast<int64_t>(h) * blocks);
        left = units;
        return cut();
    }
    __device__ __forceinline__ bool cut()
    {
        if (left <= 0) return false;
        t0 = static_cast<int>(at > kGap ? at - kGap : 0);
        const int64_t end = at + left, cost = tiles + kGap;
        if (end < cost && end <= kGap) {   // not behind the gap: the next warp's
            left = 0;
            return false;
        }
        t1 = end < cost ? static_cast<int>(end) - kGap : tiles;
        left = end - cost;
        return true;
    }
    __device__ __forceinline__ bool next(const Kv4AttnParams &p)
    {
        if (left <= 0) return false;
        at = 0;
        if (++b == blocks) {
            b = 0;
            if (++h == p.kv_heads) {
                h = 0;
                do {
                    if (++r >= p.R) return false;
                    take(p);
                } while (q.n == 0);
            }
        }
        return cut();
    }
    // tiles of the piece that some row of the block sees: [t0, this)
    __device__ __forceinline__ int end(const Kv4AttnParams &p) const
    {
        const int last = min(q.n - 1, token_of(p, b * NC + NC - 1));
        return min(t1, (max(0, q.keys - q.n + last + 1) + 15) >> 4);
    }
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == tiles; }
};

// A warp's last piece takes its ring's place; a first one that others follow goes to
// the workspace.  NT 1: queries in registers, else in shared memory.
template <int DP, int NT>
struct Smem {
    static constexpr int NC = 8 * NT;
    static constexpr int kPad = DP + 4;                                  // floats from a column of results to the next
    static constexpr int kTile = Kv4Tile<DP>::kBytes;
    static constexpr int kSlot = NC * kPad * 4;                          // a piece's results
    static constexpr int kStages = DP == 128 ? 3 : 4;   // of a warp's ring
    static constexpr int kRing = kStages * kBatch * kTile;
    static_assert(kRing >= kSlot, "a warp's last piece takes its ring's place");
    static constexpr int kQ = kWarps * kRing;                            // [kWarps][NT][DP / 16][32] uint2
    static constexpr int kQWarp = NT == 1 ? 0 : NT * (DP / 16) * 32 * 8;
    static constexpr int kMl = kQ + kWarps * kQWarp;                     // [2][kWarps][NC] (m, l): first and last pieces
    static constexpr int kGroups = kMl + 2 * kWarps * NC * 8;            // [2][kWarps] their groups
    static constexpr int kNow = kGroups + 2 * kWarps * static_cast<int>(sizeof(Group));     // [kWarps] Group
    static constexpr int kPieces = kNow + kWarps * static_cast<int>(sizeof(Group));         // [kWarps][2] Pieces
    static constexpr int kBars = kPieces + 2 * kWarps * static_cast<int>(sizeof(Pieces<NC>));   // [kWarps][kStages]
    static constexpr int kMisc = kBars + kWarps * kStages * 8;           // scan, flags
    static constexpr int kTotal = kMisc + 32 * 8 + 32;
};

enum { kHasFirst = 1, kFirstGoesOn = 2, kHasLast = 4, kFirstInRing = 8 };   // a warp's pieces of cut groups

template <int DP, int NT>
__global__ void __launch_bounds__(kThreads, 2) kv4_attn_kernel(const Kv4AttnParams p)
{
    pdl_launch_dependents();
    using S = Smem<DP, NT>;
    using Tile = Kv4Tile<DP>;
    constexpr int NC = S::NC, KB = DP / 16, W = DP / 32;   // W: words of 8 codes of a lane's share of a key
    constexpr int kStages = S::kStages;
    extern __shared__ __align__(128) uint8_t sm[];
    float2 *ml = reinterpret_cast<float2 *>(sm + S::kMl);
    Group *groups = reinterpret_cast<Group *>(sm + S::kGroups);
    int64_t *scan = reinterpret_cast<int64_t *>(sm + S::kMisc);          // [32]
    int64_t *bases = reinterpret_cast<int64_t *>(sm);                    // [kThreads] units before a thread's requests, in place of rings
    volatile int *abort = reinterpret_cast<volatile int *>(scan + 32);
    uint32_t *cuts = reinterpret_cast<uint32_t *>(scan + 32) + 1;        // the warps' pieces of cut groups, 4 bits each
    int *joins = reinterpret_cast<int *>(cuts + 1);                      // [2][3]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    uint8_t *ring = sm + warp * S::kRing;
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + S::kBars) + warp * kStages;
    if (tid == 0) {
        *abort = 0;
        *cuts = 0;
    }
    if (lane == 0)
        for (int i = 0; i < kStages; ++i) mbar_init(full + i, 1);
    fence_mbarrier_init();
    int32_t *status = p.counters;
    pdl_wait();

    if (p.wide_status && blockIdx.x == 0 && tid == 0) {   // what the attention over a bf16 cache has to report
        if (const int32_t bits = *p.wide_status) atomicOr(status, bits);
        *p.wide_status = 0;
    }

    // ---- the warps' shares of all units: every CTA counts them for itself
    const int run = (p.R + kThreads - 1) / kThreads, r0 = min(p.R, tid * run), r1 = min(p.R, r0 + run);
    auto units = [&](int r, int *bad) {
        const Kv4Request q = request(p, r, bad);
        const int64_t blocks = (q.n * p.group + NC - 1) / NC;
        return blocks * p.kv_heads * (kGap + max(1, (q.keys + 15) >> 4));
    };
    int bad = 0;
    int64_t mine = 0, total;
    for (int r = r0; r < r1; ++r) mine += units(r, &bad);
    const int64_t base = block_scan_i64(mine, scan, &total);
    if (bad) atomicOr(status, LORA_DEV_BAD_LENGTH);
    if (total == 0) return;
    const int64_t most = total / kMinShare;   // at least 1: a group has kGap + 1 units, and no share is empty
    const int warps = static_cast<int>(most < gridDim.x * kWarps ? most : gridDim.x * kWarps), cta = blockIdx.x;
    if (cta * kWarps >= warps) return;
    const int64_t quot = quotient(total, warps), rem = total - quot * warps;
    auto share_of = [&](int w) { return w * quot + min(static_cast<int64_t>(w), rem); };        // first unit of warp w
    auto warp_of = [&](int64_t u) {                                                             // whose share has unit u
        const int64_t longer = rem * (quot + 1);
        return static_cast<int>(u < longer ? quotient(u, quot + 1) : rem + quotient(u - longer, quot));
    };
    bases[tid] = base;
    __syncthreads();

    const int me = cta * kWarps + warp;
    const int64_t u0 = share_of(me), u1 = share_of(me + 1);
    Pieces<NC> piece = {};
    bool going = false;
    if (me < warps) {
        // the thread whose requests have the first unit: the last one of a base up to there
        const int j0 = (31 - __clz(__ballot_sync(0xffffffffu, bases[kWarps * lane] <= u0))) * kWarps;
        const int j = j0 + 31 - __clz(__ballot_sync(0xffffffffu, lane < kWarps && bases[j0 + lane % kWarps] <= u0));
        int r = j * run;
        int64_t in = u0 - bases[j];
        if (run > 1)
            for (int64_t n; in >= (n = units(r, &bad)); ++r) in -= n;
        going = piece.start(p, r, in, u1 - u0);
    }
    bool more = going;

    // What only the ends of pieces need stays in shared memory (the loop over tiles has no registers for it): the
    // piece in work with its group, and the one whose tiles are being fetched.
    Pieces<NC> *cur = reinterpret_cast<Pieces<NC> *>(sm + S::kPieces) + 2 * warp, *ahead = cur + 1;
    Group *now = reinterpret_cast<Group *>(sm + S::kNow) + warp;
    if (lane == 0) {
        *cur = *ahead = piece;
        now->start = u0 - piece.at;
        now->cost = 0;
    }
    fence_proxy_async_smem();   // `bases` was written and read as ordinary memory; the ring's copies go there next
    __syncthreads();   // everybody is done with `bases`

    // ---- the warp's ring: tiles [fetch_t, fetch_e) of the piece `ahead`, then of those after it, up to
    // kBatch of a piece a stage.  The lanes have the addresses of 32 tiles from fetch_0 on, and each issues its own.
    int fetch_t = piece.t0, fetch_e = more ? piece.end(p) : fetch_t, fetch_0 = fetch_t - 32;
    int put = 0, flying = 0;   // the stage that is filled next, and stages filled and not used up
    const uint8_t *src = nullptr;
    const uint64_t policy = read_once_policy();
    const int in_page = p.page_shift - 4;   // log2 of the tiles of a page
    auto fetch = [&]() {       // one more stage, if there is anything
        while (fetch_t >= fetch_e) {
            if (!more) return;
            Pieces<NC> x = *ahead;
            more = x.next(p);
            __syncwarp();
            if (lane == 0) *ahead = x;
            __syncwarp();
            if (!more) return;
            fetch_t = x.t0;
            fetch_e = x.end(p);
            fetch_0 = fetch_t - 32;
        }
        if (fetch_t - fetch_0 >= 32) {
            fetch_0 = fetch_t;
            const int t = fetch_t + lane;
            if (t < fetch_e) {
                const int page = p.table[ahead->r * p.table_stride + (t >> in_page)];
                if (page < 0 || page >= p.num_pages) {
                    atomicOr(status, LORA_DEV_BAD_PAGE);
                    src = p.zeros;
                } else {
                    src = p.data + page * p.page_stride + ahead->h * p.head_stride +
                          (t & ((1 << in_page) - 1)) * static_cast<int64_t>(S::kTile);
                }
            }
        }
        static_assert(32 % kBatch == 0, "a stage's addresses are there together");
        const int n = min(kBatch, fetch_e - fetch_t), i = lane - (fetch_t - fetch_0);
        if (i == 0) mbar_expect_tx(full + put, n * S::kTile);
        __syncwarp();
        if (i >= 0 && i < n) bulk_load_once(ring + (put * kBatch + i) * S::kTile, src, S::kTile, full + put, policy);
        put = put + 1 == kStages ? 0 : put + 1;
        ++flying;
        fetch_t += n;
    };
#pragma unroll 1
    for (int i = 0; i < kStages; ++i) fetch();
    int stage = 0, parity = 0;
    bool live = true;   // until a wait gives up

    // a row of the output; by: 1 / l
    auto row_of = [&](const Group &gr, int n, int *h) {
        const int row = gr.first_row + n, i = token_of(p, row);
        *h = gr.h * p.group + row - i * p.group;
        return static_cast<int64_t>(gr.tok0 + i);
    };
    auto store_lse = [&](int64_t t, int h, float m, float l) {
        p.lse[t * p.heads + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    };

#pragma unroll 1
    while (going) {
        piece = *cur;
        Group gr;
        gr.start = now->start + now->cost;   // after the group before
        gr.cost = piece.tiles + kGap;
        gr.tok0 = piece.q.tok0;
        gr.h = piece.h;
        gr.first_row = piece.b * NC;
        gr.cols = min(NC, piece.q.n * p.group - piece.b * NC);
        __syncwarp();
        if (lane == 0) *now = gr;

        // ---- queries: lane (g, c) has elements [c * DP / 4, (c + 1) * DP / 4) of column g, as fp16
        // scaled by a power of two, four at a time in the order of the B operand
        uint2 qf[NT == 1 ? KB : 1];
        uint2 *qs = reinterpret_cast<uint2 *>(sm + S::kQ + warp * S::kQWarp) + lane;
        float fac[NT][2], m[NT][2], l[NT][2], o[NT][KB][4];
        int lim[NT][2];   // keys that a column sees
        if (NT > 1) __syncwarp();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            uint4 x[KB / 2];
            int h;
            const int n = nt * 8 + g;
            const int64_t t = row_of(gr, n, &h);
            const uint16_t *from = p.q + t * p.q_tok + h * p.q_head + c * (DP / 4);
#pragma unroll
            for (int i = 0; i < KB / 2; ++i) {
                x[i] = make_uint4(0, 0, 0, 0);
                if (n < gr.cols && c * (DP / 4) + 8 * i < p.head_dim) x[i] = *reinterpret_cast<const uint4 *>(from + 8 * i);
            }
            uint32_t top = 0;   // the largest magnitude, by its bits
#pragma unroll
            for (int i = 0; i < KB / 2; ++i) {
                const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7FFFu, (w[e] >> 16) & 0x7FFFu));
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // 2^(12 - e) for a largest magnitude in [2^e, 2^(e + 1)); rows of zeros or infinities stay as they are
            const int e = top >> 7;
            const bool as_is = e < 13 || e > 254;
            const float by = as_is ? 1.f : __uint_as_float((266 - e) << 23);
            const float f = p.scale * 1.4426950408889634f * (as_is ? 1.f : __uint_as_float((e - 12) << 23));
#pragma unroll
            for (int i = 0; i < 2; ++i) fac[nt][i] = __shfl_sync(0xffffffffu, f, (2 * c + i) * 4);
#pragma unroll
            for (int i = 0; i < KB; ++i) {
                const uint32_t a = i & 1 ? x[i / 2].z : x[i / 2].x, b = i & 1 ? x[i / 2].w : x[i / 2].y;
                const uint2 v = make_uint2(pack_f16x2(bf16_lo(a) * by, bf16_hi(a) * by), pack_f16x2(bf16_lo(b) * by, bf16_hi(b) * by));
                if (NT == 1) qf[NT == 1 ? i : 0] = v;
                else qs[(nt * KB + i) * 32] = v;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int col = nt * 8 + 2 * c + i;
                lim[nt][i] = col < gr.cols ? max(0, piece.q.keys - piece.q.n + token_of(p, gr.first_row + col) + 1) : 0x7fffffff;
                m[nt][i] = kNone;
                l[nt][i] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < KB; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[nt][j][i] = 0.f;
        }
        if (NT > 1) __syncwarp();
        const int first_limit = max(0, piece.q.keys - piece.q.n + token_of(p, gr.first_row) + 1);   // of the first column, the fewest

        // S^T of a tile: rows are the keys g and g + 8, columns 2c and 2c + 1
        auto scores = [&](const uint8_t *tile, float (&sc)[NT][4]) {
            uint32_t kw[2][W], ks[2][W / 2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint8_t *at = tile + e * (4 * DP) + lane * (4 * W);
                if (W == 4) *reinterpret_cast<uint4 *>(kw[e]) = *reinterpret_cast<const uint4 *>(at);
                else *reinterpret_cast<uint2 *>(kw[e]) = *reinterpret_cast<const uint2 *>(at);
                at = tile + Tile::kKeyScales + (8 * e + g) * Tile::kGroups + c * (W / 2);
#pragma unroll
                for (int i = 0; i < W / 2; ++i) ks[e][i] = at[i] * 0x00800080u;   // the scale as an fp16 pair
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[nt][e] = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) {   // 8 elements of each key, of one scale
                uint32_t f[2][4];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    e2m1x8_to_f16(kw[e][w], f[e]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) f[e][i] = mul_f16x2(f[e][i], ks[e][w / 2]);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t a[4] = {f[0][2 * i], f[1][2 * i], f[0][2 * i + 1], f[1][2 * i + 1]};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const uint2 b = NT == 1 ? qf[NT == 1 ? 2 * w + i : 0] : qs[(nt * KB + 2 * w + i) * 32];
                        mma_f16(sc[nt], a, b.x, b.y);
                    }
                }
            }
        };
        // O^T += V^T P^T: rows are elements of the values, inner dimension the keys 2c, 2c + 1 and 2c + 8, 2c + 9
        auto values = [&](const uint8_t *tile, const uint32_t (&pb)[NT][2], int keys) {
            uint32_t vw[2][W];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint8_t *at = tile + Tile::kValues + e * (4 * DP) + lane * (4 * W);
                if (W == 4) *reinterpret_cast<uint4 *>(vw[e]) = *reinterpret_cast<const uint4 *>(at);
                else *reinterpret_cast<uint2 *>(vw[e]) = *reinterpret_cast<const uint2 *>(at);
            }
            uint32_t vs = *reinterpret_cast<const uint32_t *>(tile + Tile::kValueScales + ((DP == 128 ? g : g / 2) * 4 + c) * 4);
            if (keys < 16) {   // keys past the request: whatever they hold, their scales may be NaN
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (2 * c + (e & 1) + 8 * (e >> 1) >= keys) vs &= ~(0xFFu << (8 * e));
            }
            const uint32_t vs2[2] = {scale_pair<0, 1>(vs), scale_pair<2, 3>(vs)};
#pragma unroll
            for (int w = 0; w < W / 2; ++w) {   // 8 elements of the four keys
                uint32_t f[2][2][4];            // [half of the keys][parity of the element][pair of elements]
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t a = vw[e][2 * w], b = vw[e][2 * w + 1];   // the even and the odd key's codes
                    e2m1x8_to_f16((a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u), f[e][0]);
                    e2m1x8_to_f16(((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u), f[e][1]);
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int i = 0; i < 4; ++i) f[e][q][i] = mul_f16x2(f[e][q][i], vs2[e]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t a[4] = {f[0][0][i], f[0][1][i], f[1][0][i], f[1][1][i]};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_f16(o[nt][4 * w + i], a, pb[nt][0], pb[nt][1]);
                }
            }
        };
        // ---- the tiles
        const int te = piece.end(p), keys = piece.q.keys;
#pragma unroll 1
        for (int t = piece.t0; t < te && live;) {
            live = __all_sync(0xffffffffu, wait(full + stage, parity, abort, status, p.wait_cycles));
            if (!live) break;
            const uint8_t *tile = ring + stage * (kBatch * S::kTile);
            const int t_end = min(t + kBatch, te);
#pragma unroll 1
            for (; t < t_end; ++t, tile += S::kTile) {
                float sc[NT][4];
                scores(tile, sc);
                // x - m, and -infinity for what is not seen
                float y[NT][4];
                auto shift = [&]() {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) y[nt][e] = fmaf(sc[nt][e], fac[nt][e & 1], -m[nt][e & 1]);
                    if (t * 16 + 16 > first_limit) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (t * 16 + g + 8 * (e >> 1) >= lim[nt][e & 1]) y[nt][e] = -INFINITY;
                    }
                };
                shift();
                float rise = kNone;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) rise = fmaxf(fmaxf(rise, fmaxf(y[nt][0], y[nt][1])), fmaxf(y[nt][2], y[nt][3]));
                if (__any_sync(0xffffffffu, rise > kSlack)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float top = m[nt][e];
#pragma unroll
                            for (int q = 0; q < 4; q += 2)
                                if (y[nt][e + q] != -INFINITY) top = fmaxf(top, fmaf(sc[nt][e + q], fac[nt][e], -kLift));
#pragma unroll
                            for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                            const float by = exp2_approx(m[nt][e] - top);
                            m[nt][e] = top;
                            l[nt][e] *= by;
#pragma unroll
                            for (int j = 0; j < KB; ++j) {
                                o[nt][j][e] *= by;
                                o[nt][j][e + 2] *= by;
                            }
                        }
                    shift();
                }
                uint32_t pb[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float x[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[e] = exp2_approx(y[nt][e]);
                        l[nt][e & 1] += x[e];   // before the rounding to fp16
                    }
                    pb[nt][0] = transposed(pack_f16x2(x[0], x[1]));
                    pb[nt][1] = transposed(pack_f16x2(x[2], x[3]));
                }
                values(tile, pb, keys - t * 16);
            }
            __syncwarp();   // every lane is done with the stage
            --flying;
            fetch();
            parity = stage + 1 == kStages ? parity ^ 1 : parity;
            stage = stage + 1 == kStages ? 0 : stage + 1;
        }

        // ---- results
        __syncwarp();
        piece = *cur;
        gr = *now;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], d);
        // a lane's elements of a column are consecutive: d = g * DP / 8 + 2j, + 1
        if (piece.whole()) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int n = nt * 8 + 2 * c + e;
                    if (n >= gr.cols) continue;
                    int h;
                    const int64_t t = row_of(gr, n, &h);
                    const float by = l[nt][e] != 0.f ? 1.f / l[nt][e] : 0.f;   // no key: zeros
                    uint16_t *to = p.o + t * p.o_tok + h * p.o_head + g * (DP / 8);
                    uint32_t v[KB];
#pragma unroll
                    for (int j = 0; j < KB; ++j) v[j] = pack_bf16x2(o[nt][j][e] * by, o[nt][j][e + 2] * by);
#pragma unroll
                    for (int j = 0; j < KB; j += 4)
                        if (g * (DP / 8) + 2 * j < p.head_dim)
                            *reinterpret_cast<uint4 *>(to + 2 * j) = make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                    if (g == 0 && p.lse) store_lse(t, h, m[nt][e], l[nt][e]);
                }
        } else {
            const int last = piece.t0 == 0;   // begins here and goes on elsewhere; else it comes from elsewhere
            const bool in_ring = last || piece.left <= 0;   // nothing after it
            float *to = in_ring ? reinterpret_cast<float *>(ring) : p.first + static_cast<int64_t>(me) * NC * S::kPad;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int n = nt * 8 + 2 * c + e;
                    float4 *v = reinterpret_cast<float4 *>(to + n * S::kPad + g * (DP / 8));
#pragma unroll
                    for (int j = 0; j < KB / 2; ++j)
                        v[j] = make_float4(o[nt][2 * j][e], o[nt][2 * j][e + 2], o[nt][2 * j + 1][e], o[nt][2 * j + 1][e + 2]);
                    if (g == 0) ml[(last * kWarps + warp) * NC + n] = make_float2(m[nt][e], l[nt][e]);
                }
            if (lane == 0) {
                groups[last * kWarps + warp] = gr;
                const uint32_t mark = last ? kHasLast
                                           : kHasFirst | (piece.t1 < piece.tiles ? kFirstGoesOn : 0) | (in_ring ? kFirstInRing : 0);
                atomicOr(cuts, mark << (4 * warp));
            }
        }
        going = piece.next(p);
        __syncwarp();
        if (lane == 0) *cur = piece;
        __syncwarp();
    }
    // after a timeout: nothing may be in flight when the CTA ends
    for (; flying > 0; --flying) {
        wait_loop(full + stage, parity, abort, status, p.wait_cycles < kWaitShort ? kWaitShort : p.wait_cycles);
        parity = stage + 1 == kStages ? parity ^ 1 : parity;
        stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    __syncthreads();

    // ---- cut groups.  A chain of pieces: the last of a warp (or, at the CTA's start, one that
    // comes from the CTA before), then the first of the warps after it as long as they go on.
    auto store = [&](const Group &gr, int n, int d, float4 v, float top, float sum) {
        int h;
        const int64_t t = row_of(gr, n, &h);
        const float by = sum != 0.f ? 1.f / sum : 0.f;   // no key: zeros
        if (d < p.head_dim)
            *reinterpret_cast<uint2 *>(p.o + t * p.o_tok + h * p.o_head + d) =
                make_uint2(pack_bf16x2(v.x * by, v.y * by), pack_bf16x2(v.z * by, v.w * by));
        if (d == 0 && p.lse) store_lse(t, h, top, sum);
    };
    auto add = [](float4 &v, float &sum, float top, float4 y, float2 x) {
        const float by = exp2_approx(x.x - top);
        sum += x.y * by;
        v.x += y.x * by;
        v.y += y.y * by;
        v.z += y.z * by;
        v.w += y.w * by;
    };
    const uint32_t marks = *cuts;
    // bit 4 + 4w for a chain that begins with warp w's last piece, bit 0 for one with warp 0's first
    const uint64_t begins = (static_cast<uint64_t>(marks / kHasLast & 0x11111111u) << 4) | (marks & kHasFirst);
    const int chains = __popcll(begins);
    // The chains side by side, some warps each: a chain is a few dependent loads, and there may be nine.
    const int each = chains > 4 ? 1 : chains > 2 ? 2 : chains > 1 ? 4 : 8;   // warps of a chain
    int shared_groups = 0, tail = 0;   // bit 0: with the CTA before, bit 1: with the CTA after, by this warp's last piece
    int k = 0;
    for (uint64_t left = begins; left; left &= left - 1, ++k) {
        const int w = (__ffsll(left) - 1) / 4 - 1;
        int to = w;   // last warp of the chain
        bool goes_on = true;
        while (goes_on && to + 1 < kWarps) goes_on = marks >> (4 * ++to) & kFirstGoesOn;
        const bool whole = w >= 0 && !goes_on;
        if (!whole) shared_groups |= w < 0 ? 1 : 2;
        if (w >= 0) tail = kWarps + w;
        if (k % (kWarps / each) != warp / each) continue;
        const Group gr = groups[w < 0 ? 0 : kWarps + w];
        const int64_t part = 2 * cta + (w >= 0);
        constexpr int kAtOnce = 4;   // elements of four of a thread
#pragma unroll 1
        for (int u0 = tid % (32 * each); u0 < gr.cols * (DP / 4); u0 += kAtOnce * 32 * each) {
            float top[kAtOnce], sum[kAtOnce];
            float4 v[kAtOnce];
            int n[kAtOnce], d[kAtOnce];
#pragma unroll
            for (int q = 0; q < kAtOnce; ++q) {
                const int u = min(u0 + q * 32 * each, gr.cols * (DP / 4) - 1);   // past the end: the last one again
                n[q] = u / (DP / 4);
                d[q] = u % (DP / 4) * 4;
                top[q] = w >= 0 ? ml[(kWarps + w) * NC + n[q]].x : kNone;
                sum[q] = 0.f;
                v[q] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
            // the largest m first: then the pieces' factors do not wait for one another
            for (int i = w + 1; i <= to; ++i)
#pragma unroll
                for (int q = 0; q < kAtOnce; ++q) top[q] = fmaxf(top[q], ml[i * NC + n[q]].x);
#pragma unroll 4
            for (int i = w; i <= to; ++i) {
                if (i < 0) continue;
                const bool last = i == w;   // the chain's first piece is its warp's last
                const float *from = last || marks >> (4 * i) & kFirstInRing
                                        ? reinterpret_cast<const float *>(sm + i * S::kRing)
                                        : p.first + static_cast<int64_t>(cta * kWarps + i) * NC * S::kPad;
                float4 y[kAtOnce];
#pragma unroll
                for (int q = 0; q < kAtOnce; ++q) y[q] = *reinterpret_cast<const float4 *>(from + n[q] * S::kPad + d[q]);
#pragma unroll
                for (int q = 0; q < kAtOnce; ++q) add(v[q], sum[q], top[q], y[q], ml[(last * kWarps + i) * NC + n[q]]);
            }
#pragma unroll
            for (int q = 0; q < kAtOnce; ++q) {
                if (u0 + q * 32 * each >= gr.cols * (DP / 4)) continue;
                if (whole) {
                    store(gr, n[q], d[q], v[q], top[q], sum[q]);
                } else {
                    *reinterpret_cast<float4 *>(p.part + (part * NC + n[q]) * DP + d[q]) = v[q];
                    if (d[q] == 0) p.part_ml[part * NC + n[q]] = make_float2(top[q], sum[q]);
                }
            }
        }
    }
    if (!shared_groups) return;
    // the CTA that stores the last part of a group joins them, in their order (the barrier
    // and the release behind it put every thread's part before the count)
    __syncthreads();
    if (tid < 2 && (shared_groups >> tid & 1)) {
        const Group &gr = groups[tid == 0 ? 0 : tail];
        const int c0 = warp_of(gr.start + kGap) / kWarps, c1 = warp_of(gr.start + gr.cost - 1) / kWarps;
        const int n = atom_acq_rel_gpu_add(p.counters + kKv4CntGroup + c0, 1);
        joins[3 * tid] = n == c1 - c0;
        joins[3 * tid + 1] = c0;
        joins[3 * tid + 2] = c1;
        if (n == c1 - c0) p.counters[kKv4CntGroup + c0] = 0;
    }
    __syncthreads();
    // two groups side by side, half of the CTA each
    const bool join0 = (shared_groups & 1) && joins[0], join1 = (shared_groups & 2) && joins[3];
    if (!join0 && !join1) return;
    const bool halves = join0 && join1;
    const int which = halves ? warp >= kWarps / 2 : join1, threads = halves ? kThreads / 2 : kThreads;
    const Group gr = groups[which == 0 ? 0 : tail];
    const int c0 = joins[3 * which + 1], c1 = joins[3 * which + 2];
#pragma unroll 1
    for (int u = tid % threads; u < gr.cols * (DP / 4); u += threads) {
        const int n = u / (DP / 4), d = u % (DP / 4) * 4;
        float top = kNone, sum = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        // (a first pass for the largest m would cost a second round trip to L2)
#pragma unroll 4
        for (int i = c0; i <= c1; ++i) {
            const int64_t part = 2 * i + (i == c0);
            const float4 y = __ldcg(reinterpret_cast<const float4 *>(p.part + (part * NC + n) * DP + d));
            const float2 x = __ldcg(p.part_ml + part * NC + n);
            const float next = fmaxf(top, x.x), by = exp2_approx(top - next);
            sum *= by;
            v = make_float4(v.x * by, v.y * by, v.z * by, v.w * by);
            top = next;
            add(v, sum, top, y, x);
        }
        store(gr, n, d, v, top, sum);
    }
}

template <int DP, int NT>
cudaError_t launch_variant(const Kv4AttnParams &p, cudaStream_t stream)
{
    using S = Smem<DP, NT>;
    constexpr int smem = S::kTotal;
    static_assert(2 * (smem + 1024) <= 228 * 1024, "two CTAs an SM");
    static int configured[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
    if (dev >= 64 || !configured[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(kv4_attn_kernel<DP, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        if (dev < 64) configured[dev] = 1;
    }
    int64_t ctas = 2 * static_cast<int64_t>(num_sms_current_device());
    ctas = ctas < kKv4MaxCtas ? ctas : kKv4MaxCtas;
    return launch_pdl(kv4_attn_kernel<DP, NT>, ctas, kThreads, smem, p, stream);
}

}  // namespace

// Blocks of 8 columns for heads of more than 64: a request of more rows has several, which read its tiles again (from
// L2) and unpack them again.  The registers of 16 columns cost the second CTA of an SM (with both, they
// spill and every case is slower), and which is faster depends on the rows:
//                                                             8 columns   16
//   32 requests of one token, 32/8 heads, over 100 to 8000       40 us     54
//   48 of up to 5 tokens, 28/4 heads, over 300 to 6000           52        56
//   64 over 1000 to 8000, 16 rows: one token, 32/2 heads         39        37
//                                  2 tokens, 32/4 heads          65        58
//                                  4 tokens, 32/8 heads         113        98
//   8 of 16 tokens, 32/8 heads, over 1000 to 8000                68        60
// So 8 throughout gives up 6 to 14 % from 16 rows on, for one kernel less.  Heads up to 64 have the registers for
// both, and take 16 where requests have more than 8 rows: 8 requests of 64 rows over 1000 to 8000 45 us with 8, 35 with 16.
cudaError_t launch_kv4_attn(const Kv4AttnParams &p, cudaStream_t stream)
{
    if (p.head_dim > 64) return launch_variant<128, 1>(p, stream);
    return static_cast<int64_t>(p.T) * p.group <= 8 * static_cast<int64_t>(p.R) ? launch_variant<64, 1>(p, stream)
                                                                              : launch_variant<64, 2>(p, stream);
}

}  // namespace lora
