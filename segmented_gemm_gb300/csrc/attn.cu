// Attention over packed rows or a paged cache (include/lora_attn.h):
//   o_i = sum_j p_ij v_j / l_i,   p_ij = 2^(c q_i.k_j - c m_i),   l_i = sum_j p_ij,   c = scale log2(e)
// over the keys j that row i sees, m_i a running maximum of the scores.
//
// A query tile is 128 rows: tq tokens times the group's query heads, which
// share the key/value head, so a key tile is loaded once for the group.  A
// CTA works on two score streams at once, so that one's softmax runs under the
// other's matrix products:
//   pair     two query tiles against the same key tiles (long chunks, prompts)
//   single   one query tile, the key tiles dealt to the streams in turn
//            (decode and short chunks, where the cache's bytes bound the call)
// Per stream and key tile of 128 keys, all on the tensor cores:
//   S = Q K^T   both from shared memory, S [128 x 128] fp32 in tensor memory
//   softmax     a thread per row: S to registers, p = 2^(..), P as bf16 back
//               over S's cells (half of them)
//   O += P V    P from tensor memory, V from shared memory as it was loaded
//               (its head dimension contiguous: an N-major operand)
// O stays in tensor memory.  m_i moves only when the maximum has grown by more
// than 2^8 in p (so p <= 256, well inside fp32 and bf16): O is rescaled then,
// by the softmax threads themselves, and the division by l_i at the end makes
// any m_i as good as the true maximum.
//
// Roles (384 threads): warps 0..3 and 4..7 the softmax and the results of
// stream 0 and 1, warp 8 takes the work and loads keys (TMA), 9 issues the
// matrix products, 10 loads values, 11 queries.  Three loaders, because a tile
// of small pages is many TMA boxes, and because a new piece's queries must not
// wait behind its tiles.
// Shared memory: two query tiles and a ring of key and value tiles.
// Persistent, one CTA per SM; work comes from the schedule (attn_schedule.cu).
// A group (block, kv head) cut into pieces leaves partial (O, m, l) in the
// workspace; the piece that finishes last joins them in their order, so
// results do not depend on timing.  Every wait is bounded.
#include <cuda_runtime.h>

#include "attn.h"
#include "attn_ptx.cuh"
#include "internal.h"

namespace lora {

constexpr int kAttnThreads = 384;
// registers a thread: 168 at launch; a softmax thread holds a row's 128 scores
constexpr int kSoftmaxRegs = 224, kOtherRegs = 56;
static_assert(2 * kSoftmaxRegs + kOtherRegs <= 3 * 168, "the split draws on the launch's registers");
constexpr int kItems = 4;             // work items in flight between the loader and the others
constexpr float kRescaleBits = 8.f;   // m_i may lag the maximum by this many powers of two

// tensor memory columns (512 in all): S of stream s at s * 128 (P over its
// first 64), O of stream s at 256 + s * DP
constexpr uint32_t kColS = 128, kColO = 256;

// a piece of one (block, kv head): key tiles [t0, t1)
struct AttnItem {
    int32_t valid, pair, req, tok0, ntok, qpos0, kv_len, kvh;
    int32_t seen;     // keys that any of its rows sees
    int32_t t0, t1;
    int32_t end0;     // pair: tiles that stream 0's rows reach
    int32_t parts;    // pieces of the group
    int32_t slot;     // this piece's partial results (parts > 1)
    int32_t unit0;    // the unit that the group starts in (its counter; parts > 1)
};

template <int DP>
struct AttnSmem {
    static constexpr int kHalves = DP / 64;                    // 128-byte column blocks of a tile
    static constexpr int kTile = 128 * DP * 2;                 // bytes of a query, key or value tile
    static constexpr int kStages = 5 * 128 / DP + (DP == 64 ? 2 : 0);
    static constexpr int kStats = 2 * kTile + kStages * kTile; // offsets
    static constexpr int kItem = kStats + 128 * 8;
    static constexpr int kBars = kItem + kItems * static_cast<int>(sizeof(AttnItem));
    static constexpr int kNumBars = 2 * kStages + 2 * kItems + 2 + 1 + 2 + 2 + 2 + 2;
    static constexpr int kEnd = kBars + kNumBars * 8 + 4 * (3 + kStages + 2);
    static constexpr int kBytes = kEnd + 1024;                 // room to align the base
    static_assert(kBytes <= 232448, "fits the opt-in shared memory of a CTA");
};

// Each lane holds 64 bytes (four 16-byte chunks) of its own row at byte `at`;
// four lanes exchange theirs so that a store instruction writes 64 bytes of
// each of eight rows instead of 16 bytes of thirty-two.  dst: the lane's row,
// or 0; bytes: the row's length.
__device__ __forceinline__ void store_rows(uint32_t (&v)[16], uint64_t dst, int at, int bytes, int lane)
{
#pragma unroll
    for (int step = 1; step <= 2; step <<= 1) {
        const bool hi = lane & step;
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            if (a & step) continue;
            const int b = a | step;   // chunks a and b change places with the other lane's
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const uint32_t t = __shfl_xor_sync(0xffffffffu, hi ? v[4 * a + w] : v[4 * b + w], step);
                if (hi) v[4 * a + w] = t;
                else v[4 * b + w] = t;
            }
        }
    }
    const int col = at + (lane & 3) * 16;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint64_t row = __shfl_sync(0xffffffffu, dst, (lane & ~3) | k);
        if (row != 0 && col < bytes)
            *reinterpret_cast<uint4 *>(row + col) = make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
    }
}

// A piece's 2 n loads, in the order in which the products need them:
//   pair    K0 V0 K1 V1 ...
//   single  K0 K1 V0 K2 V1 K3 ... V(n-2) V(n-1)   (n = 1: K0 V0)
__device__ __forceinline__ uint32_t load_of_key(int pair, int t) { return pair ? 2 * t : t < 2 ? t : 2 * t - 1; }
__device__ __forceinline__ uint32_t load_of_value(int pair, int t, int n) { return pair ? 2 * t + 1 : min(2 * t + 2, n + t); }

struct AttnMaps {
    CUtensorMap q, q1, k, v;   // q: tq tokens of a group's heads; q1: one token's
};

template <int DP, bool kPaged>
__global__ void __launch_bounds__(kAttnThreads, 1)
    attn_kernel(const __grid_constant__ AttnMaps maps, const __grid_constant__ AttnParams p)
{
    using Sm = AttnSmem<DP>;
    constexpr int kStages = Sm::kStages, kTile = Sm::kTile, kHalves = Sm::kHalves;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *qbuf = smem, *ring = smem + 2 * kTile;
    float2 *stats = reinterpret_cast<float2 *>(smem + Sm::kStats);   // stream 1's (m, l), single items
    AttnItem *items = reinterpret_cast<AttnItem *>(smem + Sm::kItem);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + Sm::kBars), *empty = full + kStages;
    uint64_t *item_full = empty + kStages, *item_empty = item_full + kItems;
    uint64_t *q_full = item_empty + kItems;   // [2]
    uint64_t *q_empty = q_full + 2;
    uint64_t *s_full = q_empty + 1;           // [2]
    uint64_t *p_full = s_full + 2;            // [2]
    uint64_t *o_full = p_full + 2;            // [2]
    uint64_t *xbar = o_full + 2;              // the 256 softmax threads meet here
    uint64_t *end_bar = xbar + 1;             // after a wait gave up: the matrix products issued so far
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(end_bar + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *join_flag = reinterpret_cast<int *>(tmem_slot + 2);
    int *drain = join_flag + 1;               // loads issued into each ring stage and query buffer

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int32_t *status = p.counters + CNT_STATUS;
    const long long budget = p.wait_cycles;
    // called by whole warps; the answer is the same for all lanes, so a wait
    // that gives up takes its warp out together
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        const bool ok = mbar_wait(bar, parity, abort_flag, status, LORA_DEV_TIMEOUT, budget);
        return __all_sync(0xffffffffu, ok) != 0;
    };
    pdl_launch_dependents();

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&item_full[i], 1);
            mbar_init(&item_empty[i], 11);   // 8 softmax warps, the MMA warp, the value and query loaders
        }
        mbar_init(&q_full[0], 1);
        mbar_init(&q_full[1], 1);
        mbar_init(q_empty, 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&s_full[s], 1);
            mbar_init(&p_full[s], 4);
            mbar_init(&o_full[s], 1);
        }
        mbar_init(xbar, 8);
        mbar_init(end_bar, 1);
        *abort_flag = 0;
        for (int s = 0; s < kStages + 2; ++s) drain[s] = 0;
        fence_mbarrier_init();
    }
    if (warp == 8 && lane == 0) {
        tma_prefetch_map(&maps.q);
        tma_prefetch_map(&maps.q1);
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
    pdl_wait();
    const AttnHdr hdr = *p.hdr;

    // A tile of 128 keys in boxes of box_rows keys (a page, or 128 keys of a
    // larger one; 32 packed rows), each 64 columns wide: one lane per box.
    const int box = p.box_rows, box_shift = __ffs(box) - 1, per_tile = kAttnTileK >> box_shift;
    const int mybox = lane / kHalves, myhalf = lane % kHalves;
    // paged: lane l holds the page of box l % per_tile of tile l / per_tile of a
    // window of 32 / per_tile tiles; the next window's pages are on their way
    // while a window is used
    const int win_shift = box_shift - 2;   // log2 of the window's tiles: 32 * box / 128
    auto pages_of = [&](int req, int tile0, int win, int seen) {
        const int64_t key = (static_cast<int64_t>(tile0 + (win << win_shift)) << 7) + (static_cast<int64_t>(lane) << box_shift);
        const int64_t col = key >> p.page_shift;
        return kPaged && key < seen && col < p.table_width ? p.block_table[req * p.table_stride + col] : -1;
    };
    // load i of the CTA's ring <- tile t of the piece; false after a wait gave up
    auto load_tile = [&](const CUtensorMap *map, uint32_t i, int tile, int page, int seen, int kvh, int row0) {
        const int boxes = (max(0, min(kAttnTileK, seen - tile * kAttnTileK)) + box - 1) >> box_shift;
        const uint32_t s = i % kStages;
        if (i >= kStages && !wait(&empty[s], (i / kStages - 1) & 1)) return false;
        if (lane == 0) {
            drain[s] = static_cast<int>(i / kStages) + 1;
            mbar_expect_tx(&full[s], boxes * box * 128 * kHalves);
        }
        __syncwarp();
        if (mybox < boxes) {
            uint8_t *dst = ring + s * kTile + myhalf * (kAttnTileK * 128) + mybox * box * 128;
            const int key = tile * kAttnTileK + mybox * box;
            if (kPaged) {
                if (page < 0 || page >= p.num_pages) {
                    atomicOr(status, LORA_DEV_BAD_PAGE);
                    page = p.num_pages;   // outside the map: reads as zeros
                }
                tma_load_4d(dst, map, &full[s], myhalf * 64, key & ((1 << p.page_shift) - 1), kvh, page);
            } else {
                tma_load_3d(dst, map, &full[s], myhalf * 64, kvh, row0 + key);
            }
        }
        return true;
    };

    if (warp == 8) {
        // ===================== work and keys ==================================
        setmaxnreg_dec<kOtherRegs>();
        uint32_t it = 0, nitem = 0;
        const bool cut = hdr.cut != 0;
        int64_t unit = blockIdx.x;
        // cut: my unit's tiles [pos, end) of the list; lo: the block that pos is in
        int64_t pos = unit * hdr.unit_tiles;
        const int64_t end = min(pos + hdr.unit_tiles, hdr.tiles);
        int lo = 0, kvh = 0;
        AttnBlock b;
        bool ok = true;
        if (cut && unit < hdr.units) {
            // the last block whose tiles start at or before pos
            int hi = hdr.nblocks;
            while (hi - lo > 1) {
                const int step = (hi - lo + 31) / 32;
                const int at = lo + step * lane;
                const bool le = at < hi && p.blocks[at].pre * p.kv_heads <= pos;
                const int k = 31 - __clz(__ballot_sync(0xffffffffu, le));   // lanes 0..k, lane 0 always
                lo += step * k;
                hi = min(hi, lo + step);
            }
            b = p.blocks[lo];
            kvh = static_cast<int>((pos - b.pre * p.kv_heads) / b.tiles);
        }
        while (ok && unit < hdr.units) {
            // the next piece: key tiles [t0, t1) of (block b, head kvh)
            int t0 = 0, t1, parts = 1, slot = 0, unit0 = 0;
            if (!cut) {
                // whole groups, longest first; the heads of a section together
                const int64_t per = static_cast<int64_t>(hdr.nblocks) * hdr.sec_heads;
                const int sec = static_cast<int>(unit / per);
                const int64_t rem = unit - sec * per;
                const int hs = min(hdr.sec_heads, p.kv_heads - sec * hdr.sec_heads);
                b = p.blocks[p.order[rem / hs]];
                kvh = sec * hdr.sec_heads + static_cast<int>(rem % hs);
                t1 = b.tiles;
            } else {
                if (pos >= end) break;
                const int64_t g0 = b.pre * p.kv_heads + static_cast<int64_t>(kvh) * b.tiles;
                t0 = static_cast<int>(pos - g0);
                t1 = static_cast<int>(min(static_cast<int64_t>(b.tiles), t0 + (end - pos)));
                const int64_t u0 = g0 / hdr.unit_tiles, u1 = (g0 + b.tiles - 1) / hdr.unit_tiles;
                parts = static_cast<int>(u1 - u0 + 1);
                slot = static_cast<int>(unit == u0 ? 2 * unit + 1 : 2 * unit);
                unit0 = static_cast<int>(u0);
            }
            const int seen = min(b.kv_len, b.qpos0 + b.ntok);   // keys past this no row sees
            // hand it to the other roles, then load its keys
            const int is = nitem % kItems;
            if (nitem >= kItems && !wait(&item_empty[is], (nitem / kItems - 1) & 1)) break;
            if (lane == 0) {
                AttnItem &w = items[is];
                w.valid = 1;
                w.pair = b.ntok > p.tq;
                w.req = b.req;
                w.tok0 = b.tok0;
                w.ntok = b.ntok;
                w.qpos0 = b.qpos0;
                w.kv_len = b.kv_len;
                w.seen = seen;
                w.kvh = kvh;
                w.t0 = t0;
                w.t1 = t1;
                w.end0 = max(1, (min(b.kv_len, b.qpos0 + min(b.ntok, p.tq)) + kAttnTileK - 1) / kAttnTileK);
                w.parts = parts;
                w.slot = slot;
                w.unit0 = unit0;
                mbar_arrive(&item_full[is]);
            }
            ++nitem;
            const int n = t1 - t0, pair = b.ntok > p.tq;
            int cur = pages_of(b.req, t0, 0, seen), nxt = pages_of(b.req, t0, 1, seen);
            int next = 0;
            for (int t = 0; t < n && ok; ++t) {
                if (kPaged && t > 0 && (t & ((1 << win_shift) - 1)) == 0) {
                    cur = nxt;
                    nxt = pages_of(b.req, t0, (t >> win_shift) + 1, seen);
                }
                const int page = kPaged ? __shfl_sync(0xffffffffu, cur, (t & ((1 << win_shift) - 1)) * per_tile + mybox) : 0;
                // the next unit is claimed under the wait for the last tile's stage
                if (!cut && t == n - 1 && lane == 0) next = atomicAdd(p.counters + ACNT_NEXT, 1);
                ok = load_tile(&maps.k, it + load_of_key(pair, t), t0 + t, page, seen, kvh, b.tok0 - b.qpos0);
            }
            it += 2 * n;
            if (!cut) {
                unit = static_cast<int64_t>(gridDim.x) + __shfl_sync(0xffffffffu, next, 0);
            } else {
                pos += n;
                if (++kvh == p.kv_heads) {
                    kvh = 0;
                    if (++lo < hdr.nblocks) b = p.blocks[lo];
                }
            }
        }
        const int is = nitem % kItems;
        if (nitem >= kItems) wait(&item_empty[is], (nitem / kItems - 1) & 1);
        if (lane == 0) {
            items[is].valid = 0;
            mbar_arrive(&item_full[is]);
        }
    } else if (warp >= 10) {
        // ===================== values (10), queries (11) ======================
        setmaxnreg_dec<kOtherRegs>();
        uint32_t it = 0, nitem = 0;
        bool ok = true;
        while (ok) {
            const int is = nitem % kItems;
            if (!wait(&item_full[is], (nitem / kItems) & 1)) break;
            const AttnItem w = items[is];
            __syncwarp();
            if (lane == 0) mbar_arrive(&item_empty[is]);
            ++nitem;
            if (!w.valid) break;
            if (warp == 10) {
                const int n = w.t1 - w.t0;
                int cur = pages_of(w.req, w.t0, 0, w.seen), nxt = pages_of(w.req, w.t0, 1, w.seen);
                for (int t = 0; t < n && ok; ++t) {
                    if (kPaged && t > 0 && (t & ((1 << win_shift) - 1)) == 0) {
                        cur = nxt;
                        nxt = pages_of(w.req, w.t0, (t >> win_shift) + 1, w.seen);
                    }
                    const int page =
                        kPaged ? __shfl_sync(0xffffffffu, cur, (t & ((1 << win_shift) - 1)) * per_tile + mybox) : 0;
                    ok = load_tile(&maps.v, it + load_of_value(w.pair, t, n), w.t0 + t, page, w.seen, w.kvh,
                                   w.tok0 - w.qpos0);
                }
                it += 2 * n;
            } else {
                // the previous piece's products have read its queries
                if (nitem > 1 && !wait(q_empty, (nitem - 2) & 1)) break;
                const int g = p.group;
                constexpr int kFew = 4;
                for (int s = 0; s < (w.pair ? 2 : 1); ++s) {
                    const int first = s * p.tq, ntok = min(p.tq, w.ntok - first);
                    uint8_t *dst = qbuf + s * kTile;
                    const bool few = ntok <= kFew;   // single tokens: their rows only, not the whole tile's
                    if (lane == 0) {
                        ++drain[kStages + s];
                        mbar_expect_tx(&q_full[s], (few ? ntok : p.tq) * g * 128 * kHalves);
                    }
                    __syncwarp();
                    if (mybox < (few ? ntok : 1))
                        tma_load_3d(dst + myhalf * (kAttnTileQ * 128) + mybox * g * 128, few ? &maps.q1 : &maps.q,
                                    &q_full[s], myhalf * 64, w.kvh * g, w.tok0 + first + mybox);
                }
            }
        }
    } else if (warp == 9) {
        setmaxnreg_dec<kOtherRegs>();
        // ===================== MMA issuer =====================================
        // All lanes run the same code and the elected one's instructions take
        // effect, and whole tiles' steps are unrolled: a product executes in 64
        // cycles, and issuing one this way takes 35 (66 with a branch around it).
        uint32_t it = 0, nitem = 0, nq0 = 0, nq1 = 0, np0 = 0, np1 = 0;
        const uint32_t qlo = umma_lo(smem_u32(qbuf), 16);
        const uint32_t klo = umma_lo(smem_u32(ring), 16), vlo = umma_lo(smem_u32(ring), kAttnTileK * 128);
        const int dsteps = (p.head_dim + 15) / 16;
        const uint32_t idesc_pv = umma_idesc_bf16_bn(kAttnTileQ, dsteps * 16);
        bool ok = true;
        while (true) {
            const int is = nitem % kItems;
            if (!wait(&item_full[is], (nitem / kItems) & 1)) break;
            const AttnItem &wi = items[is];
            const int valid = uniform(wi.valid), pair = uniform(wi.pair), t0 = uniform(wi.t0);
            const int n = uniform(wi.t1) - t0;
            const int seen = uniform(wi.seen) - t0 * kAttnTileK;   // keys that any row sees
            const int n0 = max(0, min(n, uniform(wi.end0) - t0));   // pair: stream 0's tiles
            __syncwarp();
            if (lane == 0) mbar_arrive(&item_empty[is]);
            ++nitem;
            if (!valid) break;
            // one more product step of a stream: the load i holds its tile, t counts from the piece's first
            auto stage_of = [&](uint32_t i) { return (it + i) % kStages; };
            auto wait_stage = [&](uint32_t i) {
                ok &= wait(&full[stage_of(i)], ((it + i) / kStages) & 1);
                tc_fence_after();
            };
            auto commit = [&](uint64_t *bar) { umma_commit_if(elect_one(), bar); };
            auto release = [&](uint32_t i) { commit(&empty[stage_of(i)]); };
            auto qk = [&](int s, int slot, uint32_t i, int t) {
                const int keys = min(kAttnTileK, seen - t * kAttnTileK);
                const uint32_t idesc = umma_idesc_bf16(kAttnTileQ, max(16, (keys + 15) & ~15));
                const uint32_t qd = qlo + ((slot * kTile) >> 4), kd = klo + stage_of(i) * (kTile >> 4);
                const uint32_t lead = elect_one(), d = tmem + s * kColS;
                auto step = [&](int kk) {
                    const uint32_t o = (kk >> 2) * ((kAttnTileK * 128) >> 4) + (kk & 3) * 2;
                    umma_ss_if(lead, d, qd + o, kd + o, idesc, kk > 0);
                };
                if (dsteps == DP / 16) {
#pragma unroll
                    for (int kk = 0; kk < DP / 16; ++kk) step(kk);
                } else {
#pragma unroll 1
                    for (int kk = 0; kk < dsteps; ++kk) step(kk);
                }
                commit(&s_full[s]);
            };
            auto pv = [&](int s, uint32_t i, int t, uint32_t acc) {
                const int keys = max(0, min(kAttnTileK, seen - t * kAttnTileK));
                const uint32_t vd = vlo + stage_of(i) * (kTile >> 4), a = tmem + s * kColS, d = tmem + kColO + s * DP;
                ok &= wait(&p_full[s], (s ? np1++ : np0++) & 1);
                tc_fence_after();
                const uint32_t lead = elect_one();
                auto step = [&](int kk) {
                    umma_ts_if(lead, d, a + kk * 8, vd + kk * (2048 >> 4), idesc_pv, kk > 0 ? 1 : acc);
                };
                if (keys == kAttnTileK) {
#pragma unroll
                    for (int kk = 0; kk < kAttnTileK / 16; ++kk) step(kk);
                } else {
#pragma unroll 1
                    for (int kk = 0; kk * 16 < keys; ++kk) step(kk);
                }
            };
            // keys past the last one that a row sees: their p is 0, but 0 times what the
            // tile holds there (another request's rows, stale pages) may be NaN
            auto clean = [&](uint32_t i, int t) {
                const int keys = seen - t * kAttnTileK, up = (keys + 15) & ~15;
                if (keys >= kAttnTileK || keys <= 0 || keys == up) return;
                uint8_t *v = ring + stage_of(i) * kTile;
                for (int e = lane; e < (up - keys) * 8 * kHalves; e += 32) {
                    const int r = keys + e / (8 * kHalves), c = e % (8 * kHalves);
                    *reinterpret_cast<uint4 *>(v + (c >> 3) * (kAttnTileK * 128) + r * 128 + (c & 7) * 16) =
                        make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                __syncwarp();
            };
            ok &= wait(&q_full[0], nq0++ & 1);
            if (pair) {
                ok &= wait(&q_full[1], nq1++ & 1);
                // loads: K0 V0 K1 V1 ...
                wait_stage(0);
                if (n0 > 0) qk(0, 0, 0, 0);
                qk(1, 1, 0, 0);
                release(0);
                if (n == 1) commit(q_empty);
                for (int t = 0; t < n && ok; ++t) {
                    const uint32_t vi = 2 * t + 1, ki = 2 * t + 2;
                    wait_stage(vi);
                    clean(vi, t);
                    if (t < n0) {
                        pv(0, vi, t, t > 0);
                        if (t == n0 - 1) commit(&o_full[0]);
                    }
                    if (t + 1 < n) {
                        wait_stage(ki);
                        if (t + 1 < n0) qk(0, 0, ki, t + 1);
                    }
                    pv(1, vi, t, t > 0);
                    release(vi);
                    if (t == n - 1) commit(&o_full[1]);
                    if (t + 1 < n) {
                        qk(1, 1, ki, t + 1);
                        release(ki);
                        if (t + 2 == n) commit(q_empty);
                    }
                }
            } else {
                // loads: K0 K1 V0 K2 V1 K3 ... V(n-2) V(n-1); tile t is stream t & 1's
                for (int t = 0; t < 2 && t < n; ++t) {
                    wait_stage(t);
                    if (t == 0) qk(0, 0, 0, 0);
                    else qk(1, 0, 1, 1);
                    release(t);
                }
                if (n <= 2) commit(q_empty);
                for (int t = 0; t < n && ok; ++t) {
                    const uint32_t vi = min(2 * t + 2, n + t), ki = 2 * t + 3;
                    wait_stage(vi);
                    clean(vi, t);
                    if (t & 1) pv(1, vi, t, t > 1);
                    else pv(0, vi, t, t > 1);
                    release(vi);
                    if (t + 2 >= n) commit(&o_full[t & 1]);
                    if (t + 2 < n) {
                        wait_stage(ki);
                        if (t & 1) qk(1, 0, ki, t + 2);
                        else qk(0, 0, ki, t + 2);
                        release(ki);
                        if (t + 3 == n) commit(q_empty);
                    }
                }
            }
            it += 2 * n;
            if (!ok) break;
        }
    } else {
        // ===================== softmax and results ============================
        setmaxnreg_inc<kSoftmaxRegs>();
        const int s = warp >> 2, quad = warp & 3;
        const int r = quad * 32 + lane;   // my row of the query tile
        const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t t_s = tmem + lanes + s * kColS, t_o = tmem + lanes + kColO + s * DP;
        const int G = p.group, D = p.head_dim;
        const float c = p.scale * 1.4426950408889634f;
        uint32_t nitem = 0, ns = 0, no0 = 0, no1 = 0, nx = 0;
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
            // key tiles of the two streams
            const int cnt0 = w.pair ? max(0, min(w.t1, w.end0) - w.t0) : (n + 1) / 2, cnt1 = w.pair ? n : n / 2;
            const int mine_n = s ? cnt1 : cnt0;
            const int i = r / G, tok = (w.pair && s ? p.tq : 0) + i;   // my token of the block
            const bool row_ok = i < p.tq && tok < w.ntok;
            const int limit = row_ok ? max(0, min(w.kv_len, w.qpos0 + tok + 1)) : 0;
            const bool live = __any_sync(0xffffffffu, limit > 0);
            float m = -INFINITY, l = 0.f;
            for (int k = 0; k < mine_n; ++k) {
                const int tile = w.pair ? w.t0 + k : w.t0 + s + 2 * k;
                const int rem = limit - tile * kAttnTileK;   // my visible columns of this tile
                if (!wait(&s_full[s], ns++ & 1)) break;
                tc_fence_after();
                if (live) {
                    if (!__any_sync(0xffffffffu, rem > 0)) {   // no row of this warp sees the tile
                        uint32_t z[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) z[e] = 0;
#pragma unroll
                        for (int q = 0; q < 4; ++q) tmem_st16(t_s + 16 * q, z);
                    } else {
                        float x[128];
#pragma unroll
                        for (int q = 0; q < 4; ++q) tmem_ld32(t_s + 32 * q, x + 32 * q);
                        tmem_ld_wait();
#pragma unroll
                        for (int q = 0; q < 4; ++q) tmem_use32(x + 32 * q);
                        if (__any_sync(0xffffffffu, rem < kAttnTileK)) {
#pragma unroll
                            for (int e = 0; e < 128; ++e) x[e] = e < rem ? x[e] : -INFINITY;
                        }
                        float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                        for (int e = 4; e < 128; e += 8) {
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                mx[q] = e + 4 + q < 128 ? fmaxf(fmaxf(mx[q], x[e + q]), x[e + 4 + q])
                                                        : fmaxf(mx[q], x[e + q]);
                        }
                        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                        // the running maximum follows when it lags too far (always from -infinity)
                        const bool grow = (top - m) * c > kRescaleBits;
                        if (__any_sync(0xffffffffu, grow)) {
                            const float mn = grow ? top : m;
                            const float f = grow ? ex2((m - mn) * c) : 1.f;   // 0 from -infinity
                            m = mn;
                            l *= f;
                            if (k > 0) {   // O holds the earlier tiles' sums: S of this tile came after them
                                float o[32];
#pragma unroll
                                for (int q = 0; q < DP / 32; ++q) {
                                    tmem_ld32(t_o + 32 * q, o);
                                    tmem_ld_wait();
                                    tmem_use32(o);
#pragma unroll
                                    for (int e = 0; e < 32; ++e) o[e] *= f;
                                    tmem_st32(t_o + 32 * q, o);
                                }
                            }
                        }
                        const float off = m == -INFINITY ? 0.f : -m * c;
                        const uint64_t c2 = pack_f2(c, c), off2 = pack_f2(off, off);
                        uint64_t sum[2] = {0, 0};
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint32_t pk[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                float a, b;
                                unpack_f2(fma_f2(pack_f2(x[32 * q + 2 * e], x[32 * q + 2 * e + 1]), c2, off2), a, b);
                                a = ex2(a);
                                b = ex2(b);
                                sum[e & 1] = add_f2(sum[e & 1], pack_f2(a, b));
                                pk[e] = pack_bf16x2(a, b);
                            }
                            tmem_st16(t_s + 16 * q, pk);
                        }
                        float a0, a1;
                        unpack_f2(add_f2(sum[0], sum[1]), a0, a1);
                        l += a0 + a1;
                    }
                    tmem_st_wait();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[s]);
            }

            // ---- results ----------------------------------------------------
            const int g = r - i * G;
            float f0 = 1.f, f1 = 0.f;   // single: factors of the two streams' sums
            bool use0 = true, use1 = false;
            if (w.pair) {
                if (mine_n > 0) wait(&o_full[s], (s ? no1 : no0) & 1);
            } else {
                // both streams worked on the same rows: stream 0's threads join them
                if (s == 1) stats[r] = make_float2(m, l);
                wait(&o_full[0], no0 & 1);
                if (cnt1 > 0) wait(&o_full[1], no1 & 1);
                meet();
                if (s == 0) {
                    const float2 st = stats[r];
                    const float mm = fmaxf(m, st.x);
                    // a stream without keys for the row has nothing defined in O
                    use0 = l != 0.f;
                    use1 = st.y != 0.f;
                    f0 = use0 ? ex2((m - mm) * c) : 0.f;
                    f1 = use1 ? ex2((st.x - mm) * c) : 0.f;
                    m = mm;
                    l = l * f0 + st.y * f1;
                }
            }
            tc_fence_after();
            no0 += cnt0 > 0;
            no1 += cnt1 > 0;
            const bool mine = w.pair || s == 0;
            const int rho = tok * G + g;   // my row of the block
            if (mine && __any_sync(0xffffffffu, row_ok)) {
                const bool whole = w.parts == 1;
                const float inv = whole && l != 0.f ? 1.f / l : 1.f;
                const int64_t row = static_cast<int64_t>(w.tok0) + tok;
                const int head = w.kvh * G + g;
                uint8_t *out = whole ? reinterpret_cast<uint8_t *>(p.o + row * p.o_tok + head * p.o_head)
                                     : reinterpret_cast<uint8_t *>(p.part + (static_cast<int64_t>(w.slot) * p.part_rows + rho) * D);
                const uint64_t dst = row_ok ? reinterpret_cast<uint64_t>(out) : 0;
                // 16 columns of fp32 or 32 of bf16 at a time: 64 bytes a row
#pragma unroll 1
                for (int q = 0; 32 * q < D; ++q) {
                    float o[32];
                    tmem_ld32(t_o + 32 * q, o);
                    tmem_ld_wait();
                    tmem_use32(o);
                    if (!w.pair) {
                        float o1[32];
                        tmem_ld32(t_o + DP + 32 * q, o1);
                        tmem_ld_wait();
                        tmem_use32(o1);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = (use0 ? o[e] * f0 : 0.f) + (use1 ? o1[e] * f1 : 0.f);
                    }
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = l == 0.f ? 0.f : o[e] * inv;
                    uint32_t v[16];
                    if (whole) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] = pack_bf16x2(o[2 * e], o[2 * e + 1]);
                        store_rows(v, dst, 64 * q, D * 2, lane);
                    } else {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
#pragma unroll
                            for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(o[16 * h + e]);
                            store_rows(v, dst, 128 * q + 64 * h, D * 4, lane);
                        }
                    }
                }
                if (row_ok) {
                    if (!whole)
                        p.part_ml[static_cast<int64_t>(w.slot) * p.part_rows + rho] = make_float2(m, l);
                    else if (p.lse)
                        p.lse[row * p.heads + head] = l == 0.f ? -INFINITY : (m * c + log2f(l)) * 0.6931471805599453f;
                }
            }
            if (w.parts > 1) {
                // the piece that finishes last joins the group's pieces, in their order
                __threadfence();
                meet();
                if (threadIdx.x == 0)
                    *join_flag = atom_acq_rel_gpu_add(p.counters + ACNT_GROUP + w.unit0, 1) == w.parts - 1;
                meet();
                if (*join_flag) {
                    const int rows = w.ntok * G, d4 = D / 4;
                    auto slot_of = [&](int k) {
                        return static_cast<int64_t>(k == 0 ? 2 * w.unit0 + 1 : 2 * (w.unit0 + k)) * p.part_rows;
                    };
                    for (int u = threadIdx.x; u < rows * d4; u += 256) {
                        const int rr = u / d4, col = (u - rr * d4) * 4;
                        float mm = -INFINITY;
                        for (int k = 0; k < w.parts; ++k) mm = fmaxf(mm, __ldcg(&p.part_ml[slot_of(k) + rr].x));
                        float ll = 0.f, a[4] = {0.f, 0.f, 0.f, 0.f};
                        for (int k = 0; k < w.parts; ++k) {
                            const float2 ml = __ldcg(p.part_ml + slot_of(k) + rr);
                            const float4 v = __ldcg(reinterpret_cast<const float4 *>(p.part + (slot_of(k) + rr) * D + col));
                            const float f = ml.y == 0.f ? 0.f : ex2((ml.x - mm) * c);
                            ll += f * ml.y;
                            a[0] += f * v.x;
                            a[1] += f * v.y;
                            a[2] += f * v.z;
                            a[3] += f * v.w;
                        }
                        const float inv = ll == 0.f ? 0.f : 1.f / ll;
                        const int tk = rr / G, hd = w.kvh * G + (rr - tk * G);
                        const int64_t row = static_cast<int64_t>(w.tok0) + tk;
                        *reinterpret_cast<uint2 *>(p.o + row * p.o_tok + hd * p.o_head + col) =
                            make_uint2(pack_bf16x2(a[0] * inv, a[1] * inv), pack_bf16x2(a[2] * inv, a[3] * inv));
                        if (p.lse && col == 0)
                            p.lse[row * p.heads + hd] = ll == 0.f ? -INFINITY : (mm * c + log2f(ll)) * 0.6931471805599453f;
                    }
                    if (threadIdx.x == 0) p.counters[ACNT_GROUP + w.unit0] = 0;
                }
            } else if (!w.pair) {
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
        // loads in flight are waited for (bounded) before the shared memory goes,
        // matrix products before the tensor memory does
        auto settle = [&](uint64_t *bar, uint32_t parity) {
            mbar_wait(bar, parity, abort_flag, status, LORA_DEV_TIMEOUT, budget);
        };
        if (warp == 8 && lane == 0)
            for (int s = 0; s < kStages; ++s)
                if (drain[s] > 0) settle(&full[s], (drain[s] - 1) & 1);
        if (warp == 11 && lane == 0)
            for (int s = 0; s < 2; ++s)
                if (drain[kStages + s] > 0) settle(&q_full[s], (drain[kStages + s] - 1) & 1);
        if (warp == 9) {
            umma_commit_if(elect_one(), end_bar);
            settle(end_bar, 0);
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    }
    if (warp == 9) tmem_dealloc(tmem, 512);
    // the work-list counters go back to zero with the last CTA
    if (threadIdx.x == 0 && !hdr.cut) {
        if (atom_acq_rel_gpu_add(p.counters + ACNT_DONE, 1) == static_cast<int>(gridDim.x) - 1) {
            p.counters[ACNT_NEXT] = 0;
            p.counters[ACNT_DONE] = 0;
        }
    }
}

template <int DP, bool kPaged>
static cudaError_t launch(const AttnMaps &maps, const AttnParams &p, cudaStream_t stream)
{
    static int configured[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
    constexpr int bytes = AttnSmem<DP>::kBytes;
    if (dev >= 64 || !configured[dev]) {
        const cudaError_t e =
            cudaFuncSetAttribute(attn_kernel<DP, kPaged>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
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
    return cudaLaunchKernelEx(&cfg, attn_kernel<DP, kPaged>, maps, p);
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
        const uint32_t box[3] = {64, G, static_cast<uint32_t>(p.tq)}, box1[3] = {64, G, 1};
        if (!encode_map(&m.q, p.q, 3, dims, st, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !encode_map(&m.q1, p.q, 3, dims, st, box1, CU_TENSOR_MAP_SWIZZLE_128B))
            return cudaErrorInvalidValue;
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
        p.box_rows = 32;   // a short prompt's tile reads at most 31 rows too many
        const uint64_t dims[3] = {D, static_cast<uint64_t>(p.kv_heads), static_cast<uint64_t>(p.T)};
        const uint64_t ks[2] = {bytes(p.k_head, p.kv_heads), bytes(p.k_tok, p.T)};
        const uint64_t vs[2] = {bytes(p.v_head, p.kv_heads), bytes(p.v_tok, p.T)};
        const uint32_t box[3] = {64, 1, static_cast<uint32_t>(p.box_rows)};
        if (!encode_map(&m.k, p.k, 3, dims, ks, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !encode_map(&m.v, p.v, 3, dims, vs, box, CU_TENSOR_MAP_SWIZZLE_128B))
            return cudaErrorInvalidValue;
    }
    if (p.head_dim <= 64) return p.paged ? launch<64, true>(m, p, stream) : launch<64, false>(m, p, stream);
    return p.paged ? launch<128, true>(m, p, stream) : launch<128, false>(m, p, stream);
}

}  // namespace lora
