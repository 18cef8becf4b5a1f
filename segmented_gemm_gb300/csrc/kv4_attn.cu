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
//     column, p of at most 2^kSlack has three bits more than in bf16;
//   - a warp is on its own: it takes tiles of 16 keys from its own ring of bulk
//     copies, so nothing but the ends of pieces is synchronised.
//
// The groups (request, key head, block of columns) in a row, a tile of each a
// unit, are cut evenly over the CTAs; a CTA's warps split each piece.  Pieces of a
// group cut by a CTA boundary go to the workspace, and the CTA that stores the
// last of them joins them in order.
#include <cuda_runtime.h>

#include "block_scan.cuh"
#include "kv4.cuh"
#include "kv_ops.h"
#include "internal.h"
#include "ptx.cuh"

namespace lora {

namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kStages = 4;          // tiles of a warp's ring
constexpr int kSlots = 4;           // results of warps in shared memory at a time
constexpr float kSlack = 8.f;       // log2 of the largest p
constexpr float kNone = -1e30f;     // m of a column that has seen no key
constexpr int kMinTiles = 16;       // least tiles of a CTA's share, two a warp

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

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t transposed(uint32_t v)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// Packed tokens of request r and its keys, clamped.
struct Request {
    int tok0, n, keys;
};

__device__ __forceinline__ Request request(const Kv4AttnParams &p, int r, int *bad)
{
    const int a0 = p.cu[r], b0 = p.cu[r + 1], k0 = p.kv_len[r];
    const int a = max(0, min(a0, p.T)), b = max(0, min(b0, p.T));
    Request q;
    q.tok0 = a;
    q.n = max(0, b - a);
    q.keys = static_cast<int>(k0 < 0 ? 0 : k0 > p.max_kv ? p.max_kv : k0);
    *bad |= (a != a0) | (b != b0) | (b < a) | (q.keys != k0);
    return q;
}

// The pieces of a CTA's share, one after another: tiles [t0, t1) of block b of key head h
// of request r.  A request has kv_heads * blocks groups of `tiles` tiles.
template <int NC>
struct Pieces {
    int r, h, b, t0, t1, tiles, blocks;
    Request q;
    int64_t left;

    __device__ __forceinline__ void take(const Kv4AttnParams &p)
    {
        int bad = 0;
        q = request(p, r, &bad);
        blocks = (q.n * p.group + NC - 1) / NC;
        tiles = max(1, (q.keys + 15) >> 4);
    }
    // the piece that starts at unit `at` of request r, of at most `share` units
    __device__ __forceinline__ void start(const Kv4AttnParams &p, int r_, int64_t at, int64_t share)
    {
        r = r_;
        take(p);
        const int64_t g = at / tiles;
        t0 = static_cast<int>(at - g * tiles);
        h = static_cast<int>(g / blocks);
        b = static_cast<int>(g - static_cast<int64_t>(h) * blocks);
        left = share;
        cut();
    }
    __device__ __forceinline__ void cut()
    {
        t1 = left < tiles - t0 ? t0 + static_cast<int>(left) : tiles;
        left -= t1 - t0;
    }
    __device__ __forceinline__ bool next(const Kv4AttnParams &p)
    {
        if (left <= 0) return false;
        t0 = t1;
        if (t0 == tiles) {
            t0 = 0;
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
        }
        cut();
        return true;
    }
    // keys that the block's last row sees, and a warp's tiles of the piece
    __device__ __forceinline__ int seen(int group) const
    {
        const int last = min(q.n - 1, (b * NC + NC - 1) / group);
        return max(0, q.keys - q.n + last + 1);
    }
    __device__ __forceinline__ void share(int group, int warp, int *a, int *e) const
    {
        const int end = min(t1, (seen(group) + 15) >> 4), len = max(0, end - t0);
        *a = t0 + len * warp / kWarps;
        *e = t0 + len * (warp + 1) / kWarps;
    }
};

template <int DP, int NT>
struct Smem {
    static constexpr int NC = 8 * NT;
    static constexpr int kPad = DP + 4;                                  // floats from a column of results to the next
    static constexpr int kTile = Kv4Tile<DP>::kBytes;
    static constexpr int kRing = kWarps * kStages * kTile;
    static constexpr int kQ = kRing;                                     // [NT][DP / 16][32] uint2
    static constexpr int kOut = kQ + NT * (DP / 16) * 32 * 8;            // [kSlots][NC][kPad] fp32
    static constexpr int kMl = kOut + kSlots * NC * kPad * 4;            // [kSlots][NC] (m, l)
    static constexpr int kFactor = kMl + kSlots * NC * 8;                // [NC] score factors
    static constexpr int kBars = kFactor + NC * 4;                       // [kWarps][kStages]
    static constexpr int kMisc = kBars + kWarps * kStages * 8;           // scan, share, flags
    static constexpr int kTotal = kMisc + 512;
};

template <int DP, int NT>
__global__ void __launch_bounds__(kThreads, NT <= 2 ? 2 : 1) kv4_attn_kernel(const Kv4AttnParams p)
{
    pdl_launch_dependents();
    using S = Smem<DP, NT>;
    using Tile = Kv4Tile<DP>;
    constexpr int NC = S::NC, KB = DP / 16, W = DP / 32;   // W: words of 8 codes of a lane's share of a key
    extern __shared__ __align__(128) uint8_t sm[];
    float *out = reinterpret_cast<float *>(sm + S::kOut);
    float2 *ml = reinterpret_cast<float2 *>(sm + S::kMl);
    float *factor = reinterpret_cast<float *>(sm + S::kFactor);
    int64_t *scan = reinterpret_cast<int64_t *>(sm + S::kMisc);          // [32]
    int64_t *found = scan + 32;                                          // request, unit in it
    volatile int *abort = reinterpret_cast<volatile int *>(found + 2);
    int *last = const_cast<int *>(abort) + 1;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    uint8_t *ring = sm + warp * kStages * S::kTile;
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + S::kBars) + warp * kStages;
    if (tid == 0) *abort = 0;
    if (lane == 0)
        for (int i = 0; i < kStages; ++i) mbar_init(full + i, 1);
    fence_mbarrier_init();
    int32_t *status = p.counters;
    pdl_wait();

    // this CTA's share of all units: every CTA counts them for itself
    const int run = (p.R + kThreads - 1) / kThreads, r0 = min(p.R, tid * run), r1 = min(p.R, r0 + run);
    auto units = [&](int r, int *bad) {
        const Request q = request(p, r, bad);
        const int64_t blocks = (q.n * p.group + NC - 1) / NC;
        return blocks * p.kv_heads * max(1, (q.keys + 15) >> 4);
    };
    int bad = 0;
    int64_t mine = 0, total;
    for (int r = r0; r < r1; ++r) mine += units(r, &bad);
    const int64_t base = block_scan_i64(mine, scan, &total);
    if (bad) atomicOr(status, LORA_DEV_BAD_LENGTH);
    const int64_t most = (total + kMinTiles - 1) / kMinTiles;
    const int ctas = static_cast<int>(most < gridDim.x ? most : gridDim.x);
    const int cta = blockIdx.x;
    if (cta >= ctas) return;
    const int64_t u0 = total * cta / ctas, u1 = total * (cta + 1) / ctas;
    if (u0 >= base && u0 < base + mine) {
        int64_t at = u0 - base;
        for (int r = r0; r < r1; ++r) {
            const int64_t n = units(r, &bad);
            if (at < n) {
                found[0] = r;
                found[1] = at;
                break;
            }
            at -= n;
        }
    }
    __syncthreads();

    Pieces<NC> piece, ahead;   // the one in work, and the one whose tiles are being fetched
    piece.start(p, static_cast<int>(found[0]), found[1], u1 - u0);
    ahead = piece;
    int64_t unit = u0;         // of the piece's first tile

    // ---- the warp's ring: tiles [fetch_t, fetch_e) of `ahead`, then of the pieces after it
    int fetch_t, fetch_e, issued = 0, pages = 0, pages_at = 0;
    bool more = true;
    ahead.share(p.group, warp, &fetch_t, &fetch_e);
    pages_at = fetch_t - 32;   // nothing loaded yet
    const int in_page = p.page_shift - 4;   // log2 of the tiles of a page
    auto fetch = [&]() {       // one more tile, if there is one
        while (more && fetch_t >= fetch_e) {
            more = ahead.next(p);
            if (more) {
                ahead.share(p.group, warp, &fetch_t, &fetch_e);
                pages_at = fetch_t - 32;
            }
        }
        if (!more) return;
        if (fetch_t - pages_at >= 32) {   // the pages of 32 tiles, one a lane
            pages_at = fetch_t;
            const int t = fetch_t + lane;
            pages = t < fetch_e ? p.table[ahead.r * p.table_stride + (t >> in_page)] : 0;
            const bool none = pages < 0 || pages >= p.num_pages;
            if (none) {
                atomicOr(status, LORA_DEV_BAD_PAGE);
                pages = -1;
            }
        }
        const int page = __shfl_sync(0xffffffffu, pages, fetch_t - pages_at);
        if (lane == 0) {
            const uint8_t *src = page < 0 ? p.zeros
                                          : p.data + page * p.page_stride + ahead.h * p.head_stride +
                                                (fetch_t & ((1 << in_page) - 1)) * static_cast<int64_t>(S::kTile);
            const int s = issued % kStages;
            mbar_expect_tx(full + s, S::kTile);
            bulk_load(ring + s * S::kTile, src, S::kTile, full + s);
        }
        ++issued;
        ++fetch_t;
    };
#pragma unroll 1
    for (int i = 0; i < kStages; ++i) fetch();
    int taken = 0;

    bool going = true;
    while (going) {
        // ---- queries: columns of fp16, scaled by a power of two, in the order of the B operand
        const int cols = min(NC, piece.q.n * p.group - piece.b * NC);   // columns with a row
        {
            constexpr int kLanes = DP / 8;                               // lanes of a column, 8 elements each
            const int sub = tid % kLanes;
#pragma unroll 1
            for (int n = tid / kLanes; n < NC; n += kThreads / kLanes) {
                uint4 x = {};
                if (n < cols && sub * 8 < p.head_dim) {
                    const int row = piece.b * NC + n, i = row / p.group, hg = row - i * p.group;
                    x = *reinterpret_cast<const uint4 *>(p.q + (piece.q.tok0 + i) * p.q_tok +
                                                         (piece.h * p.group + hg) * p.q_head + sub * 8);
                }
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                float f[8], top = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f[2 * i] = bf16_lo(w[i]);
                    f[2 * i + 1] = bf16_hi(w[i]);
                    top = fmaxf(top, fmaxf(fabsf(f[2 * i]), fabsf(f[2 * i + 1])));
                }
#pragma unroll   // whole warps have a column or none
                for (int d = kLanes / 2; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                // 2^(12 - e) for a largest magnitude in [2^e, 2^(e + 1)); rows of zeros or infinities stay as they are
                const int e = __float_as_uint(top) >> 23;
                const bool as_is = e < 13 || e > 254;
                const float by = as_is ? 1.f : __uint_as_float((266 - e) << 23);
                if (sub == 0) factor[n] = p.scale * 1.4426950408889634f * (as_is ? 1.f : __uint_as_float((e - 12) << 23));
                uint2 *to = reinterpret_cast<uint2 *>(sm + S::kQ) + (n / 8) * KB * 32;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int u = 2 * sub + i, cc = u / KB, kb = u % KB;   // 4 elements: part kb of lane cc's share
                    to[kb * 32 + (n % 8) * 4 + cc] = make_uint2(pack_f16x2(f[4 * i] * by, f[4 * i + 1] * by),
                                                                pack_f16x2(f[4 * i + 2] * by, f[4 * i + 3] * by));
                }
            }
        }
        __syncthreads();
        const uint2 *qs = reinterpret_cast<const uint2 *>(sm + S::kQ) + lane;
        uint2 qf[NT == 1 ? KB : 1];
        if (NT == 1)
#pragma unroll
            for (int i = 0; i < KB; ++i) qf[NT == 1 ? i : 0] = qs[i * 32];

        float fac[NT][2], m[NT][2], l[NT][2], o[NT][KB][4];
        int lim[NT][2], first_limit = 0x7fffffff;   // keys that a column sees; the fewest of any column
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int n = nt * 8 + 2 * c + e, i = (piece.b * NC + n) / p.group;
                fac[nt][e] = factor[n];
                lim[nt][e] = n < cols ? max(0, piece.q.keys - piece.q.n + i + 1) : 0x7fffffff;
                m[nt][e] = kNone;
                l[nt][e] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < KB; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nt][j][e] = 0.f;
        }
        first_limit = max(0, piece.q.keys - piece.q.n + (piece.b * NC) / p.group + 1);

        int t, te;
        piece.share(p.group, warp, &t, &te);
#pragma unroll 1
        for (; t < te; ++t) {
            const int s = taken % kStages;
            if (!mbar_wait(full + s, (taken / kStages) & 1, abort, status, LORA_DEV_TIMEOUT, p.wait_cycles)) break;
            const uint8_t *tile = ring + s * S::kTile;

            // ---- S^T: rows are the keys g and g + 8, columns 2c and 2c + 1
            float sc[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[nt][e] = 0.f;
            uint32_t kw[2][W];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint8_t *at = tile + e * (4 * DP) + lane * (4 * W);
                if (W == 4) *reinterpret_cast<uint4 *>(kw[e]) = *reinterpret_cast<const uint4 *>(at);
                else *reinterpret_cast<uint2 *>(kw[e]) = *reinterpret_cast<const uint2 *>(at);
            }
            uint32_t ks[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint8_t *at = tile + Tile::kKeyScales + (8 * e + g) * Tile::kGroups + c * (W / 2);
                ks[e] = W == 4 ? *reinterpret_cast<const uint16_t *>(at) : *at;
            }
#pragma unroll
            for (int w = 0; w < W; ++w) {   // 8 elements of each key, of one scale
                uint32_t f[2][4];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t s2 = w < 2 ? scale_pair<0, 0>(ks[e]) : scale_pair<1, 1>(ks[e]);
                    e2m1x8_to_f16(kw[e][w], f[e]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) f[e][i] = mul_f16x2(f[e][i], s2);
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

            // ---- p, and its sums
            const int key = t * 16 + g;
            const bool edge = t * 16 + 16 > first_limit;
            float rise = kNone;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float x = sc[nt][e] * fac[nt][e & 1];
                    if (edge && key + 8 * (e >> 1) >= lim[nt][e & 1]) x = -INFINITY;
                    sc[nt][e] = x;
                    rise = fmaxf(rise, x - m[nt][e & 1]);
                }
            if (__any_sync(0xffffffffu, rise > kSlack)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float top = fmaxf(sc[nt][e], sc[nt][e + 2]);
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                        top = fmaxf(top, m[nt][e]);
                        const float by = exp2_approx(m[nt][e] - top);
                        m[nt][e] = top;
                        l[nt][e] *= by;
#pragma unroll
                        for (int j = 0; j < KB; ++j) {
                            o[nt][j][e] *= by;
                            o[nt][j][e + 2] *= by;
                        }
                    }
            }
            uint32_t pb[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[e] = exp2_approx(sc[nt][e] - m[nt][e & 1]);
                    l[nt][e & 1] += x[e];   // before the rounding to fp16
                }
                pb[nt][0] = transposed(pack_f16x2(x[0], x[1]));
                pb[nt][1] = transposed(pack_f16x2(x[2], x[3]));
            }

            // ---- O^T: rows are elements of the values, inner dimension the keys 2c, 2c + 1 and 2c + 8, 2c + 9
            uint32_t vw[2][W];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint8_t *at = tile + Tile::kValues + e * (4 * DP) + lane * (4 * W);
                if (W == 4) *reinterpret_cast<uint4 *>(vw[e]) = *reinterpret_cast<const uint4 *>(at);
                else *reinterpret_cast<uint2 *>(vw[e]) = *reinterpret_cast<const uint2 *>(at);
            }
            uint32_t vs = *reinterpret_cast<const uint32_t *>(tile + Tile::kValueScales + ((DP == 128 ? g : g / 2) * 4 + c) * 4);
            if (t * 16 + 16 > piece.q.keys) {   // keys past the request: whatever they hold, their scales may be NaN
                const int k0 = t * 16 + 2 * c;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (k0 + (e & 1) + 8 * (e >> 1) >= piece.q.keys) vs &= ~(0xFFu << (8 * e));
            }
            __syncwarp();
            ++taken;
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
            fetch();
        }

        // ---- the warps' results: four at a time through shared memory
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], d);
        const int slot = warp % kSlots;
        float *mine_o = out + slot * NC * S::kPad;
        // a lane's elements of a column are consecutive: d = g * DP / 8 + 2j, + 1
        auto put = [&]() {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int n = nt * 8 + 2 * c + e;
                    float4 *to = reinterpret_cast<float4 *>(mine_o + n * S::kPad + g * (DP / 8));
#pragma unroll
                    for (int j = 0; j < KB / 2; ++j)
                        to[j] = make_float4(o[nt][2 * j][e], o[nt][2 * j][e + 2], o[nt][2 * j + 1][e], o[nt][2 * j + 1][e + 2]);
                    if (g == 0) ml[slot * NC + n] = make_float2(m[nt][e], l[nt][e]);
                }
        };
        if (warp >= kSlots) put();
        __syncthreads();
        if (warp < kSlots) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int n = nt * 8 + 2 * c + e;
                    const float2 other = ml[slot * NC + n];
                    const float top = fmaxf(m[nt][e], other.x);
                    const float by = exp2_approx(m[nt][e] - top), by2 = exp2_approx(other.x - top);
                    m[nt][e] = top;
                    l[nt][e] = l[nt][e] * by + other.y * by2;
                    const float4 *from = reinterpret_cast<const float4 *>(mine_o + n * S::kPad + g * (DP / 8));
#pragma unroll
                    for (int j = 0; j < KB / 2; ++j) {
                        const float4 v = from[j];
                        o[nt][2 * j][e] = o[nt][2 * j][e] * by + v.x * by2;
                        o[nt][2 * j][e + 2] = o[nt][2 * j][e + 2] * by + v.y * by2;
                        o[nt][2 * j + 1][e] = o[nt][2 * j + 1][e] * by + v.z * by2;
                        o[nt][2 * j + 1][e + 2] = o[nt][2 * j + 1][e + 2] * by + v.w * by2;
                    }
                }
            __syncwarp();
            put();
        }
        __syncthreads();

        // ---- their sum: the rows, or a part of a cut group
        const bool whole = piece.t0 == 0 && piece.t1 == piece.tiles;
        constexpr int kUnits = NC * (DP / 4);   // four elements of a column
        auto store = [&](int n, int d, float4 v, float top, float sum) {
            const int row = piece.b * NC + n, i = row / p.group, h = piece.h * p.group + row - i * p.group;
            const float by = sum != 0.f ? 1.f / sum : 0.f;   // no key: zeros
            if (sum == 0.f) v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (d < p.head_dim)
                *reinterpret_cast<uint2 *>(p.o + (piece.q.tok0 + i) * p.o_tok + h * p.o_head + d) =
                    make_uint2(pack_bf16x2(v.x * by, v.y * by), pack_bf16x2(v.z * by, v.w * by));
            if (d == 0 && p.lse)
                p.lse[static_cast<int64_t>(piece.q.tok0 + i) * p.heads + h] =
                    sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
        };
        const int at = 2 * cta + (piece.t0 == 0);
#pragma unroll 1
        for (int u = tid; u < kUnits; u += kThreads) {
            const int n = u / (DP / 4), d = u % (DP / 4) * 4;
            if (n >= cols) break;
            float top = kNone;
#pragma unroll
            for (int w = 0; w < kSlots; ++w) top = fmaxf(top, ml[w * NC + n].x);
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < kSlots; ++w) {
                const float2 x = ml[w * NC + n];
                const float by = exp2_approx(x.x - top);
                const float4 y = *reinterpret_cast<const float4 *>(out + (w * NC + n) * S::kPad + d);
                sum += x.y * by;
                v.x += y.x * by;
                v.y += y.y * by;
                v.z += y.z * by;
                v.w += y.w * by;
            }
            if (whole) {
                store(n, d, v, top, sum);
            } else {
                *reinterpret_cast<float4 *>(p.part + (static_cast<int64_t>(at) * NC + n) * DP + d) = v;
                if (d == 0) p.part_ml[at * NC + n] = make_float2(top, sum);
            }
        }
        if (!whole) {
            // the CTA that stores the last part joins them, in their order
            const int64_t from = unit - piece.t0, to = from + piece.tiles - 1;
            const int c0 = static_cast<int>(((from + 1) * ctas - 1) / total), c1 = static_cast<int>(((to + 1) * ctas - 1) / total);
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const int n = atom_acq_rel_gpu_add(p.counters + kKv4CntGroup + c0, 1);
                *last = n == c1 - c0;
                if (n == c1 - c0) p.counters[kKv4CntGroup + c0] = 0;
            }
            __syncthreads();
            if (*last) {
                __threadfence();
#pragma unroll 1
                for (int u = tid; u < kUnits; u += kThreads) {
                    const int n = u / (DP / 4), d = u % (DP / 4) * 4;
                    if (n >= cols) break;
                    float top = kNone, sum = 0.f;
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                    for (int i = c0; i <= c1; ++i) {
                        const int part = 2 * i + (i == c0);
                        const float2 x = __ldcg(p.part_ml + part * NC + n);
                        const float4 y = __ldcg(reinterpret_cast<const float4 *>(p.part + (static_cast<int64_t>(part) * NC + n) * DP + d));
                        const float next = fmaxf(top, x.x), by = exp2_approx(top - next), by2 = exp2_approx(x.x - next);
                        top = next;
                        sum = sum * by + x.y * by2;
                        v.x = v.x * by + y.x * by2;
                        v.y = v.y * by + y.y * by2;
                        v.z = v.z * by + y.z * by2;
                        v.w = v.w * by + y.w * by2;
                    }
                    store(n, d, v, top, sum);
                }
            }
        }
        unit += piece.t1 - piece.t0;
        going = piece.next(p);
        // `out` is written again only after the next piece's first barrier
    }
    // after a timeout: nothing may be in flight when the CTA ends
    for (; taken < issued; ++taken)
        mbar_wait(full + taken % kStages, (taken / kStages) & 1, abort, status, LORA_DEV_TIMEOUT,
                  p.wait_cycles < kWaitShort ? kWaitShort : p.wait_cycles);
}

template <int DP, int NT>
cudaError_t launch_variant(const Kv4AttnParams &p, cudaStream_t stream)
{
    constexpr int smem = Smem<DP, NT>::kTotal;
    static_assert(smem <= (NT <= 2 ? 113 : 227) * 1024, "shared memory");
    const cudaError_t e = cudaFuncSetAttribute(kv4_attn_kernel<DP, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    int64_t ctas = (NT <= 2 ? 2 : 1) * static_cast<int64_t>(num_sms_current_device());
    ctas = ctas < kKv4MaxCtas ? ctas : kKv4MaxCtas;
    return launch_pdl(kv4_attn_kernel<DP, NT>, ctas, kThreads, smem, p, stream);
}

}  // namespace

// Columns of a block: as many as an average request has rows.
cudaError_t launch_kv4_attn(const Kv4AttnParams &p, cudaStream_t stream)
{
    const int64_t rows = (static_cast<int64_t>(p.T) * p.group + p.R - 1) / p.R;
    if (p.head_dim <= 64)
        return rows <= 8 ? launch_variant<64, 1>(p, stream) : rows <= 16 ? launch_variant<64, 2>(p, stream)
                                                                        : launch_variant<64, 4>(p, stream);
    return rows <= 8 ? launch_variant<128, 1>(p, stream) : rows <= 16 ? launch_variant<128, 2>(p, stream)
                                                                     : launch_variant<128, 4>(p, stream);
}

}  // namespace lora
