// Pieces of the attention's work: what a CTA is told of the next one, for the
// kernel that runs them and the one that lays out each CTA's first.
#pragma once
#include "attn.h"

namespace lora {

// Everything of a piece but its place in the cut.
__device__ __forceinline__ AttnItem item_of(const AttnBlock &b, int blk, int kvh, int tq)
{
    AttnItem w = {};
    w.valid = 1;
    w.pair = b.ntok > tq;
    w.base = b.base;
    w.tok0 = b.tok0;
    w.ntok = b.ntok;
    w.qpos0 = b.qpos0;
    w.kv_len = b.kv_len;
    w.seen = min(b.kv_len, b.qpos0 + b.ntok);
    w.kvh = kvh;
    w.t1 = b.tiles;
    w.end0 = max(1, (min(b.kv_len, b.qpos0 + min(b.ntok, tq)) + kAttnTileK - 1) / kAttnTileK);
    w.parts = 1;
    w.blk = blk;
    return w;
}

// whole: unit u is a group, or two of a block; the heads of a section together, blocks
// longest first
__device__ __forceinline__ void whole_unit(const AttnHdr &h, int kv_heads, uint32_t u, int *blk, int *kvh)
{
    const int two = h.unit_cost;
    kv_heads >>= two;
    const uint32_t per = h.nblocks * h.sec_heads, sec = u / per, rem = u - sec * per;
    const uint32_t hs = min(h.sec_heads, kv_heads - static_cast<int>(sec) * h.sec_heads), at = rem / hs;
    *blk = static_cast<int>(at);
    *kvh = static_cast<int>(sec * h.sec_heads + rem - at * hs) << two;
}

// cut: where the tiles of group (b, kvh) start in the list, a gap into its share
__device__ __forceinline__ int group_start(const AttnHdr &h, const AttnBlock &b, int kvh, int kv_heads, bool pair)
{
    return b.pre * kv_heads + kvh * attn_share(b.tiles, pair, h.cut) + attn_gap(h.cut);
}

// cut: the part of group (b, kvh) that lies in [pos, end) of the list, where unit
// `unit` ends; valid 0 if it starts past the end.  *pos moves to the end of what was taken.
__device__ __forceinline__ AttnItem cut_piece(const AttnHdr &h, const AttnBlock &b, int blk, int kvh, int kv_heads, int tq,
                                              int unit, int end, int *pos)
{
    AttnItem w = item_of(b, blk, kvh, tq);
    const int g0 = group_start(h, b, kvh, kv_heads, w.pair), shift = w.pair ? h.cut - 1 : 0;   // a tile weighs 1 << shift
    w.valid = *pos < end && g0 < end;
    w.t0 = max(0, *pos - g0) >> shift;
    w.t1 = min(b.tiles, (end - g0) >> shift);
    const uint32_t c = h.unit_cost, u0 = static_cast<uint32_t>(g0) / c;
    const uint32_t u1 = static_cast<uint32_t>(g0 + ((b.tiles - 1) << shift)) / c;
    w.parts = static_cast<int>(u1 - u0 + 1);
    w.slot = 2 * unit + (static_cast<uint32_t>(unit) == u0);
    w.unit0 = static_cast<int>(u0);
    *pos = g0 + (w.t1 << shift);
    return w;
}

}  // namespace lora
