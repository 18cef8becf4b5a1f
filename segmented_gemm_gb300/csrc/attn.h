// Internal declarations of the attention operators (include/lora_attn.h).
//
// Workspace (offsets 256-byte aligned):
//   counters   status word, work-list counters, arrival counters of split
//              groups                                   (zero at rest but the status)
//   hdr        schedule header (AttnHdr)
//   first      each CTA's first piece of work (AttnItem)
//   blocks     query blocks of the step (AttnBlock), longest first or (cut) in
//              request order
//   part       partial results of split groups: fp32 O rows, then (m, l) pairs
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "lora_attn.h"

namespace lora {

constexpr int kAttnTileQ = 128;     // rows of one query tile (UMMA M): tokens x the group's heads
constexpr int kAttnTileK = 128;     // keys of one key tile (UMMA N)
constexpr int kAttnFewRows = 16;    // rows of a block that take the quads' path
constexpr int kAttnMaxCtas = 160;   // upper bound on the persistent grid

// counter block entries (int32); the status word is lora.h's CNT_STATUS (0)
enum AttnCounters {
    ACNT_NEXT = 2,      // units taken beyond each CTA's first
    ACNT_DONE = 3,      // CTAs finished
    ACNT_GROUP = 32,    // [kAttnMaxCtas] partial results stored of the group that starts in a unit
    ACNT_WORDS = ACNT_GROUP + kAttnMaxCtas
};

// What starting and ending a piece costs, in key tiles: the cut schedule leaves
// that much room ahead of each group.
constexpr int kAttnItemCost = 2;

// A group's share of the cut list, gap and tiles.  In a list with pairs (key tiles
// against two query tiles) these weigh 2 against 1 for a tile against one query tile;
// all shares are even there, and so are the units, so that pieces of pairs begin and
// end on whole tiles.  In a list without any the weight is 1.  Decoding 31 requests of
// 1000 to 8000 tokens beside a chunk of 256 takes 116 us so, 161 with all tiles alike.
inline __host__ __device__ int32_t attn_gap(int32_t weight) { return kAttnItemCost * weight; }
inline __host__ __device__ int32_t attn_share(int32_t tiles, bool pair, int32_t weight)
{
    return (weight == 1 ? tiles : pair ? 2 * tiles : (tiles + 1) & ~1) + attn_gap(weight);
}

// A query block: up to two query tiles of one request, for every kv head.
struct __align__(16) AttnBlock {
    int32_t pre;      // cut: cost of the blocks before it (one head)
    int32_t base;     // where key 0 is found: paged, the request (its row of the block table); packed, its first row
    int32_t tok0;     // first packed row
    int32_t ntok;
    int32_t qpos0;    // row tok0 sees keys [0, qpos0 + 1) (none when that is <= 0)
    int32_t kv_len;
    int32_t tiles;    // key tiles its last row reaches, at least 1
    int32_t unused;
};

struct __align__(16) AttnHdr {
    int32_t nblocks;
    int32_t units;      // pieces of work
    int32_t cut;        // 0: a unit is one (block, head), blocks longest first; 1, 2: unit_cost of the list's
                        // cost, with this weight of a pair's tiles
    int32_t sec_heads;  // heads whose blocks run together (cut 0)
    int32_t unit_cost;  // cut; whole: 1 if a unit is a block and two kv heads
    int32_t cost;       // of all blocks and heads (cut)
    uint64_t stamp;     // of the sizes that it was made for (sched_stamp)
};

// A piece of one (block, kv head) group: key tiles [t0, t1).
struct __align__(16) AttnItem {
    int32_t valid;    // 0: no more; 2: two kv heads, kvh and the next, a stream each (few rows)
    int32_t pair;     // two query tiles (their streams share the key tiles), or one
    int32_t base, tok0, ntok, qpos0, kv_len;
    int32_t seen;     // keys that any of its rows sees
    int32_t kvh, t0, t1;
    int32_t end0;     // pair: tiles that stream 0's rows reach
    int32_t parts;    // pieces of the group
    int32_t slot;     // this piece's partial results (parts > 1)
    int32_t unit0;    // the unit that the group starts in (its counter; parts > 1)
    int32_t blk;      // its block
};

struct AttnLayout {
    int32_t tq;          // tokens of one query tile
    int64_t max_blocks;
    int32_t part_rows;   // rows of a partial slot
    size_t counters, hdr, first, blocks, part, part_ml, total;
};

struct AttnSchedParams {
    const int32_t *cu, *kv_len;
    int32_t R, tq, group, kv_heads, head_dim, ctas, two;
    int64_t T, max_kv, max_blocks;
    uint64_t stamp;
    AttnHdr *hdr;
    AttnItem *first;
    AttnBlock *blocks;
    int32_t *counters;
};

struct AttnParams {
    const uint16_t *q;
    uint16_t *o;
    float *lse;
    int64_t q_tok, q_head, o_tok, o_head;   // element strides
    int32_t heads, kv_heads, group, head_dim, tq;
    float scale;
    const AttnHdr *hdr;
    const AttnItem *first;
    const AttnBlock *blocks;
    int64_t max_blocks;
    uint64_t stamp;          // a list with another one is not run
    int32_t *counters;
    // keys and values: paged or packed rows
    const uint16_t *k, *v;
    int64_t k_tok, k_head, v_tok, v_head;   // packed: element strides
    const int32_t *block_table;
    int64_t table_stride;
    int32_t table_width, num_pages, page_shift;
    int64_t page_stride, head_stride, slot_stride;
    int32_t paged;
    int32_t f16;             // paged: the values are fp16, and p is rounded to it (the unpacked keys and values of a 4-bit cache)
    int32_t box_rows;        // keys of one TMA box
    int32_t o_wide;          // every row of o starts on a 32-byte boundary
    int64_t T;
    int32_t requests;
    int32_t two;             // units of two heads may be in the list (two_heads)
    int32_t short_list;      // 1: the list is made from cu in the kernel (hdr and blocks are not read)
    const int32_t *cu;
    int32_t ctas;
    float *part;             // [2 * kAttnMaxCtas][part_rows][head_dim] partial O
    float2 *part_ml;         // [2 * kAttnMaxCtas][part_rows] partial (m, l)
    int32_t part_rows;
    uint32_t wait_cycles;    // long budget of the bounded waits, in SM clock cycles
};

struct KvPlanParams {
    lora_kv_plan_t a;
    int32_t *status;
};

struct KvStoreParams {
    const uint16_t *k, *v;
    int64_t k_tok, k_head, v_tok, v_head;
    uint16_t *kc, *vc;
    int64_t page_stride, head_stride, slot_stride;
    int64_t slots;
    int32_t page_shift, kv_heads, vecs;   // vecs: 16-byte units of one head
    int64_t T;
    const int32_t *slot_map;
    int32_t *status;
};

cudaError_t launch_kv_plan(const KvPlanParams &p, cudaStream_t stream);
cudaError_t launch_kv_store(const KvStoreParams &p, cudaStream_t stream);
cudaError_t launch_attn_schedule(const AttnSchedParams &p, cudaStream_t stream);
cudaError_t launch_attn(AttnParams &p, cudaStream_t stream);   // fills in box_rows

// lora_attn_paged; f16: over values in fp16 instead of bf16 (batches of single tokens, two_heads, have no such kernel)
int attn_paged(const lora_attn_t *attn, const lora_kv_cache_t *cache, const int32_t *block_table, int32_t table_width,
               int64_t table_stride, const int32_t *kv_len, const lora_attn_sched_t *sched, bool f16, void *ws,
               size_t ws_bytes, cudaStream_t stream);

// Launch attribute of a programmatic dependent launch: the kernel may start
// its prologue while the one ahead finishes (every kernel here waits for it
// with griddepcontrol.wait before it touches memory).
inline void pdl_attribute(cudaLaunchConfig_t &cfg, cudaLaunchAttribute (&at)[1])
{
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
}

// defined in lora_api.cu
bool device_supported();
int num_sms_current_device();
bool encode_map(CUtensorMap *m, const void *base, int rank, const uint64_t *dims, const uint64_t *strides,
                const uint32_t *box, CUtensorMapSwizzle sw);

}  // namespace lora
