// Internal declarations of the cache operators (include/lora_kv.h).
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "attn.h"
#include "lora_kv.h"

namespace lora {

// Elements of a head's row in the 4-bit cache, and bytes of a tile of 16 keys.
constexpr int kv4_padded(int head_dim) { return head_dim <= 64 ? 64 : 128; }
constexpr int kv4_tile_bytes(int padded) { return 18 * padded; }

struct QkRopeParams {
    int32_t cta_tokens;                         // of a CTA, set by the launch
    lora_qk_rope_t a;
    uint16_t *kc, *vc;                       // the cache, or NULL
    int64_t page_stride, head_stride, slot_stride;
    int64_t slots;
    int32_t page_shift;
    int32_t *status;
};

struct Kv4StoreParams {
    const uint16_t *k, *v;
    int64_t k_tok, k_head, v_tok, v_head;
    uint8_t *data;
    int64_t page_stride, head_stride;
    int64_t slots;
    int32_t page_shift, kv_heads, head_dim;
    int32_t sectors;                         // groups of 16 elements start on 32 bytes
    int64_t T;
    const int32_t *slot_map;
    int32_t *status;
};

struct Kv4LoadParams {
    uint16_t *k, *v;                         // either may be NULL
    int64_t k_tok, k_head, v_tok, v_head;
    const uint8_t *data;
    int64_t page_stride, head_stride;
    int64_t slots;
    int32_t page_shift, kv_heads, head_dim;
    int32_t sectors;
    int64_t n;
    const int32_t *slot_list;
    int32_t *status;
};

constexpr int kKv4MaxCtas = 2 * kAttnMaxCtas;   // upper bound on the 4-bit attention's grid

// Workspace of the 4-bit attention (offsets 256-byte aligned).  In front, at the same places in
// every call's layout, what is zero at rest: the status word and the arrival counters of
// split groups, a tile of zeros that stands for pages outside the cache, and the counters of the
// attention over a bf16 cache, whose workspace begins there.  Then partial results, of warps
// and of CTAs, and the wide requests' lists and unpacked pages.
struct Kv4Layout {
    size_t counters, zeros, attn, first, part, part_ml, cu, kv_len, wide, pages_of, used, table, k, v, total;
    size_t attn_bytes;
    int32_t max_wide, pages;
};
constexpr int kKv4CntGroup = 32;                // first arrival counter; one for each CTA
constexpr int kKv4WidePage = 128;               // keys of a page of the unpacked cache
// Most rows (tokens times a group's heads) of a request that is not wide.  8 requests over 1000 to 8000 take, 32/8
// heads of 128, with 64, 96 and 128 rows each 68, 93 and 119 us by blocks of 8 columns, 79, 83 and 87
// unpacked; with heads of 64, 64, 128 and 256 rows: 36, 58 and 102, and 50, 54 and 71.
// Least rows of all heads of a step with wide requests.  Microseconds by blocks and unpacked, one request:
//   heads       rows    over 1000        over 8000
//   8/1 of 128  1600    19 and 34        51 and 121
//               3200    26 and 36        89 and 85
//               6400    46 and 41       172 and 81
//   32/32       6400    37 and 37       164 and 106
//   32/4 of 64  3200    17 and 30        43 and 56
//               6400    23 and 31        74 and 55
//              12800    35 and 32       137 and 65
constexpr int kv4_wide_rows(int head_dim) { return head_dim <= 64 ? 160 : 96; }
constexpr int kKv4WideTotal = 6400;

struct Kv4AttnParams {
    const uint16_t *q;
    uint16_t *o;
    float *lse;
    int64_t q_tok, q_head, o_tok, o_head;       // element strides
    const int32_t *cu, *kv_len, *table;
    const uint8_t *wide;                        // [R] what is left out, or NULL
    int32_t *wide_status;                       // its status word, or NULL
    int64_t table_stride;
    int64_t max_kv;                             // table_width * page_size
    const uint8_t *data;
    int64_t page_stride, head_stride;           // bytes
    int32_t num_pages, page_shift;
    int32_t T, R;
    int32_t heads, kv_heads, group, head_dim;
    uint64_t group_inverse;                     // 2^64 / group, rounded up (group > 1)
    float scale;
    const uint8_t *zeros;
    int32_t *counters;
    float *first;                               // [warps][columns][padded head_dim + 4] first pieces of wide blocks
    float *part;                                // [2 * CTAs][columns][padded head_dim] partial O
    float2 *part_ml;                            // [2 * CTAs][columns] partial (m, l)
    int64_t wait_cycles;
};

struct Kv4WideParams {
    int32_t *cu, *kv_len;                       // [2 max_wide + 2], [2 max_wide + 1]: request 2i + 1 is the i-th wide one
    uint8_t *wide;                              // [R]
    int4 *pages_of;                             // [pages] request, page of the request, its keys
    int32_t *used;                              // unpacked pages
    int32_t *table;                             // [2 max_wide + 1][pages]
    uint16_t *k, *v;                            // [pages][kv_heads][kKv4WidePage][head_dim], bf16 and fp16
    int32_t max_wide, pages;
};

// Workspace of the calls on pages: the status and the counters, then a block for every kBlockPages pages with what is
// kept of them: the counts of its chunks, the pages' marks (used, free) and the map.  A page's place
// does not depend on how many there are, so a workspace may serve caches of different sizes in turn: the
// marks are zero at rest, counts and map are written before they are read.  (Every CTA reads all counts: a million
// pages are compacted in 44 us, 49 with blocks of one chunk.)
constexpr int kPagesArrived = 2;                // counter: CTAs done with their reading
constexpr int kPageChunk = 1024;                // pages that one CTA counts and lists
constexpr int kBlockChunks = 16, kBlockPages = kBlockChunks * kPageChunk;
constexpr int kPagesUsed = kBlockChunks * 16, kPagesFree = kPagesUsed + kBlockPages, kPagesMap = kPagesFree + kBlockPages;   // in a block
constexpr int kPagesBlock = kPagesMap + 4 * kBlockPages;

struct KvPagesParams {
    lora_kv_pages_t a;
    int32_t *counters;
    uint8_t *blocks;                            // [blocks][kPagesBlock]
    // release: rows; fork: parent and child
    const int32_t *rows, *parent, *child;
    int32_t num;
    int32_t *src, *dst;
    // compact
    int32_t limit, max_copies;
    int32_t *table_out, *ref_out, *free_out, *head_out;

    __host__ __device__ uint8_t *block(uint32_t i) const { return blocks + static_cast<int64_t>(i) * kPagesBlock; }
    __host__ __device__ uint8_t *used(uint32_t page) const { return block(page / kBlockPages) + kPagesUsed + page % kBlockPages; }
    __host__ __device__ uint8_t *free(uint32_t page) const { return used(page) + kBlockPages; }
    __host__ __device__ int4 *counts(uint32_t chunk) const
    {
        return reinterpret_cast<int4 *>(block(chunk / kBlockChunks)) + chunk % kBlockChunks;
    }
    // place + 1 of a page that moves, or 0
    __host__ __device__ int32_t *map(uint32_t page) const
    {
        return reinterpret_cast<int32_t *>(block(page / kBlockPages) + kPagesMap) + page % kBlockPages;
    }
};

struct PageCopyParams {
    const int32_t *src, *dst;
    int32_t num;
    int32_t num_pages;
    uint4 *base[2];                             // keys and values; the 4-bit cache has one
    int64_t page_stride;                        // in 16-byte units, as all below
    int64_t head_stride, slot_stride;
    int32_t rows, heads, vecs;                  // a page: heads x rows x vecs units (heads = rows = 1: contiguous)
    int32_t *status;
};

cudaError_t launch_qk_rope(QkRopeParams &p, cudaStream_t stream);
cudaError_t launch_kv4_store(const Kv4StoreParams &p, cudaStream_t stream);
cudaError_t launch_kv4_load(const Kv4LoadParams &p, cudaStream_t stream);
cudaError_t launch_kv4_wide_plan(const Kv4WideParams &w, const Kv4AttnParams &p, cudaStream_t stream);
cudaError_t launch_kv4_unpack(const Kv4WideParams &w, const Kv4AttnParams &p, cudaStream_t stream);   // behind the list
cudaError_t launch_kv4_attn(const Kv4AttnParams &p, cudaStream_t stream);
cudaError_t launch_kv_release(const KvPagesParams &p, cudaStream_t stream);
cudaError_t launch_kv_fork(const KvPagesParams &p, cudaStream_t stream);
cudaError_t launch_kv_compact(const KvPagesParams &p, cudaStream_t stream);
cudaError_t launch_page_copy(const PageCopyParams &p, cudaStream_t stream);

// A launch that may start its prologue while the one ahead finishes.
template <typename P>
inline cudaError_t launch_pdl(void (*kernel)(P), int64_t ctas, int threads, size_t smem, const P &p, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    pdl_attribute(cfg, at);
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace lora
