/*
 * lora_kv.h — C ABI of the cache operators around the serving attention of
 * lora_attn.h: norms and rotation of queries and keys on their way into the
 * cache, a cache held in 4 bits with the attention over it, and the sharing,
 * freeing and moving of pages.
 *
 * The conventions of lora_attn.h hold: raw bf16, caller-owned buffers, no
 * allocation, no synchronisation, LORA_ERR_* for what the host can see,
 * status bits in the workspace (lora_get_status) for what only the device
 * sees, all work in order on `stream`.  int32 and fp32 arrays start on 4
 * bytes, tensors on 16 and workspaces on 256 (LORA_ERR_ALIGN).  Calls that may
 * run at the same time have workspaces of their own.
 *
 * The operators are an extension of this library: the page it follows leaves
 * attention to the serving engine.
 */
#ifndef LORA_GB300_LORA_KV_H
#define LORA_GB300_LORA_KV_H

#include "lora_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Device-side status bit of these operators (next to lora.h's and lora_attn.h's). */
enum {
    LORA_DEV_BAD_ROW = 1 << 11    /* a row of the block table out of range, named twice, or parent and child at once (skipped) */
};

/* ------------------------------------------------------------------------
 * Norms and rotation of queries and keys
 * ------------------------------------------------------------------------
 * For every token t and every head's row x of q and k (head_dim elements):
 *   z = x * w / sqrt(mean(x^2) + eps)            with a weight, else z = x
 *   y_a = z_a cos(f) - z_b sin(f),  y_b = z_b cos(f) + z_a sin(f),
 *   f = position[t] * inv_freq[i]                for i < rot_dim / 2
 * where (a, b) = (i, i + rot_dim / 2), or (2i, 2i + 1) if interleaved; elements
 * from rot_dim on are not rotated.  fp32 arithmetic on angles reduced exactly
 * (positions up to 2^31 lose nothing), y rounded to bf16 once.
 *
 * q_out, k_out: where the rows go, q and k themselves with the same strides or
 * memory that does not overlap them.  With a cache, the keys y and the values of v
 * (copied) also go to slot slot_map[t] as in lora_kv_store, and k_out may be
 * NULL; without one, v and slot_map are not used.  A token of negative
 * position (lora_kv_plan gives -1 behind the last one) is passed over:
 * nothing of it is written.
 *
 * q, k, v, q_out, k_out: DEVICE bf16 rows with strides as in lora_attn_t.
 * q_weight, k_weight: DEVICE bf16 [head_dim], 16-byte aligned, each NULL for no norm.
 * position, slot_map: DEVICE int32 [num_tokens].  inv_freq: DEVICE fp32
 * [rot_dim / 2], finite.  head_dim a multiple of 8 up to LORA_MAX_HEAD_DIM,
 * rot_dim a multiple of 8 in [0, head_dim]; eps >= 0 and finite.  heads or
 * kv_heads may be 0 (without a cache), when those rows are not touched.
 * ws: lora_attn_workspace_size bytes (any heads).
 */
typedef struct {
    const lora_bf16_t *q, *k, *v;
    lora_bf16_t *q_out, *k_out;
    const lora_bf16_t *q_weight, *k_weight;
    const int32_t *position;
    const float *inv_freq;
    const int32_t *slot_map;
    int64_t q_token_stride, q_head_stride;
    int64_t k_token_stride, k_head_stride;
    int64_t v_token_stride, v_head_stride;
    int64_t qo_token_stride, qo_head_stride;
    int64_t ko_token_stride, ko_head_stride;
    int64_t num_tokens;
    int32_t heads;
    int32_t kv_heads;
    int32_t head_dim;
    int32_t rot_dim;
    int32_t interleaved;
    float eps;
} lora_qk_rope_t;

int lora_qk_rope(const lora_qk_rope_t *rope, const lora_kv_cache_t *cache, void *ws, size_t ws_bytes,
                 lora_stream_t stream);

/* ------------------------------------------------------------------------
 * A cache held in 4 bits
 * ------------------------------------------------------------------------
 * Every 16 consecutive elements of a head's key or value row share a scale:
 *   s    = max |x| / 6, rounded to the nearest number of 5 exponent and 3
 *          fraction bits (a 16-bit float's bits 14 to 7; at most 10240)
 *   code = x / s rounded to the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 (codes 0
 *          to 7, ties to the even code), + 8 for x < 0; 0 if s = 0
 * and stand for s * code, which bf16 holds exactly: 4.5 bits a value.  A group
 * of values below 2^-18 * 6 reads as zeros, values past 61440 as 61440; a group
 * with a NaN reads as NaN.
 *
 * Layout.  Dp = 64 for head_dim up to 64, else 128; elements past head_dim are
 * zeros.  16 slots of one head make a tile of 18 * Dp bytes, for key j < 16:
 *   0        key codes [16][Dp / 2], element d in byte d / 2, the even one in the low half
 *   8 * Dp   key scales [16][Dp / 16]
 *   9 * Dp   value codes: byte ((((j/8)*8 + d/(Dp/8))*4 + j%8/2)*(Dp/64) + d%(Dp/8)/8)*8 + (j%2)*4 + d%8/2
 *   17 * Dp  value scales: byte (d/16*4 + j%8/2)*4 + j/8*2 + j%2
 * the form in which the lanes of a warp take keys and values to the tensor
 * cores.  The tiles of a page's head are contiguous, head h of page p starts at
 * data + p * page_stride + h * head_stride bytes (multiples of 16, below 2^36; data
 * 16-byte aligned; a stride over a dimension of extent 1 is not looked at).
 * page_size a power of two in [16, 4096]; num_pages * page_size < 2^31.
 * Memory that was never written is to be zeros (or any bytes whose scales
 * are numbers): the padding past head_dim is read.
 */
typedef struct {
    uint8_t *data;
    int64_t page_stride;
    int64_t head_stride;
    int32_t num_pages;
    int32_t page_size;
    int32_t kv_heads;
    int32_t head_dim;
} lora_kv4_cache_t;

/* Bytes of one head of one page (0 for arguments out of range). */
size_t lora_kv4_block_size(int32_t page_size, int32_t head_dim);

/* lora_kv_store into a 4-bit cache; k, v, strides, slot_map and ws as there (of two tokens with one slot
 * groups of either may stay). */
int lora_kv4_store(const lora_bf16_t *k, const lora_bf16_t *v, int64_t num_tokens, int64_t k_token_stride,
                   int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride, const lora_kv4_cache_t *cache,
                   const int32_t *slot_map, void *ws, size_t ws_bytes, lora_stream_t stream);

/*
 * The keys and values that slots[i] hold, in bf16 (exactly): row i of k and v.
 * A slot of -1 gives zeros; so does any other outside the cache, with
 * LORA_DEV_BAD_PAGE.  k, v: DEVICE bf16, as in lora_kv_store, either may be NULL.
 * A request's tokens are read back so to move it to a bf16 cache, or to attend
 * over its prompt by lora_attn_prompt.
 */
int lora_kv4_load(const lora_kv4_cache_t *cache, const int32_t *slots, int64_t num_slots, lora_bf16_t *k,
                  lora_bf16_t *v, int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                  int64_t v_head_stride, void *ws, size_t ws_bytes, lora_stream_t stream);

/* Bytes of workspace for lora_kv4_attn over steps of up to num_tokens tokens and num_requests requests with
 * this unpack_tokens (0 for arguments out of range); zero-filled once. */
size_t lora_kv4_workspace_size(int64_t num_tokens, int32_t num_requests, int32_t heads, int32_t kv_heads,
                               int32_t head_dim, int64_t unpack_tokens);

/*
 * lora_attn_paged over a 4-bit cache: the same arguments, the same rows, over
 * the values that the cache stands for.  Needs no schedule.  q keeps its bf16
 * values (elements below 2^-26 of their row's largest lose bits, rows below 2^-114
 * are zeros), p is rounded to fp16 (11 bits) for the second product whichever way a request
 * takes, o to bf16 once; scores, statistics and sums are fp32.  Keys and values past a row's
 * request are never mixed in, whatever they hold.  kv_len is clamped to [0, table_width * page_size], offsets to [0,
 * num_tokens] (LORA_DEV_BAD_LENGTH).  A page outside the cache reads as zeros
 * (LORA_DEV_BAD_PAGE).
 *
 * unpack_tokens: keys and values that the workspace has room for in 16 bits (0: none).
 * In steps with chunks of prompts (of 6400 rows of all heads), requests of more than 96 rows (new tokens times
 * heads / kv_heads; 160 for a head_dim up to 64), in order as long as they fit, are
 * unpacked there, exactly, and go through lora_attn_paged's kernel in a form with p in fp16 (8 chunks of 64 tokens over
 * 1000 to 8000, 32/8 heads of 128: 113 us so, 224 without).  Up to 2^24, in units of 128 (others are
 * rounded down); each such request needs its cached tokens, rounded up to 128.  The host tells such steps by their
 * sizes: more rows of a key head than 96 (160) a request, or 1536 (2560) beyond one token a request.
 *
 * Faster than lora_attn_paged over a bf16 cache wherever the cache's bytes count; slower for one request
 * over some 1000 tokens (12 us, 9 there with a schedule made) and for few long chunks (one of
 * 512 over 8000: 102 to 104 us, 87 there).
 */
int lora_kv4_attn(const lora_attn_t *attn, const lora_kv4_cache_t *cache, const int32_t *block_table,
                  int32_t table_width, int64_t table_stride, const int32_t *kv_len, int64_t unpack_tokens, void *ws,
                  size_t ws_bytes, lora_stream_t stream);

/* ------------------------------------------------------------------------
 * Pages
 * ------------------------------------------------------------------------
 * What lora_kv_plan keeps a row (request) of the block table's pages in, and
 * counts beside it: ref[p] is the number of rows that hold page p beyond the
 * first, so it is 0 for a page that one row holds or none, and for every page
 * that lora_kv_plan hands out.  Row r holds the first ceil(ctx_len[r] /
 * page_size) entries of its table row.  A page that several rows hold is full:
 * new tokens never go there.
 *
 * block_table: DEVICE int32, num_rows rows (up to LORA_MAX_REQUESTS) of table_width
 * entries at table_stride.  ctx_len: DEVICE int32 [num_rows].  ref: DEVICE
 * int32 [num_pages], zero-filled once.  free_pages: DEVICE int32 [num_free], of
 * which [*free_head, num_free) are free; free_head: DEVICE int32 [1], read and
 * written (lora_kv_plan's free_head_out goes in, and its next free_head comes
 * out).  Lengths are clamped to [0, table_width * page_size] (LORA_DEV_BAD_LENGTH);
 * a page outside [0, num_pages) in a table or list is passed over (LORA_DEV_BAD_PAGE).
 * page_size as in lora_kv_cache_t.
 */
typedef struct {
    int32_t *block_table;
    int64_t table_stride;
    int32_t table_width;
    int32_t num_rows;
    int32_t *ctx_len;
    int32_t *ref;
    int32_t *free_pages;
    int32_t *free_head;
    int32_t num_free;
    int32_t page_size;
    int32_t num_pages;
} lora_kv_pages_t;

/* Bytes of workspace for the calls below (0 for arguments out of range); zero-filled once.  One for a cache of
 * num_pages serves smaller ones too, in any order. */
size_t lora_kv_pages_workspace_size(int32_t num_pages);

/*
 * Rows rows[0 .. num) give up their pages: each page loses one holder a row,
 * and a page without any joins the free list, in front of *free_head, which goes
 * down by as many; the pages freed stand there in ascending order.  ctx_len of
 * the rows becomes 0; their table entries stay as they were.  A row named twice
 * or out of range counts once or not at all (LORA_DEV_BAD_ROW).  Where the list
 * has no room in front of *free_head (more pages come back than were taken
 * from it), the last ones are lost to it, LORA_DEV_NO_PAGE.
 * rows: DEVICE int32 [num], num up to LORA_MAX_REQUESTS.
 */
int lora_kv_release(const lora_kv_pages_t *pages, const int32_t *rows, int32_t num, void *ws, size_t ws_bytes,
                    lora_stream_t stream);

/*
 * Row child[i] becomes a continuation of row parent[i] (parallel samples, beams),
 * for i < num in order: it shares the parent's full pages, and where the last one is not
 * full it gets a fresh page from the free list for its own copy of it:
 *   copy_src[i], copy_dst[i]   that page and the fresh one, or -1 and -1
 * which lora_kv_copy (lora_kv4_copy) then copies in every layer's cache.
 * ctx_len[child[i]] = ctx_len[parent[i]].  If the list runs short, the first
 * fork it cannot serve and every later one that needs a page get none: ctx_len
 * 0, no pages shared, LORA_DEV_NO_PAGE.
 * A child row holds no pages before (lora_kv_release).  A row out of range, a
 * child named twice (the later times) or that is a parent of this call
 * is skipped: pair -1, the child's row as it was, LORA_DEV_BAD_ROW.
 * parent, child, copy_src, copy_dst: DEVICE int32 [num], num up to LORA_MAX_REQUESTS.
 */
int lora_kv_fork(const lora_kv_pages_t *pages, const int32_t *parent, const int32_t *child, int32_t num,
                 int32_t *copy_src, int32_t *copy_dst, void *ws, size_t ws_bytes, lora_stream_t stream);

/*
 * Moves held pages >= limit to free ones < limit, so that the cache can be cut to
 * its first `limit` pages: the i-th such held page, in ascending order, takes the
 * i-th such free one, as long as there are both, and max_copies at most:
 *   copy_src[i], copy_dst[i]   from and to, -1 and -1 behind the last pair
 * which lora_kv_copy (lora_kv4_copy) then copies in every layer's cache.  The
 * tables (held entries) and counts follow; a page that several rows hold moves once.
 * The free pages, the vacated ones among them, stand at the end of the list in
 * ascending order, *free_head at the first.  A page that no row holds and that
 * is not free stays as it is.  A page that is held and free is held (LORA_DEV_BAD_PAGE).
 * table_out (rows of table_width at table_stride), ref_out, free_out, head_out:
 * where the new state goes, whole (all the table's entries, the list's taken ones too): NULL or the arrays of
 * `pages` themselves for in place, or memory that does not overlap them.
 */
int lora_kv_compact(const lora_kv_pages_t *pages, int32_t limit, int32_t *copy_src, int32_t *copy_dst,
                    int32_t max_copies, int32_t *table_out, int32_t *ref_out, int32_t *free_out, int32_t *head_out,
                    void *ws, size_t ws_bytes, lora_stream_t stream);

/*
 * Copies page src[i] of the cache, keys and values of all heads, to page dst[i],
 * for i < num.  A pair of -1 is skipped; so is one with either outside the
 * cache, with LORA_DEV_BAD_PAGE.  A page that is the destination of one pair is
 * in no other (the outcome is not defined).  src, dst: DEVICE int32 [num].
 * ws: lora_kv_pages_workspace_size or lora_attn_workspace_size bytes.
 */
int lora_kv_copy(const int32_t *src, const int32_t *dst, int32_t num, const lora_kv_cache_t *cache, void *ws,
                 size_t ws_bytes, lora_stream_t stream);
int lora_kv4_copy(const int32_t *src, const int32_t *dst, int32_t num, const lora_kv4_cache_t *cache, void *ws,
                  size_t ws_bytes, lora_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* LORA_GB300_LORA_KV_H */
