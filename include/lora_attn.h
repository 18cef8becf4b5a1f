/*
 * lora_attn.h — C ABI of the attention step between a layer's LoRA
 * projections: a paged key/value cache and causal attention over it.
 *
 * A serving step runs  merged QKV projection (lora_linear)  ->  lora_kv_store
 * ->  lora_attn_paged  ->  output projection (lora_linear)  in every layer,
 * after one lora_kv_plan (and one lora_attn_schedule) for the whole step.
 * Prompts that need no cache go through lora_attn_prompt.
 *
 * The conventions of lora.h hold: raw bf16, caller-owned buffers, no
 * allocation, no synchronisation, LORA_ERR_* for what the host can see,
 * status bits in the workspace (lora_get_status) for what only the device
 * sees, all work in order on `stream`.  lora_set_wait_budget bounds the
 * attention kernel's waits too.  int32 and fp32 arrays start on 4 bytes, tensors
 * on 16 and workspaces on 256 (LORA_ERR_ALIGN).
 *
 * The operators are an extension of this library: the page it follows leaves
 * attention to the serving engine.
 */
#ifndef LORA_GB300_LORA_ATTN_H
#define LORA_GB300_LORA_ATTN_H

#include "lora.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Device-side status bits of these operators (next to lora.h's). */
enum {
    LORA_DEV_BAD_LENGTH = 1 << 8, /* a length or an offset was negative, decreasing or past its bound (clamped) */
    LORA_DEV_NO_PAGE = 1 << 9,    /* the free list was too short: some request got no pages this step */
    LORA_DEV_BAD_PAGE = 1 << 10   /* a page or slot number outside the cache (not written; read as zeros) */
};

#define LORA_MAX_REQUESTS 4096    /* most requests of one step */
#define LORA_MAX_HEAD_DIM 128     /* largest head dimension (a multiple of 8) */
#define LORA_MAX_GROUP 128        /* most query heads that share a key/value head */

/*
 * A paged key/value cache of one layer.  Key (page, kv head, slot) is the
 * head_dim elements at k + page * page_stride + head * head_stride + slot *
 * slot_stride, and v likewise with the same strides: both the [pages, heads,
 * slots, dim] order and the [pages, slots, heads, dim] order fit.  Token
 * position p of a request lives in the page that its block table names at
 * p / page_size, in slot p % page_size.
 * k, v: DEVICE, 16-byte aligned.  Strides in elements, multiples of 8, below
 * 2^35 (a stride over a dimension of extent 1 is not looked at).  page_size a
 * power of two in [8, 4096]; num_pages * page_size < 2^31.
 */
typedef struct {
    lora_bf16_t *k;
    lora_bf16_t *v;
    int64_t page_stride;
    int64_t head_stride;
    int64_t slot_stride;
    int32_t num_pages;
    int32_t page_size;
    int32_t kv_heads;
    int32_t head_dim;
} lora_kv_cache_t;

/*
 * Block tables and slot map of one step, from the requests' lengths.
 *
 * Request r has ctx_len[r] tokens in the cache and adds new_len[r] (0 or
 * more).  The step's tokens are packed in request order:
 *   cu_new[r]     first packed token of request r, cu_new[num_requests] = all
 *   kv_len[r]     ctx_len[r] + new_len[r]
 * and for packed token t of request r, at position p = ctx_len[r] + t - cu_new[r]:
 *   position[t]   p
 *   slot_map[t]   table[r][p / page_size] * page_size + p % page_size
 *   lora_id_map[t] req_adapter[r]
 * with -1 in all three for max_tokens > t >= cu_new[num_requests].
 * The pages a request lacks, ceil(kv_len / page_size) - ceil(ctx_len /
 * page_size) of them, are taken from free_pages[*free_head ...] in request
 * order and entered in its table row; *free_head_out counts those taken.  If
 * the list runs short, the first request it cannot serve and every later one
 * that needs a page get none: kv_len 0 and slots -1 (their attention rows
 * come out as zeros), LORA_DEV_NO_PAGE.  Such a request keeps its ctx_len tokens
 * and pages: a caller goes on from kv_len where that is not 0 and from ctx_len
 * where it is, and offers the refused tokens again.  Table entries that are not
 * new stay as they were; calling again with the same inputs gives the same result.
 *
 * Lengths are clamped to [0, table_width * page_size] in all and to
 * max_tokens packed tokens (LORA_DEV_BAD_LENGTH).  A page number outside
 * [0, num_pages) gives slot -1 (LORA_DEV_BAD_PAGE).
 *
 * All arrays DEVICE int32: new_len, ctx_len, kv_len [num_requests], cu_new
 * [num_requests + 1], block_table [num_requests] rows of table_width entries
 * at table_stride, free_pages [num_free], free_head and free_head_out [1]
 * (different words), position and slot_map [max_tokens].  req_adapter
 * [num_requests] and lora_id_map [max_tokens] may both be NULL.
 * ws: DEVICE, lora_attn_workspace_size bytes (any heads), zero-filled once.
 */
typedef struct {
    const int32_t *new_len;
    const int32_t *ctx_len;
    const int32_t *req_adapter;
    int32_t num_requests;
    int32_t *block_table;
    int32_t table_width;
    int64_t table_stride;
    const int32_t *free_pages;
    int32_t num_free;
    const int32_t *free_head;
    int32_t page_size;
    int32_t num_pages;
    int64_t max_tokens;
    int32_t *cu_new;
    int32_t *kv_len;
    int32_t *slot_map;
    int32_t *position;
    int32_t *lora_id_map;
    int32_t *free_head_out;
} lora_kv_plan_t;

int lora_kv_plan(const lora_kv_plan_t *plan, void *ws, size_t ws_bytes, lora_stream_t stream);

/*
 * Write num_tokens new keys and values into the cache: token t's heads go to
 * slot slot_map[t] (page slot_map[t] / page_size).  A slot of -1 is skipped;
 * any other outside the cache is skipped with LORA_DEV_BAD_PAGE.  Two tokens
 * with one slot: which of them stays is not defined.
 * k, v: DEVICE bf16, head h of token t at t * token_stride + h * head_stride
 * elements (multiples of 8, bases 16-byte aligned), for instance the K and V
 * columns of a merged QKV projection's output.  They must not overlap the cache.
 */
int lora_kv_store(const lora_bf16_t *k, const lora_bf16_t *v, int64_t num_tokens, int64_t k_token_stride,
                  int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride, const lora_kv_cache_t *cache,
                  const int32_t *slot_map, void *ws, size_t ws_bytes, lora_stream_t stream);

/*
 * What both attentions take.  For request r with n = cu[r+1] - cu[r] packed
 * query rows and L keys, row i (0 <= i < n) of query head h sees the keys
 * j < max(0, L - n + i + 1) of key/value head h / (heads / kv_heads):
 *   o[cu[r] + i, h, :] = sum_j p_j v_j,   p = softmax_j(scale * q . k_j)
 *   lse[cu[r] + i, h]  = log sum_j exp(scale * q . k_j)
 * A row that sees no key gives o = 0 and lse = -infinity.  Rows that belong to
 * no request are not written.  Keys and values past a row's request are never
 * mixed in, whatever they hold (NaN and infinities included); a NaN or an
 * infinity in a value of the request itself may reach the request's other rows.
 * Scores, softmax sums and o accumulate in fp32; p is rounded to bf16 for the
 * second product (its sum is taken before that rounding), o once at the end.
 * The p of a row are taken relative to a score that may lie up to 2^40 below its
 * largest, so the unnormalised sums have that much less range: o is sure to be finite
 * for values of up to 2^60 in magnitude; larger ones may give infinity or NaN.
 *
 * q, o: DEVICE bf16, head h of row t at t * token_stride + h * head_stride
 * elements (multiples of 8; 16-byte aligned bases); o must not overlap q, the
 * keys or the values.  Rows of o that start on 32 bytes are written faster.
 * lse: DEVICE fp32
 * [num_tokens, heads] or NULL.  cu: DEVICE int32 [num_requests + 1].
 * heads a multiple of kv_heads, heads / kv_heads <= LORA_MAX_GROUP, head_dim
 * a multiple of 8 up to LORA_MAX_HEAD_DIM, scale positive and finite.
 */
typedef struct {
    const lora_bf16_t *q;
    lora_bf16_t *o;
    float *lse;
    const int32_t *cu;
    int64_t q_token_stride, q_head_stride;
    int64_t o_token_stride, o_head_stride;
    int64_t num_tokens;
    int32_t num_requests;
    int32_t heads;
    int32_t kv_heads;
    int32_t head_dim;
    float scale;
} lora_attn_t;

/*
 * Schedule of a step's attention: the work list that the kernel's CTAs take
 * their pieces from, built on the device from the lengths.  It serves every
 * layer of the step with the same head counts, and lives in ws.
 * cu as above; kv_len: DEVICE int32 [num_requests], the keys of each request
 * (NULL: as many as it has query rows, for lora_attn_prompt).  Lengths are
 * clamped to [0, max_kv] and offsets to [0, num_tokens]
 * (LORA_DEV_BAD_LENGTH).
 * *out: HOST; passed to the attention calls with the same ws.  It stands until
 * another schedule is built in that ws (an attention call without one does so
 * too).  An attention call that finds one of other sizes there, of another max_kv,
 * or of prompts for a cache (or the reverse), runs nothing and sets
 * LORA_DEV_CHECK; one of the same sizes with other lengths is not told apart.
 * After LORA_DEV_TIMEOUT build it anew.
 */
typedef struct {
    void *plan;
    int64_t num_tokens;
    int64_t max_kv;
    int32_t num_requests;
    int32_t heads;
    int32_t kv_heads;
    int32_t head_dim;
    int32_t prompt;      /* 1: built with kv_len NULL */
} lora_attn_sched_t;

/* Bytes of workspace for the calls of a step with up to num_tokens packed
 * tokens and num_requests requests (0 for arguments out of range).  heads,
 * kv_heads, head_dim 0: enough for lora_kv_plan and lora_kv_store only. */
size_t lora_attn_workspace_size(int64_t num_tokens, int32_t num_requests, int32_t heads, int32_t kv_heads,
                                int32_t head_dim);

int lora_attn_schedule(const int32_t *cu, const int32_t *kv_len, int32_t num_requests, int64_t num_tokens,
                       int64_t max_kv, int32_t heads, int32_t kv_heads, int32_t head_dim, lora_attn_sched_t *out,
                       void *ws, size_t ws_bytes, lora_stream_t stream);

/*
 * Attention of a step's new tokens over the paged cache (their own keys and
 * values stored there before): one token a request, a few, or a chunk of a
 * prompt, mixed freely.  kv_len: DEVICE int32 [num_requests].  block_table:
 * rows of table_width entries at table_stride (elements).  A page number
 * outside the cache reads as zeros (LORA_DEV_BAD_PAGE).  sched: a schedule
 * built for the same cu and kv_len with max_kv <= table_width * page_size,
 * or NULL to build one in ws first.
 */
int lora_attn_paged(const lora_attn_t *attn, const lora_kv_cache_t *cache, const int32_t *block_table,
                    int32_t table_width, int64_t table_stride, const int32_t *kv_len, const lora_attn_sched_t *sched,
                    void *ws, size_t ws_bytes, lora_stream_t stream);

/*
 * Causal attention over whole prompts packed one after another: request r's
 * queries, keys and values are rows [cu[r], cu[r+1]).  k, v: DEVICE bf16 like
 * q, with kv_heads heads.  sched: built with kv_len NULL, or NULL (the list of a
 * few short prompts is then made by the attention kernel itself).
 */
int lora_attn_prompt(const lora_attn_t *attn, const lora_bf16_t *k, int64_t k_token_stride, int64_t k_head_stride,
                     const lora_bf16_t *v, int64_t v_token_stride, int64_t v_head_stride,
                     const lora_attn_sched_t *sched, void *ws, size_t ws_bytes, lora_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* LORA_GB300_LORA_ATTN_H */
