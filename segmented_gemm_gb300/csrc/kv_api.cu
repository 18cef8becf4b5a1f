// Host side of include/lora_kv.h: argument checks, workspace carving and
// launches.  Nothing here allocates, synchronises or copies.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "attn_checks.h"
#include "internal.h"
#include "kv_ops.h"

namespace lora {

constexpr size_t kStatusBytes = 256;   // workspace of the calls that only report

static bool page_size_ok(int32_t page_size, int32_t least)
{
    return page_size >= least && page_size <= 4096 && (page_size & (page_size - 1)) == 0;
}

// Bytes from one page or head of the 4-bit cache to the next.
static bool kv4_stride_ok(int64_t s, int64_t extent)
{
    return extent <= 1 || (s > 0 && s % 16 == 0 && s < (int64_t(1) << 36));
}

// Whether groups of 16 elements of every row start on 32 bytes, and none is half a group.
static bool whole_sectors(const void *base, int64_t token, int64_t tokens, int64_t head, int32_t heads, int32_t head_dim)
{
    return aligned(base, 32) && head_dim % 16 == 0 && (tokens == 1 || token % 16 == 0) && (heads == 1 || head % 16 == 0);
}

static int check_cache4(const lora_kv4_cache_t *c)
{
    if (!c || !c->data) return LORA_ERR_NULL;
    if (c->kv_heads <= 0 || c->head_dim <= 0 || c->head_dim > LORA_MAX_HEAD_DIM || c->head_dim % 8) return LORA_ERR_SHAPE;
    if (!page_size_ok(c->page_size, 16)) return LORA_ERR_SHAPE;
    if (c->num_pages <= 0 || static_cast<int64_t>(c->num_pages) * c->page_size >= (int64_t(1) << 31))
        return LORA_ERR_SHAPE;
    if (!kv4_stride_ok(c->page_stride, c->num_pages) || !kv4_stride_ok(c->head_stride, c->kv_heads)) return LORA_ERR_SHAPE;
    return aligned(c->data, 16) ? LORA_OK : LORA_ERR_ALIGN;
}

// Whether a step of T tokens of R requests, with room for wide ones (kv4_layout: rows enough altogether, as the bf16
// kernel is slow over a few long rows), is likely to have some: many rows a request, or many beyond one token each.
// One request of 48 tokens of 32/8 heads of 128 over 8000 takes 49 us by blocks of 8 columns, 90 unpacked, 400 tokens
// 160 and 97; over 1000 keys 48 tokens 18 and 33; 4 requests of 48 over 1000 to 8000 71 and 83; 8 of 32 119 and 87.
static bool maybe_wide(int64_t T, int32_t R, int32_t group, int32_t kv_heads, int32_t head_dim)
{
    const int64_t rows = kv4_wide_rows(head_dim);
    return T * group > R * rows || (T - R) * group >= 16 * rows;
}

static bool unpack_ok(int64_t tokens) { return tokens >= 0 && tokens <= (int64_t(1) << 24); }

static Kv4Layout kv4_layout(int64_t T, int32_t R, int32_t heads, int32_t kv_heads, int32_t head_dim, int64_t unpack)
{
    Kv4Layout L;
    std::memset(&L, 0, sizeof L);
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t a = o;
        o = align256(o + bytes);
        return a;
    };
    L.counters = take((kKv4CntGroup + kKv4MaxCtas) * 4);
    L.zeros = take(kv4_tile_bytes(128));
    // wide requests: none in steps of few rows, and no more than the rows allow, or than lists have places
    L.max_wide = T * heads < kKv4WideTotal ? 0 : static_cast<int32_t>(
        std::min<int64_t>({R, T * (heads / kv_heads) / (kv4_wide_rows(head_dim) + 1), LORA_MAX_REQUESTS / 2 - 1}));
    L.pages = static_cast<int32_t>(unpack / kKv4WidePage);
    if (L.max_wide == 0 || L.pages == 0) L.max_wide = L.pages = 0;
    L.attn_bytes = lora_attn_workspace_size(T, 2 * L.max_wide + 1, heads, kv_heads, head_dim);
    L.attn = take(L.max_wide ? L.attn_bytes : ACNT_WORDS * 4);
    const size_t dp = kv4_padded(head_dim), columns = static_cast<size_t>(kKv4MaxCtas) * (dp == 64 ? 16 : 8);
    L.first = take(8 * columns * (dp + 4) * 4);
    L.part = take(2 * columns * dp * 4);
    L.part_ml = take(2 * columns * 8);
    if (L.max_wide) {
        const size_t lists = 2 * static_cast<size_t>(L.max_wide) + 2, rows = static_cast<size_t>(L.pages) * kv_heads * kKv4WidePage;
        L.cu = take(lists * 4);
        L.kv_len = take(lists * 4);
        L.wide = take(R);
        L.pages_of = take(static_cast<size_t>(L.pages) * sizeof(int4));
        L.used = take(4);
        L.table = take((lists - 1) * L.pages * 4);
        L.k = take(rows * head_dim * 2);
        L.v = take(rows * head_dim * 2);
    }
    L.total = o;
    return L;
}

static size_t pages_workspace(int32_t num_pages)
{
    return kStatusBytes + (static_cast<size_t>(num_pages) + kBlockPages - 1) / kBlockPages * kPagesBlock;
}

static bool num_pages_ok(int32_t n) { return n > 0 && n < (1 << 28); }

static int check_pages(const lora_kv_pages_t *a)
{
    if (!a) return LORA_ERR_NULL;
    if (!page_size_ok(a->page_size, 8) || !num_pages_ok(a->num_pages) ||
        static_cast<int64_t>(a->num_pages) * a->page_size >= (int64_t(1) << 31))
        return LORA_ERR_SHAPE;
    if (a->num_rows < 0 || a->num_rows > LORA_MAX_REQUESTS || a->table_width < 0 || a->num_free < 0 ||
        static_cast<int64_t>(a->table_width) * a->page_size >= (int64_t(1) << 31))
        return LORA_ERR_SHAPE;
    if (a->num_rows > 1 && a->table_stride < a->table_width) return LORA_ERR_SHAPE;
    if (!a->ref || !a->free_head || (a->num_free > 0 && !a->free_pages)) return LORA_ERR_NULL;
    if (a->num_rows > 0 && (!a->ctx_len || (a->table_width > 0 && !a->block_table))) return LORA_ERR_NULL;
    return ints_aligned({a->block_table, a->ctx_len, a->ref, a->free_pages, a->free_head}) ? LORA_OK : LORA_ERR_ALIGN;
}

// The workspace, and the parameters that all calls on pages share.
static int prepare_pages(const lora_kv_pages_t *a, void *ws, size_t ws_bytes, KvPagesParams *p)
{
    const int rc = check_ws(ws, ws_bytes, pages_workspace(a->num_pages));
    if (rc) return rc;
    std::memset(p, 0, sizeof *p);
    p->a = *a;
    p->counters = at<int32_t>(ws, 0);
    p->blocks = at<uint8_t>(ws, kStatusBytes);
    return LORA_OK;
}

static int launched(cudaError_t e) { return e == cudaSuccess ? LORA_OK : LORA_ERR_CUDA; }

}  // namespace lora

using namespace lora;

extern "C" int lora_qk_rope(const lora_qk_rope_t *rope, const lora_kv_cache_t *cache, void *ws, size_t ws_bytes,
                            lora_stream_t stream)
{
    if (!rope) return LORA_ERR_NULL;
    const lora_qk_rope_t &a = *rope;
    if (cache) {
        const int rc = check_cache(cache);
        if (rc) return rc;
        if (cache->kv_heads != a.kv_heads || cache->head_dim != a.head_dim) return LORA_ERR_SHAPE;
    }
    if (a.num_tokens < 0 || a.num_tokens > kMaxTokens || a.heads < 0 || a.kv_heads < 0 || a.heads > 65536 ||
        a.kv_heads > 65536 || a.head_dim <= 0 || a.head_dim > LORA_MAX_HEAD_DIM || a.head_dim % 8 || a.rot_dim < 0 ||
        a.rot_dim > a.head_dim || a.rot_dim % 8)
        return LORA_ERR_SHAPE;
    if (!(a.eps >= 0.f) || !std::isfinite(a.eps)) return LORA_ERR_SHAPE;
    if (!stride_ok(a.q_token_stride, a.heads ? a.num_tokens : 0) || !stride_ok(a.q_head_stride, a.heads) ||
        !stride_ok(a.qo_token_stride, a.heads ? a.num_tokens : 0) || !stride_ok(a.qo_head_stride, a.heads) ||
        !stride_ok(a.k_token_stride, a.kv_heads ? a.num_tokens : 0) || !stride_ok(a.k_head_stride, a.kv_heads))
        return LORA_ERR_SHAPE;
    if (a.k_out && a.kv_heads &&
        (!stride_ok(a.ko_token_stride, a.num_tokens) || !stride_ok(a.ko_head_stride, a.kv_heads)))
        return LORA_ERR_SHAPE;
    if (cache && (!stride_ok(a.v_token_stride, a.num_tokens) || !stride_ok(a.v_head_stride, a.kv_heads)))
        return LORA_ERR_SHAPE;
    if (a.num_tokens == 0 || (a.heads == 0 && a.kv_heads == 0)) return LORA_OK;
    if ((a.heads && (!a.q || !a.q_out)) || (a.kv_heads && (!a.k || (!cache && !a.k_out)))) return LORA_ERR_NULL;
    if ((cache && (!a.v || !a.slot_map)) || !a.position || (a.rot_dim && !a.inv_freq)) return LORA_ERR_NULL;
    for (const void *x : {static_cast<const void *>(a.q), static_cast<const void *>(a.k), static_cast<const void *>(a.v),
                          static_cast<const void *>(a.q_out), static_cast<const void *>(a.k_out),
                          static_cast<const void *>(a.q_weight), static_cast<const void *>(a.k_weight)})
        if (!aligned(x, 16)) return LORA_ERR_ALIGN;
    if (!ints_aligned({a.position, a.inv_freq, a.slot_map})) return LORA_ERR_ALIGN;
    // in place means row by row
    if ((a.heads && a.q_out == a.q && ((a.num_tokens > 1 && a.qo_token_stride != a.q_token_stride) ||
                                       (a.heads > 1 && a.qo_head_stride != a.q_head_stride))) ||
        (a.kv_heads && a.k_out == a.k && ((a.num_tokens > 1 && a.ko_token_stride != a.k_token_stride) ||
                                          (a.kv_heads > 1 && a.ko_head_stride != a.k_head_stride))))
        return LORA_ERR_SHAPE;
    const int rc = check_ws(ws, ws_bytes, kStatusBytes);
    if (rc) return rc;
    QkRopeParams p;
    std::memset(&p, 0, sizeof p);
    p.a = a;
    p.status = at<int32_t>(ws, 0) + CNT_STATUS;
    if (cache) {
        p.kc = cache->k;
        p.vc = cache->v;
        p.page_stride = cache->page_stride;
        p.head_stride = cache->head_stride;
        p.slot_stride = cache->slot_stride;
        p.slots = static_cast<int64_t>(cache->num_pages) * cache->page_size;
        p.page_shift = page_shift(cache->page_size);
    }
    return launched(launch_qk_rope(p, static_cast<cudaStream_t>(stream)));
}

extern "C" size_t lora_kv4_block_size(int32_t page_size, int32_t head_dim)
{
    if (!page_size_ok(page_size, 16) || head_dim <= 0 || head_dim > LORA_MAX_HEAD_DIM || head_dim % 8) return 0;
    return static_cast<size_t>(page_size / 16) * kv4_tile_bytes(kv4_padded(head_dim));
}

extern "C" int lora_kv4_store(const lora_bf16_t *k, const lora_bf16_t *v, int64_t num_tokens, int64_t k_token_stride,
                              int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                              const lora_kv4_cache_t *cache, const int32_t *slot_map, void *ws, size_t ws_bytes,
                              lora_stream_t stream)
{
    int rc = check_cache4(cache);
    if (rc) return rc;
    if (num_tokens < 0 || num_tokens > kMaxTokens) return LORA_ERR_SHAPE;
    if (!stride_ok(k_token_stride, num_tokens) || !stride_ok(v_token_stride, num_tokens) ||
        !stride_ok(k_head_stride, cache->kv_heads) || !stride_ok(v_head_stride, cache->kv_heads))
        return LORA_ERR_SHAPE;
    if (num_tokens == 0) return LORA_OK;
    if (!k || !v || !slot_map) return LORA_ERR_NULL;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slot_map, 4)) return LORA_ERR_ALIGN;
    rc = check_ws(ws, ws_bytes, kStatusBytes);
    if (rc) return rc;
    Kv4StoreParams p;
    p.k = k;
    p.v = v;
    p.k_tok = k_token_stride;
    p.k_head = k_head_stride;
    p.v_tok = v_token_stride;
    p.v_head = v_head_stride;
    p.data = cache->data;
    p.page_stride = cache->page_stride;
    p.head_stride = cache->head_stride;
    p.slots = static_cast<int64_t>(cache->num_pages) * cache->page_size;
    p.page_shift = page_shift(cache->page_size);
    p.kv_heads = cache->kv_heads;
    p.head_dim = cache->head_dim;
    p.sectors = whole_sectors(k, k_token_stride, num_tokens, k_head_stride, cache->kv_heads, cache->head_dim) &&
                whole_sectors(v, v_token_stride, num_tokens, v_head_stride, cache->kv_heads, cache->head_dim);
    p.T = num_tokens;
    p.slot_map = slot_map;
    p.status = at<int32_t>(ws, 0) + CNT_STATUS;
    return launched(launch_kv4_store(p, static_cast<cudaStream_t>(stream)));
}

extern "C" int lora_kv4_load(const lora_kv4_cache_t *cache, const int32_t *slots, int64_t num_slots, lora_bf16_t *k,
                             lora_bf16_t *v, int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                             int64_t v_head_stride, void *ws, size_t ws_bytes, lora_stream_t stream)
{
    int rc = check_cache4(cache);
    if (rc) return rc;
    if (num_slots < 0 || num_slots > kMaxTokens) return LORA_ERR_SHAPE;
    if ((k && (!stride_ok(k_token_stride, num_slots) || !stride_ok(k_head_stride, cache->kv_heads))) ||
        (v && (!stride_ok(v_token_stride, num_slots) || !stride_ok(v_head_stride, cache->kv_heads))))
        return LORA_ERR_SHAPE;
    if (num_slots == 0 || (!k && !v)) return LORA_OK;
    if (!slots) return LORA_ERR_NULL;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4)) return LORA_ERR_ALIGN;
    rc = check_ws(ws, ws_bytes, kStatusBytes);
    if (rc) return rc;
    Kv4LoadParams p;
    p.k = k;
    p.v = v;
    p.k_tok = k_token_stride;
    p.k_head = k_head_stride;
    p.v_tok = v_token_stride;
    p.v_head = v_head_stride;
    p.data = cache->data;
    p.page_stride = cache->page_stride;
    p.head_stride = cache->head_stride;
    p.slots = static_cast<int64_t>(cache->num_pages) * cache->page_size;
    p.page_shift = page_shift(cache->page_size);
    p.kv_heads = cache->kv_heads;
    p.head_dim = cache->head_dim;
    p.sectors = whole_sectors(k, k_token_stride, num_slots, k_head_stride, cache->kv_heads, cache->head_dim) &&
                whole_sectors(v, v_token_stride, num_slots, v_head_stride, cache->kv_heads, cache->head_dim);
    p.n = num_slots;
    p.slot_list = slots;
    p.status = at<int32_t>(ws, 0) + CNT_STATUS;
    return launched(launch_kv4_load(p, static_cast<cudaStream_t>(stream)));
}

extern "C" size_t lora_kv4_workspace_size(int64_t num_tokens, int32_t num_requests, int32_t heads, int32_t kv_heads,
                                          int32_t head_dim, int64_t unpack_tokens)
{
    if (!step_ok(num_tokens, num_requests) || !heads_ok(heads, kv_heads, head_dim) || !unpack_ok(unpack_tokens)) return 0;
    return kv4_layout(num_tokens, num_requests, heads, kv_heads, head_dim, unpack_tokens).total;
}

extern "C" int lora_kv4_attn(const lora_attn_t *attn, const lora_kv4_cache_t *cache, const int32_t *block_table,
                             int32_t table_width, int64_t table_stride, const int32_t *kv_len, int64_t unpack_tokens,
                             void *ws, size_t ws_bytes, lora_stream_t stream)
{
    int rc = check_attn(attn);
    if (rc) return rc;
    rc = check_cache4(cache);
    if (rc) return rc;
    if (cache->kv_heads != attn->kv_heads || cache->head_dim != attn->head_dim) return LORA_ERR_SHAPE;
    if (table_width < 0 || static_cast<int64_t>(table_width) * cache->page_size > kMaxTokens) return LORA_ERR_SHAPE;
    if (attn->num_requests > 1 && table_stride < table_width) return LORA_ERR_SHAPE;
    if (attn->num_tokens * (attn->heads / attn->kv_heads) > kMaxTokens) return LORA_ERR_SHAPE;   // rows of a key head
    if (!unpack_ok(unpack_tokens)) return LORA_ERR_SHAPE;
    if (attn->num_tokens == 0 || attn->num_requests == 0) return LORA_OK;
    if (!kv_len || (table_width > 0 && !block_table)) return LORA_ERR_NULL;
    if (!ints_aligned({kv_len, block_table})) return LORA_ERR_ALIGN;
    const Kv4Layout L = kv4_layout(attn->num_tokens, attn->num_requests, attn->heads, attn->kv_heads, attn->head_dim,
                                   unpack_tokens);
    rc = check_ws(ws, ws_bytes, L.total);
    if (rc) return rc;
    Kv4AttnParams p;
    p.q = attn->q;
    p.o = attn->o;
    p.lse = attn->lse;
    p.q_tok = attn->q_token_stride;
    p.q_head = attn->q_head_stride;
    p.o_tok = attn->o_token_stride;
    p.o_head = attn->o_head_stride;
    p.cu = attn->cu;
    p.kv_len = kv_len;
    p.table = block_table;
    p.table_stride = table_stride;
    p.max_kv = static_cast<int64_t>(table_width) * cache->page_size;
    p.data = cache->data;
    p.page_stride = cache->page_stride;
    p.head_stride = cache->head_stride;
    p.num_pages = cache->num_pages;
    p.page_shift = page_shift(cache->page_size);
    p.T = static_cast<int32_t>(attn->num_tokens);
    p.R = attn->num_requests;
    p.heads = attn->heads;
    p.kv_heads = attn->kv_heads;
    p.group = attn->heads / attn->kv_heads;
    p.group_inverse = p.group > 1 ? ~uint64_t(0) / p.group + 1 : 0;
    p.head_dim = attn->head_dim;
    p.scale = attn->scale;
    p.zeros = at<uint8_t>(ws, L.zeros);
    p.counters = at<int32_t>(ws, L.counters);
    p.first = at<float>(ws, L.first);
    p.part = at<float>(ws, L.part);
    p.part_ml = at<float2>(ws, L.part_ml);
    p.wait_cycles = tc_wait_cycles();
    p.wide = nullptr;
    p.wide_status = nullptr;
    if (L.max_wide && maybe_wide(p.T, p.R, p.group, p.kv_heads, p.head_dim)) {   // the wide requests, by the attention over a bf16 cache; then the others
        Kv4WideParams w;
        w.cu = at<int32_t>(ws, L.cu);
        w.kv_len = at<int32_t>(ws, L.kv_len);
        w.wide = at<uint8_t>(ws, L.wide);
        w.pages_of = at<int4>(ws, L.pages_of);
        w.used = at<int32_t>(ws, L.used);
        w.table = at<int32_t>(ws, L.table);
        w.k = at<uint16_t>(ws, L.k);
        w.v = at<uint16_t>(ws, L.v);
        w.max_wide = L.max_wide;
        w.pages = L.pages;
        if (launch_kv4_wide_plan(w, p, static_cast<cudaStream_t>(stream)) != cudaSuccess) return LORA_ERR_CUDA;
        lora_attn_t a = *attn;
        a.cu = w.cu;
        a.num_requests = 2 * L.max_wide + 1;
        const int64_t slot = a.head_dim, head = slot * kKv4WidePage;
        const lora_kv_cache_t c = {w.k, w.v, head * a.kv_heads, head, slot, w.pages, kKv4WidePage, a.kv_heads, a.head_dim};
        lora_attn_sched_t list;
        rc = lora_attn_schedule(w.cu, w.kv_len, a.num_requests, a.num_tokens, static_cast<int64_t>(w.pages) * kKv4WidePage, a.heads,
                                a.kv_heads, a.head_dim, &list, at<void>(ws, L.attn), L.attn_bytes, stream);
        if (rc) return rc;
        if (launch_kv4_unpack(w, p, static_cast<cudaStream_t>(stream)) != cudaSuccess) return LORA_ERR_CUDA;
        rc = attn_paged(&a, &c, w.table, w.pages, w.pages, w.kv_len, &list, true, at<void>(ws, L.attn), L.attn_bytes,
                        static_cast<cudaStream_t>(stream));
        if (rc) return rc;
        p.wide = w.wide;
        p.wide_status = at<int32_t>(ws, L.attn) + CNT_STATUS;
    }
    return launched(launch_kv4_attn(p, static_cast<cudaStream_t>(stream)));
}

extern "C" size_t lora_kv_pages_workspace_size(int32_t num_pages)
{
    return num_pages_ok(num_pages) ? pages_workspace(num_pages) : 0;
}

extern "C" int lora_kv_release(const lora_kv_pages_t *pages, const int32_t *rows, int32_t num, void *ws, size_t ws_bytes,
                               lora_stream_t stream)
{
    int rc = check_pages(pages);
    if (rc) return rc;
    if (num < 0 || num > LORA_MAX_REQUESTS) return LORA_ERR_SHAPE;
    if (num == 0) return LORA_OK;
    if (!rows) return LORA_ERR_NULL;
    if (!aligned(rows, 4)) return LORA_ERR_ALIGN;
    KvPagesParams p;
    rc = prepare_pages(pages, ws, ws_bytes, &p);
    if (rc) return rc;
    p.rows = rows;
    p.num = num;
    return launched(launch_kv_release(p, static_cast<cudaStream_t>(stream)));
}

extern "C" int lora_kv_fork(const lora_kv_pages_t *pages, const int32_t *parent, const int32_t *child, int32_t num,
                            int32_t *copy_src, int32_t *copy_dst, void *ws, size_t ws_bytes, lora_stream_t stream)
{
    int rc = check_pages(pages);
    if (rc) return rc;
    if (num < 0 || num > LORA_MAX_REQUESTS) return LORA_ERR_SHAPE;
    if (num == 0) return LORA_OK;
    if (!parent || !child || !copy_src || !copy_dst) return LORA_ERR_NULL;
    if (!ints_aligned({parent, child, copy_src, copy_dst})) return LORA_ERR_ALIGN;
    KvPagesParams p;
    rc = prepare_pages(pages, ws, ws_bytes, &p);
    if (rc) return rc;
    p.parent = parent;
    p.child = child;
    p.num = num;
    p.src = copy_src;
    p.dst = copy_dst;
    return launched(launch_kv_fork(p, static_cast<cudaStream_t>(stream)));
}

extern "C" int lora_kv_compact(const lora_kv_pages_t *pages, int32_t limit, int32_t *copy_src, int32_t *copy_dst,
                               int32_t max_copies, int32_t *table_out, int32_t *ref_out, int32_t *free_out,
                               int32_t *head_out, void *ws, size_t ws_bytes, lora_stream_t stream)
{
    int rc = check_pages(pages);
    if (rc) return rc;
    if (limit < 0 || max_copies < 0) return LORA_ERR_SHAPE;
    if (max_copies > 0 && (!copy_src || !copy_dst)) return LORA_ERR_NULL;
    if (!ints_aligned({copy_src, copy_dst, table_out, ref_out, free_out, head_out})) return LORA_ERR_ALIGN;
    KvPagesParams p;
    rc = prepare_pages(pages, ws, ws_bytes, &p);
    if (rc) return rc;
    p.limit = limit;
    p.max_copies = max_copies;
    p.src = copy_src;
    p.dst = copy_dst;
    p.table_out = table_out ? table_out : pages->block_table;
    p.ref_out = ref_out ? ref_out : pages->ref;
    p.free_out = free_out ? free_out : pages->free_pages;
    p.head_out = head_out ? head_out : pages->free_head;
    return launched(launch_kv_compact(p, static_cast<cudaStream_t>(stream)));
}

// The common part of both copies.
static int copy_pages(const int32_t *src, const int32_t *dst, int32_t num, PageCopyParams *p, void *ws, size_t ws_bytes,
                      lora_stream_t stream)
{
    if (num < 0) return LORA_ERR_SHAPE;
    if (num == 0) return LORA_OK;
    if (!src || !dst) return LORA_ERR_NULL;
    if (!ints_aligned({src, dst})) return LORA_ERR_ALIGN;
    const int rc = check_ws(ws, ws_bytes, kStatusBytes);
    if (rc) return rc;
    p->src = src;
    p->dst = dst;
    p->num = num;
    p->status = at<int32_t>(ws, 0) + CNT_STATUS;
    return launched(launch_page_copy(*p, static_cast<cudaStream_t>(stream)));
}

extern "C" int lora_kv_copy(const int32_t *src, const int32_t *dst, int32_t num, const lora_kv_cache_t *cache, void *ws,
                            size_t ws_bytes, lora_stream_t stream)
{
    const int rc = check_cache(cache);
    if (rc) return rc;
    PageCopyParams p;
    std::memset(&p, 0, sizeof p);
    p.base[0] = reinterpret_cast<uint4 *>(cache->k);
    p.base[1] = reinterpret_cast<uint4 *>(cache->v);
    p.num_pages = cache->num_pages;
    p.page_stride = cache->page_stride / 8;
    p.heads = cache->kv_heads;
    p.rows = cache->page_size;
    p.vecs = cache->head_dim / 8;
    p.head_stride = cache->head_stride / 8;
    p.slot_stride = cache->slot_stride / 8;
    // a page's units without gaps, in either order of heads and slots: one run
    const bool heads_outer = p.slot_stride == p.vecs && (p.heads == 1 || p.head_stride == static_cast<int64_t>(p.rows) * p.vecs);
    const bool rows_outer = (p.heads == 1 || p.head_stride == p.vecs) && p.slot_stride == static_cast<int64_t>(p.heads) * p.vecs;
    if (static_cast<int64_t>(p.heads) * p.rows * p.vecs > (1 << 30)) return LORA_ERR_SHAPE;
    if (heads_outer || rows_outer) {
        p.vecs *= p.heads * p.rows;
        p.heads = p.rows = 1;
    }
    return copy_pages(src, dst, num, &p, ws, ws_bytes, stream);
}

extern "C" int lora_kv4_copy(const int32_t *src, const int32_t *dst, int32_t num, const lora_kv4_cache_t *cache,
                             void *ws, size_t ws_bytes, lora_stream_t stream)
{
    const int rc = check_cache4(cache);
    if (rc) return rc;
    PageCopyParams p;
    std::memset(&p, 0, sizeof p);
    p.base[0] = reinterpret_cast<uint4 *>(cache->data);
    p.num_pages = cache->num_pages;
    p.page_stride = cache->page_stride / 16;
    p.heads = cache->kv_heads;
    p.rows = 1;
    p.vecs = static_cast<int32_t>(lora_kv4_block_size(cache->page_size, cache->head_dim) / 16);
    p.head_stride = cache->head_stride / 16;
    if (static_cast<int64_t>(p.heads) * p.vecs > (1 << 30)) return LORA_ERR_SHAPE;
    if (p.heads == 1 || p.head_stride == p.vecs) {
        p.vecs *= p.heads;
        p.heads = 1;
    }
    return copy_pages(src, dst, num, &p, ws, ws_bytes, stream);
}
