// Host side of include/lora_attn.h: argument checks, workspace carving and
// launches.  Nothing here allocates, synchronises or copies.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "attn.h"
#include "attn_checks.h"
#include "internal.h"
#include "lora_attn.h"

namespace lora {

static AttnLayout make_layout(int64_t T, int32_t R, int32_t heads, int32_t kv_heads, int32_t head_dim)
{
    AttnLayout L;
    std::memset(&L, 0, sizeof L);
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t a = o;
        o = align256(o + bytes);
        return a;
    };
    L.counters = take(ACNT_WORDS * 4);
    if (heads > 0) {
        const int group = heads / kv_heads;
        L.tq = kAttnTileQ / group;
        L.max_blocks = T / (2 * L.tq) + R;
        L.part_rows = static_cast<int32_t>(std::min<int64_t>(2 * L.tq, std::max<int64_t>(T, 1)) * group);
        L.hdr = take(sizeof(AttnHdr));
        L.first = take(static_cast<size_t>(kAttnMaxCtas) * sizeof(AttnItem));
        L.blocks = take(static_cast<size_t>(L.max_blocks) * sizeof(AttnBlock));
        L.part = take(static_cast<size_t>(2 * kAttnMaxCtas) * L.part_rows * head_dim * 4);
        L.part_ml = take(static_cast<size_t>(2 * kAttnMaxCtas) * L.part_rows * 8);
    }
    L.total = o;
    return L;
}

// What the places, the extents and the meaning of a list in ws depend on (but the
// lengths themselves), in 64 bits: a workspace may have been given to a step of other
// sizes since, to prompts instead of a cache, or to a cache of another bound.
static uint64_t sched_stamp(const AttnLayout &L, int64_t T, int32_t R, int32_t kv_heads, int32_t head_dim, int32_t ctas,
                            int32_t two, bool prompt, int64_t max_kv)
{
    uint64_t h = 0x243f6a8885a308d3ull;
    for (const uint64_t v : {uint64_t(T), uint64_t(R), uint64_t(kv_heads), uint64_t(head_dim), uint64_t(L.tq),
                             uint64_t(L.part_rows), uint64_t(ctas), uint64_t(two), uint64_t(prompt), uint64_t(max_kv)}) {
        h = (h ^ v) * 0x9e3779b97f4a7c15ull;   // odd: one value is told from another exactly
        h ^= h >> 29;
    }
    return h;
}

// Whether a step's list may have units of two heads of few rows, a stream each: a
// batch of single tokens (or a few) with more groups than the GPU holds several times
// over.  512 requests of one token over 50 to 300 take 96 us so and 119 by one head a
// unit, whose few tiles leave the second stream idle.  The kernel that can run both is
// about 1 % slower elsewhere, so it is launched for such batches only.
static bool two_heads(int64_t T, int32_t R, int32_t heads, int32_t kv_heads, bool paged, int32_t ctas)
{
    return paged && kv_heads % 2 == 0 && static_cast<int64_t>(R) * kv_heads >= 4 * ctas &&
           T * (heads / kv_heads) <= static_cast<int64_t>(R) * kAttnFewRows;
}

// Whether an attention over prompts makes its list itself (ShortList, attn.cu): whole
// groups, without the launch that builds a list (5 us of 13 for a prompt of 77 tokens).  At
// most 32 requests, a lane each, and two groups a CTA.  And no prompt may be so long that
// its groups had better be cut, of which the host knows the tokens in all.  A lone prompt
// that does not give every CTA a group: up to 6144 tokens with a head dimension of 128 (one
// head: 4096 tokens 48 us so, 53 by a schedule; 6144 70 and 67; 12000 130 and 73) and 4096
// with 64, whose pieces are joined faster (4096: 42 and 49; 6144 61 and 43; 12000 116 and
// 51).  With a group for every CTA, or several prompts, taken to be alike, up to 8192 (8
// heads on 1, 8000 tokens: 92 us, 98 by a schedule; 16 of 400 to 600 tokens, one head: 14
// and 18; but 15 of 50 beside one of 6000 67 and 65, with 64 59 and 43).
static bool makes_own_list(int64_t T, int32_t R, int32_t kv_heads, int32_t head_dim, const AttnLayout &L, int32_t ctas)
{
    if (R > 32 || L.max_blocks * kv_heads > 2 * ctas) return false;
    const bool busy = T / (2 * L.tq) * kv_heads >= ctas;
    return T <= (R > 1 || busy ? 8192 : 32 * (64 + head_dim));
}

static int enqueue_schedule(const int32_t *cu, const int32_t *kv_len, int32_t R, int64_t T, int64_t max_kv,
                            int32_t group, int32_t kv_heads, int32_t head_dim, const AttnLayout &L, void *ws,
                            cudaStream_t stream)
{
    const int32_t ctas = std::min(num_sms_current_device(), kAttnMaxCtas);
    AttnSchedParams p;
    p.cu = cu;
    p.kv_len = kv_len;
    p.R = R;
    p.tq = L.tq;
    p.group = group;
    p.two = two_heads(T, R, group * kv_heads, kv_heads, kv_len != nullptr, ctas);
    p.kv_heads = kv_heads;
    p.head_dim = head_dim;
    p.ctas = ctas;
    p.T = T;
    p.max_kv = max_kv;
    p.max_blocks = L.max_blocks;
    p.stamp = sched_stamp(L, T, R, kv_heads, head_dim, ctas, p.two, !kv_len, max_kv);
    p.hdr = at<AttnHdr>(ws, L.hdr);
    p.first = at<AttnItem>(ws, L.first);
    p.blocks = at<AttnBlock>(ws, L.blocks);
    p.counters = at<int32_t>(ws, L.counters);
    return launch_attn_schedule(p, stream) == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}

// The common part of both attentions: a schedule in ws, and the parameters.
static int prepare_attn(const lora_attn_t *a, const int32_t *kv_len, int64_t max_kv, const lora_attn_sched_t *sched,
                        void *ws, size_t ws_bytes, cudaStream_t stream, AttnParams *p)
{
    const AttnLayout L = make_layout(a->num_tokens, a->num_requests, a->heads, a->kv_heads, a->head_dim);
    const int rc = check_ws(ws, ws_bytes, L.total);
    if (rc) return rc;
    const int ctas = std::min(num_sms_current_device(), kAttnMaxCtas);
    const bool short_list = !sched && !kv_len &&
                            makes_own_list(a->num_tokens, a->num_requests, a->kv_heads, a->head_dim, L, ctas);
    if (sched) {
        if (sched->plan != ws || sched->num_tokens != a->num_tokens || sched->num_requests != a->num_requests ||
            sched->heads != a->heads || sched->kv_heads != a->kv_heads || sched->head_dim != a->head_dim ||
            sched->max_kv > max_kv || sched->prompt != (kv_len ? 0 : 1))
            return LORA_ERR_SEGMENTS;
    } else if (!short_list) {
        const int e = enqueue_schedule(a->cu, kv_len, a->num_requests, a->num_tokens, max_kv,
                                       a->heads / a->kv_heads, a->kv_heads, a->head_dim, L, ws, stream);
        if (e) return e;
    }
    std::memset(p, 0, sizeof *p);
    p->q = a->q;
    p->o = a->o;
    p->lse = a->lse;
    p->q_tok = a->q_token_stride;
    p->q_head = a->q_head_stride;
    p->o_tok = a->o_token_stride;
    p->o_head = a->o_head_stride;
    p->o_wide = aligned(a->o, 32) && (a->num_tokens == 1 || a->o_token_stride % 16 == 0) &&
                (a->heads == 1 || a->o_head_stride % 16 == 0);
    p->heads = a->heads;
    p->kv_heads = a->kv_heads;
    p->group = a->heads / a->kv_heads;
    p->head_dim = a->head_dim;
    p->tq = L.tq;
    p->scale = a->scale;
    p->hdr = at<AttnHdr>(ws, L.hdr);
    p->first = at<AttnItem>(ws, L.first);
    p->blocks = at<AttnBlock>(ws, L.blocks);
    p->max_blocks = L.max_blocks;
    p->counters = at<int32_t>(ws, L.counters);
    p->T = a->num_tokens;
    p->requests = a->num_requests;
    p->two = two_heads(a->num_tokens, a->num_requests, a->heads, a->kv_heads, kv_len != nullptr, ctas);
    p->stamp = sched_stamp(L, a->num_tokens, a->num_requests, a->kv_heads, a->head_dim, ctas, p->two, !kv_len,
                           sched ? sched->max_kv : max_kv);
    p->short_list = short_list;
    p->cu = a->cu;
    p->ctas = ctas;
    p->part = at<float>(ws, L.part);
    p->part_ml = at<float2>(ws, L.part_ml);
    p->part_rows = L.part_rows;
    p->wait_cycles = static_cast<uint32_t>(std::min<int64_t>(tc_wait_cycles(), 2000000000));
    return LORA_OK;
}

int attn_paged(const lora_attn_t *attn, const lora_kv_cache_t *cache, const int32_t *block_table, int32_t table_width,
               int64_t table_stride, const int32_t *kv_len, const lora_attn_sched_t *sched, bool f16, void *ws,
               size_t ws_bytes, cudaStream_t stream)
{
    int rc = check_attn(attn);
    if (rc) return rc;
    rc = check_cache(cache);
    if (rc) return rc;
    if (cache->kv_heads != attn->kv_heads || cache->head_dim != attn->head_dim) return LORA_ERR_SHAPE;
    if (table_width < 0 || static_cast<int64_t>(table_width) * cache->page_size > kMaxTokens) return LORA_ERR_SHAPE;
    if (attn->num_requests > 1 && table_stride < table_width) return LORA_ERR_SHAPE;
    if (attn->num_tokens == 0 || attn->num_requests == 0) return LORA_OK;
    if (!kv_len || (table_width > 0 && !block_table)) return LORA_ERR_NULL;
    if (!ints_aligned({kv_len, block_table})) return LORA_ERR_ALIGN;
    AttnParams p;
    rc = prepare_attn(attn, kv_len, static_cast<int64_t>(table_width) * cache->page_size, sched, ws, ws_bytes,
                      stream, &p);
    if (rc) return rc;
    if (f16 && p.two) return LORA_ERR_SHAPE;
    p.k = cache->k;
    p.v = cache->v;
    p.paged = 1;
    p.f16 = f16;
    p.block_table = block_table;
    p.table_stride = table_stride;
    p.table_width = table_width;
    p.num_pages = cache->num_pages;
    p.page_shift = page_shift(cache->page_size);
    p.page_stride = cache->page_stride;
    p.head_stride = cache->head_stride;
    p.slot_stride = cache->slot_stride;
    return launch_attn(p, stream) == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}

}  // namespace lora

using namespace lora;

extern "C" size_t lora_attn_workspace_size(int64_t num_tokens, int32_t num_requests, int32_t heads, int32_t kv_heads,
                                           int32_t head_dim)
{
    if (!step_ok(num_tokens, num_requests)) return 0;
    const bool none = heads == 0 && kv_heads == 0 && head_dim == 0;
    if (!none && !heads_ok(heads, kv_heads, head_dim)) return 0;
    return make_layout(num_tokens, num_requests, heads, kv_heads, head_dim).total;
}

extern "C" int lora_kv_plan(const lora_kv_plan_t *plan, void *ws, size_t ws_bytes, lora_stream_t stream)
{
    if (!plan) return LORA_ERR_NULL;
    const lora_kv_plan_t &a = *plan;
    if (!step_ok(a.max_tokens, a.num_requests) || a.table_width < 0 || a.num_free < 0) return LORA_ERR_SHAPE;
    if (a.page_size < 8 || a.page_size > 4096 || (a.page_size & (a.page_size - 1))) return LORA_ERR_SHAPE;
    if (a.num_pages <= 0 || static_cast<int64_t>(a.num_pages) * a.page_size >= (int64_t(1) << 31) ||
        static_cast<int64_t>(a.table_width) * a.page_size >= (int64_t(1) << 31))
        return LORA_ERR_SHAPE;
    if (a.num_requests > 1 && a.table_stride < a.table_width) return LORA_ERR_SHAPE;
    if (!a.free_head || !a.free_head_out || !a.cu_new || (a.num_free > 0 && !a.free_pages)) return LORA_ERR_NULL;
    if (a.num_requests > 0 && (!a.new_len || !a.ctx_len || !a.kv_len || (a.table_width > 0 && !a.block_table)))
        return LORA_ERR_NULL;
    if (a.max_tokens > 0 && (!a.slot_map || !a.position)) return LORA_ERR_NULL;
    if (!a.req_adapter != !a.lora_id_map && a.num_requests > 0 && a.max_tokens > 0) return LORA_ERR_NULL;
    // every CTA reads the lengths, the free count and the free list while others write
    if (a.free_head == a.free_head_out || a.cu_new == a.new_len || a.cu_new == a.ctx_len || a.kv_len == a.ctx_len ||
        a.kv_len == a.new_len)
        return LORA_ERR_SHAPE;
    if (!ints_aligned({a.new_len, a.ctx_len, a.req_adapter, a.block_table, a.free_pages, a.free_head, a.cu_new, a.kv_len,
                       a.slot_map, a.position, a.lora_id_map, a.free_head_out}))
        return LORA_ERR_ALIGN;
    const int rc = check_ws(ws, ws_bytes, make_layout(0, 0, 0, 0, 0).total);
    if (rc) return rc;
    KvPlanParams p;
    p.a = a;
    p.status = at<int32_t>(ws, 0) + CNT_STATUS;
    return launch_kv_plan(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}

extern "C" int lora_kv_store(const lora_bf16_t *k, const lora_bf16_t *v, int64_t num_tokens, int64_t k_token_stride,
                             int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                             const lora_kv_cache_t *cache, const int32_t *slot_map, void *ws, size_t ws_bytes,
                             lora_stream_t stream)
{
    int rc = check_cache(cache);
    if (rc) return rc;
    if (num_tokens < 0 || num_tokens > kMaxTokens) return LORA_ERR_SHAPE;
    if (!stride_ok(k_token_stride, num_tokens) || !stride_ok(v_token_stride, num_tokens) ||
        !stride_ok(k_head_stride, cache->kv_heads) || !stride_ok(v_head_stride, cache->kv_heads))
        return LORA_ERR_SHAPE;
    if (num_tokens == 0) return LORA_OK;
    if (!k || !v || !slot_map) return LORA_ERR_NULL;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slot_map, 4)) return LORA_ERR_ALIGN;
    rc = check_ws(ws, ws_bytes, make_layout(0, 0, 0, 0, 0).total);
    if (rc) return rc;
    KvStoreParams p;
    p.k = k;
    p.v = v;
    p.k_tok = k_token_stride;
    p.k_head = k_head_stride;
    p.v_tok = v_token_stride;
    p.v_head = v_head_stride;
    p.kc = cache->k;
    p.vc = cache->v;
    p.page_stride = cache->page_stride;
    p.head_stride = cache->head_stride;
    p.slot_stride = cache->slot_stride;
    p.slots = static_cast<int64_t>(cache->num_pages) * cache->page_size;
    p.page_shift = page_shift(cache->page_size);
    p.kv_heads = cache->kv_heads;
    p.vecs = cache->head_dim / 8;
    p.T = num_tokens;
    p.slot_map = slot_map;
    p.status = at<int32_t>(ws, 0) + CNT_STATUS;
    return launch_kv_store(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}

extern "C" int lora_attn_schedule(const int32_t *cu, const int32_t *kv_len, int32_t num_requests, int64_t num_tokens,
                                  int64_t max_kv, int32_t heads, int32_t kv_heads, int32_t head_dim,
                                  lora_attn_sched_t *out, void *ws, size_t ws_bytes, lora_stream_t stream)
{
    if (!step_ok(num_tokens, num_requests) || !heads_ok(heads, kv_heads, head_dim) || max_kv < 0 || max_kv > kMaxTokens)
        return LORA_ERR_SHAPE;
    if (!out || (num_requests > 0 && num_tokens > 0 && !cu)) return LORA_ERR_NULL;
    if (!ints_aligned({cu, kv_len})) return LORA_ERR_ALIGN;
    const AttnLayout L = make_layout(num_tokens, num_requests, heads, kv_heads, head_dim);
    const int rc = check_ws(ws, ws_bytes, L.total);
    if (rc) return rc;
    out->plan = ws;
    out->num_tokens = num_tokens;
    out->max_kv = max_kv;
    out->num_requests = num_requests;
    out->heads = heads;
    out->kv_heads = kv_heads;
    out->head_dim = head_dim;
    out->prompt = kv_len ? 0 : 1;
    if (num_requests == 0 || num_tokens == 0) return LORA_OK;
    return enqueue_schedule(cu, kv_len, num_requests, num_tokens, max_kv, heads / kv_heads, kv_heads, head_dim, L, ws,
                            static_cast<cudaStream_t>(stream));
}

extern "C" int lora_attn_paged(const lora_attn_t *attn, const lora_kv_cache_t *cache, const int32_t *block_table,
                               int32_t table_width, int64_t table_stride, const int32_t *kv_len,
                               const lora_attn_sched_t *sched, void *ws, size_t ws_bytes, lora_stream_t stream)
{
    return attn_paged(attn, cache, block_table, table_width, table_stride, kv_len, sched, false, ws, ws_bytes,
                      static_cast<cudaStream_t>(stream));
}

extern "C" int lora_attn_prompt(const lora_attn_t *attn, const lora_bf16_t *k, int64_t k_token_stride,
                                int64_t k_head_stride, const lora_bf16_t *v, int64_t v_token_stride,
                                int64_t v_head_stride, const lora_attn_sched_t *sched, void *ws, size_t ws_bytes,
                                lora_stream_t stream)
{
    int rc = check_attn(attn);
    if (rc) return rc;
    if (!stride_ok(k_token_stride, attn->num_tokens) || !stride_ok(v_token_stride, attn->num_tokens) ||
        !stride_ok(k_head_stride, attn->kv_heads) || !stride_ok(v_head_stride, attn->kv_heads))
        return LORA_ERR_SHAPE;
    if (attn->num_tokens == 0 || attn->num_requests == 0) return LORA_OK;
    if (!k || !v) return LORA_ERR_NULL;
    if (!aligned(k, 16) || !aligned(v, 16)) return LORA_ERR_ALIGN;
    AttnParams p;
    rc = prepare_attn(attn, nullptr, attn->num_tokens, sched, ws, ws_bytes, static_cast<cudaStream_t>(stream), &p);
    if (rc) return rc;
    p.k = k;
    p.v = v;
    p.k_tok = k_token_stride;
    p.k_head = k_head_stride;
    p.v_tok = v_token_stride;
    p.v_head = v_head_stride;
    return launch_attn(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}
