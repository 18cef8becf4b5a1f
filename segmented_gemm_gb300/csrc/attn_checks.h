// Host-side argument checks that the attention's and the cache's entry points
// share (include/lora_attn.h, include/lora_kv.h).
#pragma once
#include <cmath>
#include <cstddef>
#include <cstdint>
#include <initializer_list>

#include "attn.h"
#include "internal.h"

namespace lora {

inline size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// int32 arrays: each is NULL or starts on 4 bytes (the kernels would fault on any other).
inline bool ints_aligned(std::initializer_list<const void *> arrays)
{
    for (const void *p : arrays)
        if (!aligned(p, 4)) return false;
    return true;
}

template <typename T>
inline T *at(void *ws, size_t off)
{
    return reinterpret_cast<T *>(static_cast<char *>(ws) + off);
}

inline bool heads_ok(int32_t heads, int32_t kv_heads, int32_t head_dim)
{
    return heads > 0 && kv_heads > 0 && heads % kv_heads == 0 && heads / kv_heads <= LORA_MAX_GROUP && head_dim > 0 &&
           head_dim <= LORA_MAX_HEAD_DIM && head_dim % 8 == 0;
}

inline bool step_ok(int64_t T, int32_t R) { return T >= 0 && T <= kMaxTokens && R >= 0 && R <= LORA_MAX_REQUESTS; }

// A stride the kernels use: elements, a multiple of 8, not negative; one over
// a dimension of extent 1 is never used and may be anything.
inline bool stride_ok(int64_t s, int64_t extent)
{
    return extent <= 1 || (s > 0 && s % 8 == 0 && s < (int64_t(1) << 35));
}

inline int check_cache(const lora_kv_cache_t *c)
{
    if (!c || !c->k || !c->v) return LORA_ERR_NULL;
    if (c->kv_heads <= 0 || c->head_dim <= 0 || c->head_dim > LORA_MAX_HEAD_DIM || c->head_dim % 8) return LORA_ERR_SHAPE;
    if (c->page_size < 8 || c->page_size > 4096 || (c->page_size & (c->page_size - 1))) return LORA_ERR_SHAPE;
    if (c->num_pages <= 0 || static_cast<int64_t>(c->num_pages) * c->page_size >= (int64_t(1) << 31))
        return LORA_ERR_SHAPE;
    if (!stride_ok(c->page_stride, c->num_pages) || !stride_ok(c->head_stride, c->kv_heads) ||
        !stride_ok(c->slot_stride, c->page_size))
        return LORA_ERR_SHAPE;
    if (!aligned(c->k, 16) || !aligned(c->v, 16)) return LORA_ERR_ALIGN;
    return LORA_OK;
}

inline int page_shift(int32_t page_size)
{
    int s = 0;
    while ((1 << s) < page_size) ++s;
    return s;
}

inline int check_attn(const lora_attn_t *a)
{
    if (!a) return LORA_ERR_NULL;
    if (!step_ok(a->num_tokens, a->num_requests) || !heads_ok(a->heads, a->kv_heads, a->head_dim))
        return LORA_ERR_SHAPE;
    if (!(a->scale > 0.f) || !std::isfinite(a->scale)) return LORA_ERR_SHAPE;
    if (!stride_ok(a->q_token_stride, a->num_tokens) || !stride_ok(a->q_head_stride, a->heads) ||
        !stride_ok(a->o_token_stride, a->num_tokens) || !stride_ok(a->o_head_stride, a->heads))
        return LORA_ERR_SHAPE;
    if (a->num_tokens == 0 || a->num_requests == 0) return LORA_OK;
    if (!a->q || !a->o || !a->cu) return LORA_ERR_NULL;
    if (!aligned(a->q, 16) || !aligned(a->o, 16) || !aligned(a->lse, 4) || !aligned(a->cu, 4)) return LORA_ERR_ALIGN;
    return LORA_OK;
}

inline int check_ws(const void *ws, size_t bytes, size_t need)
{
    if (!ws || bytes < need) return LORA_ERR_WORKSPACE;
    if (!aligned(ws, 256)) return LORA_ERR_ALIGN;
    return device_supported() ? LORA_OK : LORA_ERR_UNSUPPORTED;
}

}  // namespace lora
