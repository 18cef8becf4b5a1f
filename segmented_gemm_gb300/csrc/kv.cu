// The paged cache's bookkeeping and its writes (include/lora_attn.h):
// lora_kv_plan and lora_kv_store.
#include <cuda_runtime.h>

#include "attn.h"
#include "block_scan.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace lora {

// ---------------------------------------------------------------------------
// lora_kv_plan
// ---------------------------------------------------------------------------
// With n_r the new and c_r the cached tokens (clamped), P slots a page:
//   cu_r   = sum_{s < r} n_s
//   need_r = ceil((c_r + n_r) / P) - ceil(c_r / P),   before_r = sum_{s < r} need_s
//   served_r  iff  need_r = 0 or before_r + need_r <= num_free - head
// before_r is increasing, so the served requests that need pages are a prefix
// and take free pages [head, head + before_r + need_r) without gaps.
//
// A few KB in all: launch latency bounds it.  So it is one launch without any
// exchange between CTAs: every CTA scans all lengths (at most 4096, in shared
// memory) for itself, then takes its share of the tokens and of the new table
// entries.  A token whose page is new in this call computes the page from the
// scan instead of reading the table that another CTA may be writing.
constexpr int kPlanThreads = 256;
constexpr int kPlanTokens = 2048;   // tokens a CTA takes at least, so that small steps stay in few CTAs

__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(const KvPlanParams prm)
{
    pdl_launch_dependents();
    const lora_kv_plan_t &a = prm.a;
    extern __shared__ int32_t sm[];
    const int R = a.num_requests;
    int32_t *cu = sm;              // [R + 1]
    int32_t *before = cu + R + 1;  // [R + 1] pages needed by the requests before r
    int32_t *ctx = before + R + 1; // [R]
    __shared__ int64_t wsum[32];
    const int tid = threadIdx.x;
    const int P = a.page_size, shift = __ffs(P) - 1;
    const int64_t cap = static_cast<int64_t>(a.table_width) << shift;
    pdl_wait();

    int bad = 0, missing = 0;
    // packed offsets: at most max_tokens in all
    int64_t carry = 0;
    for (int r0 = 0; r0 < R; r0 += kPlanThreads) {
        const int r = r0 + tid;
        int64_t n = 0;
        if (r < R) {
            const int n0 = a.new_len[r], c0 = a.ctx_len[r];
            const int64_t c = c0 < 0 ? 0 : c0 > cap ? cap : c0;
            n = n0 < 0 ? 0 : n0 > cap - c ? cap - c : n0;
            bad |= (c != c0) | (n != n0);
            ctx[r] = static_cast<int32_t>(c);
        }
        int64_t total;
        const int64_t ex = carry + block_scan_i64(n, wsum, &total);
        if (r < R) cu[r] = static_cast<int32_t>(ex < a.max_tokens ? ex : a.max_tokens);
        carry += total;
    }
    if (tid == 0) cu[R] = static_cast<int32_t>(carry < a.max_tokens ? carry : a.max_tokens);
    bad |= carry > a.max_tokens;
    __syncthreads();
    // pages needed: below 2^31 in all unless the free list is short of them anyway
    const int32_t head = max(0, min(*a.free_head, a.num_free));
    bad |= head != *a.free_head;
    const int32_t left = a.num_free - head;
    carry = 0;
    for (int r0 = 0; r0 < R; r0 += kPlanThreads) {
        const int r = r0 + tid;
        int64_t need = 0;
        if (r < R) {
            const int64_t c = ctx[r], n = cu[r + 1] - cu[r];
            need = ((c + n + P - 1) >> shift) - ((c + P - 1) >> shift);
        }
        int64_t total;
        const int64_t ex = carry + block_scan_i64(need, wsum, &total);
        // saturated one above what the list can serve: such a request is not served
        const int64_t lim = static_cast<int64_t>(left) + 1;
        if (r < R) {
            before[r] = static_cast<int32_t>(ex < lim ? ex : lim);
            missing |= need > 0 && ex + need > left;
        }
        carry += total;
    }
    if (tid == 0) before[R] = static_cast<int32_t>(carry < left + int64_t(1) ? carry : left + int64_t(1));
    __syncthreads();

    auto need_of = [&](int r) {
        const int64_t c = ctx[r], n = cu[r + 1] - cu[r];
        return static_cast<int32_t>(((c + n + P - 1) >> shift) - ((c + P - 1) >> shift));
    };
    auto served = [&](int r, int32_t need) { return need == 0 || static_cast<int64_t>(before[r]) + need <= left; };

    const int64_t gid = static_cast<int64_t>(blockIdx.x) * kPlanThreads + tid;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kPlanThreads;
    // per request
    int32_t taken = 0;
    for (int r = tid; r < R; r += kPlanThreads) {
        const int32_t need = need_of(r);
        const bool ok = served(r, need);
        if (ok) taken += need;
        if (r % gridDim.x == blockIdx.x) {
            a.cu_new[r] = cu[r];
            a.kv_len[r] = ok ? ctx[r] + cu[r + 1] - cu[r] : 0;
        }
    }
    if (blockIdx.x == 0) {
        int64_t total;
        block_scan_i64(taken, wsum, &total);
        if (tid == 0) {
            a.cu_new[R] = cu[R];
            *a.free_head_out = head + static_cast<int32_t>(total);
        }
    }
    // new table entries: entry e is one of the pages the served requests take
    const int64_t entries = before[R] < left ? before[R] : left;
    for (int64_t e = gid; e < entries; e += stride) {
        const int r = last_le(before, R, static_cast<int32_t>(e));
        const int32_t need = need_of(r);
        if (!served(r, need)) continue;
        const int64_t col = ((static_cast<int64_t>(ctx[r]) + P - 1) >> shift) + (e - before[r]);
        a.block_table[r * a.table_stride + col] = a.free_pages[head + e];
    }
    // tokens
    const int32_t tokens = cu[R];
    int bad_page = 0;
    for (int64_t t = gid; t < a.max_tokens; t += stride) {
        int32_t slot = -1, pos = -1, id = -1;
        if (t < tokens) {
            const int r = last_le(cu, R, static_cast<int32_t>(t));
            pos = ctx[r] + static_cast<int32_t>(t) - cu[r];
            if (a.req_adapter) id = a.req_adapter[r];
            if (served(r, need_of(r))) {
                const int32_t j = pos >> shift;
                const int32_t have = static_cast<int32_t>((static_cast<int64_t>(ctx[r]) + P - 1) >> shift);
                const int32_t page = j >= have ? a.free_pages[head + before[r] + (j - have)]
                                               : a.block_table[r * a.table_stride + j];
                if (page >= 0 && page < a.num_pages) slot = (page << shift) + (pos & (P - 1));
                else bad_page = 1;
            }
        }
        a.slot_map[t] = slot;
        a.position[t] = pos;
        if (a.lora_id_map) a.lora_id_map[t] = id;
    }
    const int flags = (bad ? LORA_DEV_BAD_LENGTH : 0) | (missing ? LORA_DEV_NO_PAGE : 0) |
                      (bad_page ? LORA_DEV_BAD_PAGE : 0);
    if (flags) atomicOr(prm.status, flags);
}

cudaError_t launch_kv_plan(const KvPlanParams &p, cudaStream_t stream)
{
    const size_t smem = (3 * static_cast<size_t>(p.a.num_requests) + 2) * 4;
    if (smem > 49152) {   // only near LORA_MAX_REQUESTS
        const cudaError_t e = cudaFuncSetAttribute(kv_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (3 * LORA_MAX_REQUESTS + 2) * 4);
        if (e != cudaSuccess) return e;
    }
    int64_t ctas = (p.a.max_tokens + kPlanTokens - 1) / kPlanTokens;
    const int64_t cap = num_sms_current_device();
    ctas = ctas < 1 ? 1 : ctas > cap ? cap : ctas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    pdl_attribute(cfg, at);
    return cudaLaunchKernelEx(&cfg, kv_plan_kernel, p);
}

// ---------------------------------------------------------------------------
// lora_kv_store
// ---------------------------------------------------------------------------
// A copy: 16-byte units of K and V, each thread one unit of both at a time, so
// two loads are in flight; consecutive threads take consecutive units of a
// head, then of a token.  HBM (or L2, for rows just written) bounds it.
constexpr int kStoreThreads = 256;

__global__ void __launch_bounds__(kStoreThreads) kv_store_kernel(const KvStoreParams p)
{
    pdl_launch_dependents();
    pdl_wait();
    const int per = p.kv_heads * p.vecs;
    const int64_t total = p.T * per;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kStoreThreads;
    int bad = 0;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kStoreThreads + threadIdx.x; i < total; i += stride) {
        const int64_t t = i / per;
        const int u = static_cast<int>(i - t * per), h = u / p.vecs, c = u - h * p.vecs;
        const int32_t slot = p.slot_map[t];
        if (slot < 0 || slot >= p.slots) {
            bad |= slot != -1;
            continue;
        }
        const int64_t page = slot >> p.page_shift, line = slot & ((1 << p.page_shift) - 1);
        const int64_t dst = page * p.page_stride + h * p.head_stride + line * p.slot_stride + c * 8;
        const uint4 kv = *reinterpret_cast<const uint4 *>(p.k + t * p.k_tok + h * p.k_head + c * 8);
        const uint4 vv = *reinterpret_cast<const uint4 *>(p.v + t * p.v_tok + h * p.v_head + c * 8);
        *reinterpret_cast<uint4 *>(p.kc + dst) = kv;
        *reinterpret_cast<uint4 *>(p.vc + dst) = vv;
    }
    if (bad) atomicOr(p.status, LORA_DEV_BAD_PAGE);
}

cudaError_t launch_kv_store(const KvStoreParams &p, cudaStream_t stream)
{
    const int64_t total = p.T * p.kv_heads * p.vecs;
    int64_t ctas = (total + kStoreThreads - 1) / kStoreThreads;
    const int64_t cap = 8ll * num_sms_current_device();
    if (ctas > cap) ctas = cap;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kStoreThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    pdl_attribute(cfg, at);
    return cudaLaunchKernelEx(&cfg, kv_store_kernel, p);
}

}  // namespace lora
