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
// A few hundred KB at most: latency bounds it.  So it is one launch without any
// exchange between CTAs: every CTA scans all lengths (at most 4096, in shared
// memory, a run of consecutive requests a thread) for itself, then takes its
// share of the tokens and of the new table entries.  A token whose page is new
// in this call computes the page from the scan instead of reading the table that
// another CTA may be writing.  One or two tokens a thread: a token costs a
// search of its request (ten dependent shared loads for 777 requests), and with
// eight a thread those searches were most of the time (13.7 us for 38 K tokens; 7.5 us
// now).  256 requests of one token: 4.8 us, the launch and two dependent scans.
constexpr int kPlanThreads = 256;
constexpr int kPlanTokens = 512;   // tokens of a CTA, more only when all SMs have some

__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(const KvPlanParams prm)
{
    pdl_launch_dependents();
    const lora_kv_plan_t &a = prm.a;
    extern __shared__ int64_t sm[];   // all of the kernel's shared memory (plan_shared)
    const int R = a.num_requests;
    int64_t *wsum = sm;            // [32] of the block scans
    int32_t *cu = reinterpret_cast<int32_t *>(sm + 32);   // [R + 1] new tokens of a request, then the offsets
    int32_t *before = cu + R + 1;  // [R + 1] pages needed by the requests before r
    int32_t *ctx = before + R + 1; // [R]
    const int tid = threadIdx.x;
    const int P = a.page_size, shift = __ffs(P) - 1;
    const int64_t cap = static_cast<int64_t>(a.table_width) << shift;
    const int run = (R + kPlanThreads - 1) / kPlanThreads, r0 = min(R, tid * run), r1 = min(R, r0 + run);
    pdl_wait();

    const int32_t head0 = *a.free_head;
    int bad = 0, missing = 0;
#pragma unroll 4
    for (int r = tid; r < R; r += kPlanThreads) {
        const int n0 = a.new_len[r], c0 = a.ctx_len[r];
        const int64_t c = c0 < 0 ? 0 : c0 > cap ? cap : c0;
        const int64_t n = n0 < 0 ? 0 : n0 > cap - c ? cap - c : n0;
        bad |= (c != c0) | (n != n0);
        ctx[r] = static_cast<int32_t>(c);
        cu[r] = static_cast<int32_t>(n);
    }
    __syncthreads();
    // packed offsets: at most max_tokens in all
    int64_t sum = 0, total;
    for (int r = r0; r < r1; ++r) sum += cu[r];
    int64_t at = block_scan_i64(sum, wsum, &total);
    for (int r = r0; r < r1; ++r) {
        const int32_t n = cu[r];
        cu[r] = static_cast<int32_t>(at < a.max_tokens ? at : a.max_tokens);
        at += n;
    }
    if (tid == 0) cu[R] = static_cast<int32_t>(total < a.max_tokens ? total : a.max_tokens);
    bad |= total > a.max_tokens;
    __syncthreads();
    // pages needed, saturated one above what the list can serve: such a request is not served
    const int32_t head = max(0, min(head0, a.num_free));
    bad |= head != head0;
    const int32_t left = a.num_free - head;
    const int64_t lim = static_cast<int64_t>(left) + 1;
    auto need_of = [&](int r) {
        const int64_t c = ctx[r], n = cu[r + 1] - cu[r];
        return static_cast<int32_t>(((c + n + P - 1) >> shift) - ((c + P - 1) >> shift));
    };
    sum = 0;
    for (int r = r0; r < r1; ++r) sum += need_of(r);
    at = block_scan_i64(sum, wsum, &total);
    for (int r = r0; r < r1; ++r) {
        const int32_t need = need_of(r);
        before[r] = static_cast<int32_t>(at < lim ? at : lim);
        missing |= need > 0 && at + need > left;
        at += need;
    }
    if (tid == 0) before[R] = static_cast<int32_t>(total < lim ? total : lim);
    __syncthreads();

    auto served = [&](int r, int32_t need) { return need == 0 || static_cast<int64_t>(before[r]) + need <= left; };

    const int64_t gid = static_cast<int64_t>(blockIdx.x) * kPlanThreads + tid;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kPlanThreads;
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
    // per request
    for (int64_t r = gid; r < R; r += stride) {
        const int i = static_cast<int>(r);
        a.cu_new[i] = cu[i];
        a.kv_len[i] = served(i, need_of(i)) ? ctx[i] + cu[i + 1] - cu[i] : 0;
    }
    // new table entries: entry e is one of the pages the served requests take
    const int64_t entries = before[R] < left ? before[R] : left;
    for (int64_t e = gid; e < entries; e += stride) {
        const int r = last_le(before, R, static_cast<int32_t>(e));
        if (!served(r, need_of(r))) continue;
        const int64_t col = ((static_cast<int64_t>(ctx[r]) + P - 1) >> shift) + (e - before[r]);
        a.block_table[r * a.table_stride + col] = a.free_pages[head + e];
    }
    if (blockIdx.x == 0) {
        int64_t taken = 0;
        for (int r = r0; r < r1; ++r) {
            const int32_t need = need_of(r);
            if (served(r, need)) taken += need;
        }
        block_scan_i64(taken, wsum, &total);
        if (tid == 0) {
            a.cu_new[R] = cu[R];
            *a.free_head_out = head + static_cast<int32_t>(total);
        }
    }
    const int flags = (bad ? LORA_DEV_BAD_LENGTH : 0) | (missing ? LORA_DEV_NO_PAGE : 0) |
                      (bad_page ? LORA_DEV_BAD_PAGE : 0);
    if (flags) atomicOr(prm.status, flags);
}

// Bytes of shared memory for R requests.  The kernel has no other: a launch's limit of 48 KB
// without opting in is on static and dynamic memory together.
static constexpr size_t plan_shared(int R) { return 32 * sizeof(int64_t) + (3 * static_cast<size_t>(R) + 2) * 4; }

cudaError_t launch_kv_plan(const KvPlanParams &p, cudaStream_t stream)
{
    const size_t smem = plan_shared(p.a.num_requests);
    if (smem > 49152) {   // only near LORA_MAX_REQUESTS
        const cudaError_t e = cudaFuncSetAttribute(kv_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(plan_shared(LORA_MAX_REQUESTS)));
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
// A copy: 16-byte units of K and V, consecutive threads taking consecutive units
// of a head, then of a token.  HBM (or L2, for rows just written) bounds it, so a
// thread has the four loads of two units in flight, and its slots with them,
// before it stores anything.  7300 tokens of 8 heads of 128 (59.5 MB moved): 11.3 us,
// 5.3 TB/s (11.5 us with one unit a thread); 32 tokens: 1.7 us.
constexpr int kStoreThreads = 256;
constexpr int kStoreUnits = 2;

__global__ void __launch_bounds__(kStoreThreads) kv_store_kernel(const KvStoreParams p)
{
    pdl_launch_dependents();
    pdl_wait();
    const uint32_t per = static_cast<uint32_t>(p.kv_heads * p.vecs);
    const int64_t total = p.T * per;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kStoreThreads;
    int bad = 0;
    for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * kStoreThreads + threadIdx.x; i0 < total;
         i0 += kStoreUnits * stride) {
        uint4 kv[kStoreUnits], vv[kStoreUnits];
        int32_t slot[kStoreUnits];
        int64_t to[kStoreUnits];
#pragma unroll
        for (int q = 0; q < kStoreUnits; ++q) {
            const int64_t i = i0 + q * stride;
            slot[q] = -1;
            if (i >= total) continue;
            const int64_t t = total < (int64_t(1) << 32) ? static_cast<uint32_t>(i) / per : i / per;
            const int u = static_cast<int>(i - t * per), h = u / p.vecs, c = u - h * p.vecs;
            slot[q] = p.slot_map[t];
            kv[q] = *reinterpret_cast<const uint4 *>(p.k + t * p.k_tok + h * p.k_head + c * 8);
            vv[q] = *reinterpret_cast<const uint4 *>(p.v + t * p.v_tok + h * p.v_head + c * 8);
            to[q] = h * p.head_stride + c * 8;
        }
#pragma unroll
        for (int q = 0; q < kStoreUnits; ++q) {
            if (slot[q] < 0 || slot[q] >= p.slots) {
                bad |= slot[q] != -1;
                continue;
            }
            const int64_t page = slot[q] >> p.page_shift, line = slot[q] & ((1 << p.page_shift) - 1);
            const int64_t dst = page * p.page_stride + line * p.slot_stride + to[q];
            *reinterpret_cast<uint4 *>(p.kc + dst) = kv[q];
            *reinterpret_cast<uint4 *>(p.vc + dst) = vv[q];
        }
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
