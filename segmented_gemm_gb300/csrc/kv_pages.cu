// Sharing, freeing, moving and copying of pages (include/lora_kv.h):
// lora_kv_release, lora_kv_fork, lora_kv_compact, lora_kv_copy, lora_kv4_copy.
//
// All but the copies touch a few hundred KB at most: latency bounds them, the number
// of dependent launches above all.  Counts go by integer atomics, and lists
// are in ascending or given order, so the outcome does not depend on timing.
#include <cuda_runtime.h>

#include "block_scan.cuh"
#include "kv_ops.h"
#include "internal.h"
#include "ptx.cuh"

namespace lora {

namespace {

constexpr int kThreads = 256;
constexpr int kPerThread = kPageChunk / kThreads;   // pages of a thread in the passes over all pages

// Pages that row r holds, clamped to its table row.
__device__ __forceinline__ int held_pages(const lora_kv_pages_t &a, int len, int *flags)
{
    const int64_t cap = static_cast<int64_t>(a.table_width) * a.page_size;
    const int64_t n = len < 0 ? 0 : len > cap ? cap : len;
    if (n != len) *flags |= LORA_DEV_BAD_LENGTH;
    return static_cast<int>((n + a.page_size - 1) / a.page_size);
}

__device__ __forceinline__ int4 add4(int4 a, int4 b) { return make_int4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w); }

// Sum of the chunks' counts before chunk `to`, and of all of them, by the whole block.
__device__ __forceinline__ int4 sum_counts(const KvPagesParams &p, int chunks, int to, int4 *all, int4 *sm /* [2] */)
{
    if (threadIdx.x < 2) sm[threadIdx.x] = make_int4(0, 0, 0, 0);
    __syncthreads();
    int4 a = make_int4(0, 0, 0, 0), b = a;
    for (int i = threadIdx.x; i < chunks; i += kThreads) {
        const int4 c = __ldcg(p.counts(i));
        a = add4(a, c);
        if (i < to) b = add4(b, c);
    }
    int *s = reinterpret_cast<int *>(sm);
    const int v[8] = {b.x, b.y, b.z, b.w, a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int w = __reduce_add_sync(0xffffffffu, v[i]);
        if ((threadIdx.x & 31) == 0 && w) atomicAdd(s + i, w);
    }
    __syncthreads();
    *all = sm[1];
    return sm[0];
}

// ---------------------------------------------------------------------------
// lora_kv_release
// ---------------------------------------------------------------------------
// A page of holders ref + 1 that d released rows name is free iff d > ref, whatever
// the order: the rows' entries subtract, then a pass over all pages finds the negative
// counts.  Three launches: subtract, count (a chunk of pages a CTA), list.
__global__ void __launch_bounds__(kThreads) release_rows_kernel(const KvPagesParams p)
{
    pdl_launch_dependents();
    const lora_kv_pages_t &a = p.a;
    pdl_wait();
    int flags = 0;
    for (int i = blockIdx.x; i < p.num; i += gridDim.x) {
        const int r = p.rows[i];
        int skip = r < 0 || r >= a.num_rows;
        for (int j = threadIdx.x; j < i && !skip; j += kThreads) skip = p.rows[j] == r;   // named before
        if (__syncthreads_or(skip)) {
            flags |= LORA_DEV_BAD_ROW;
            continue;
        }
        const int n = held_pages(a, a.ctx_len[r], &flags);
        for (int j = threadIdx.x; j < n; j += kThreads) {
            const int page = a.block_table[r * a.table_stride + j];
            if (page >= 0 && page < a.num_pages) atomicSub(a.ref + page, 1);
            else flags |= LORA_DEV_BAD_PAGE;
        }
        __syncthreads();   // everybody has read the length
        if (threadIdx.x == 0) a.ctx_len[r] = 0;
    }
    if (flags) atomicOr(p.counters, flags);
}

__global__ void __launch_bounds__(kThreads) release_count_kernel(const KvPagesParams p)
{
    pdl_launch_dependents();
    __shared__ int sum;
    const lora_kv_pages_t &a = p.a;
    if (threadIdx.x == 0) sum = 0;
    __syncthreads();
    pdl_wait();
    const int64_t base = static_cast<int64_t>(blockIdx.x) * kPageChunk + threadIdx.x;
    int n = 0;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int64_t page = base + i * kThreads;
        n += page < a.num_pages && a.ref[page] < 0;
    }
    n = __reduce_add_sync(0xffffffffu, n);
    if ((threadIdx.x & 31) == 0 && n) atomicAdd(&sum, n);
    __syncthreads();
    if (threadIdx.x == 0) *p.counts(blockIdx.x) = make_int4(sum, 0, 0, 0);
}

__global__ void __launch_bounds__(kThreads) release_list_kernel(const KvPagesParams p)
{
    pdl_launch_dependents();
    __shared__ int4 sm[2];
    __shared__ int64_t scan[32];
    const lora_kv_pages_t &a = p.a;
    pdl_wait();
    int4 all;
    const int before = sum_counts(p, gridDim.x, blockIdx.x, &all, sm).x;
    const int head0 = *a.free_head, head = max(0, min(head0, a.num_free)), first = max(0, head - all.x);
    const int64_t base = static_cast<int64_t>(blockIdx.x) * kPageChunk + threadIdx.x * kPerThread;
    uint32_t freed = 0;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i)
        if (base + i < a.num_pages && a.ref[base + i] < 0) freed |= 1u << i;
    int64_t total;
    int at = first + before + static_cast<int>(block_scan_i64(__popc(freed), scan, &total));
    for (; freed; freed &= freed - 1) {
        const int page = static_cast<int>(base) + __ffs(freed) - 1;
        a.ref[page] = 0;
        if (at < head) a.free_pages[at] = page;
        ++at;
    }
    // every CTA reads the old head; the last one done writes the new one
    __shared__ int done;
    __syncthreads();
    if (threadIdx.x == 0) done = atom_acq_rel_gpu_add(p.counters + kPagesArrived, 1);
    __syncthreads();
    if (done == static_cast<int>(gridDim.x) - 1 && threadIdx.x == 0) {
        p.counters[kPagesArrived] = 0;
        *a.free_head = first;
        const int flags = (head != head0 ? LORA_DEV_BAD_LENGTH : 0) | (all.x > head ? LORA_DEV_NO_PAGE : 0);
        if (flags) atomicOr(p.counters, flags);
    }
}

// For caches of up to kSmallPages one CTA counts and lists, 32 pages a thread; and takes the rows before, a
// warp each, where these are few (ROWS): one launch.  8 rows of 49 pages 4 us so, 192 of up to 94
// pages 15, 10 by a launch of their own for the rows.
constexpr int kSmallThreads = 1024, kSmallPages = 32 * kSmallThreads, kSmallEntries = 4096;

template <bool ROWS>
__global__ void __launch_bounds__(kSmallThreads) release_small_kernel(const KvPagesParams p)
{
    pdl_launch_dependents();
    __shared__ uint32_t named[LORA_MAX_REQUESTS / 32];
    __shared__ int64_t scan[32];
    const lora_kv_pages_t &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31;
    if (ROWS)
        for (int i = tid; i < LORA_MAX_REQUESTS / 32; i += kSmallThreads) named[i] = 0;
    __syncthreads();
    pdl_wait();
    const int head0 = *a.free_head, head = max(0, min(head0, a.num_free));
    int flags = head != head0 ? LORA_DEV_BAD_LENGTH : 0;
    for (int i = ROWS ? tid >> 5 : p.num; i < p.num; i += kSmallThreads / 32) {
        const int r = p.rows[i];
        bool skip = r < 0 || r >= a.num_rows;
        if (!skip) {
            uint32_t old = 0;
            if (lane == 0) old = atomicOr(named + r / 32, 1u << (r % 32));
            skip = __shfl_sync(0xffffffffu, old, 0) >> (r % 32) & 1;   // by another i; which one does not matter
        }
        if (skip) {
            flags |= LORA_DEV_BAD_ROW;
            continue;
        }
        const int n = held_pages(a, a.ctx_len[r], &flags);
        for (int j = lane; j < n; j += 32) {
            const int page = a.block_table[r * a.table_stride + j];
            if (page >= 0 && page < a.num_pages) atomicSub(a.ref + page, 1);
            else flags |= LORA_DEV_BAD_PAGE;
        }
        __syncwarp();
        if (lane == 0) a.ctx_len[r] = 0;
    }
    __syncthreads();
    const int each = (a.num_pages + kSmallThreads - 1) / kSmallThreads, base = tid * each;
    uint32_t freed = 0;
#pragma unroll 8
    for (int i = 0; i < each; ++i)
        if (base + i < a.num_pages && __ldcg(a.ref + base + i) < 0) freed |= 1u << i;
    int64_t total;
    const int64_t before = block_scan_i64(__popc(freed), scan, &total);
    const int first = max(0, head - static_cast<int>(total));
    int at = first + static_cast<int>(before);
    for (; freed; freed &= freed - 1) {
        const int page = base + __ffs(freed) - 1;
        a.ref[page] = 0;
        if (at < head) a.free_pages[at] = page;
        ++at;
    }
    if (tid == 0) {
        *a.free_head = first;
        if (total > head) flags |= LORA_DEV_NO_PAGE;
    }
    if (flags) atomicOr(p.counters, flags);
}

// ---------------------------------------------------------------------------
// lora_kv_fork
// ---------------------------------------------------------------------------
// One launch: every CTA checks all forks and scans the pages they need for itself, then
// takes its share of the forks.  192 forks of up to 94 pages 4.3 us, 8 of 49 3.6: four dependent passes.
constexpr size_t fork_shared(int num, int rows)
{
    return 32 * sizeof(int64_t) + (static_cast<size_t>(num) + 1 + rows + (rows + 31) / 32) * 4;
}

__global__ void __launch_bounds__(kThreads) fork_kernel(const KvPagesParams p)
{
    pdl_launch_dependents();
    extern __shared__ int64_t smem[];
    int64_t *scan = smem;                                      // [32]
    int32_t *before = reinterpret_cast<int32_t *>(smem + 32);  // [num + 1] pages needed by the forks before i
    int32_t *first = before + p.num + 1;                       // [num_rows] the first fork that names a row as a child
    uint32_t *is_parent = reinterpret_cast<uint32_t *>(first + p.a.num_rows);   // [num_rows] bits
    const lora_kv_pages_t &a = p.a;
    const int tid = threadIdx.x, shift = __ffs(a.page_size) - 1;
    for (int i = tid; i < a.num_rows; i += kThreads) first[i] = p.num;
    for (int i = tid; i < (a.num_rows + 31) / 32; i += kThreads) is_parent[i] = 0;
    __syncthreads();
    pdl_wait();
    const int head0 = *a.free_head, head = max(0, min(head0, a.num_free)), left = a.num_free - head;
    auto known = [&](int r) { return r >= 0 && r < a.num_rows; };
    for (int i = tid; i < p.num; i += kThreads) {
        const int f = p.parent[i], c = p.child[i];
        if (!known(f) || !known(c)) continue;
        atomicMin(first + c, i);
        atomicOr(is_parent + f / 32, 1u << (f % 32));
    }
    __syncthreads();
    auto valid = [&](int i, int f, int c) {
        return known(f) && known(c) && first[c] == i && !(is_parent[c / 32] >> (c % 32) & 1);
    };
    const int64_t cap = static_cast<int64_t>(a.table_width) << shift;
    auto length = [&](int f) {
        const int n = a.ctx_len[f];
        return static_cast<int>(n < 0 ? 0 : n > cap ? cap : n);
    };
    // need of a fork: 0 or 1 page, 2 marks one that is skipped
    for (int i = tid; i < p.num; i += kThreads) {
        const int f = p.parent[i], c = p.child[i];
        before[i] = !valid(i, f, c) ? 2 : (length(f) & (a.page_size - 1)) != 0;
    }
    __syncthreads();
    const int run = (p.num + kThreads - 1) / kThreads, i0 = min(p.num, tid * run), i1 = min(p.num, i0 + run);
    int64_t sum = 0, total;
    for (int i = i0; i < i1; ++i) sum += before[i] & 1;
    int at = static_cast<int>(block_scan_i64(sum, scan, &total));
    for (int i = i0; i < i1; ++i) {
        const int need = before[i];
        before[i] = 4 * at + need;
        at += need & 1;
    }
    __syncthreads();

    int flags = 0;
    for (int i = blockIdx.x; i < p.num; i += gridDim.x) {
        const int need = before[i] & 3, place = before[i] >> 2;
        if (need == 2) {
            flags |= LORA_DEV_BAD_ROW;
            if (tid == 0) p.src[i] = p.dst[i] = -1;
            continue;
        }
        const int f = p.parent[i], c = p.child[i], n = length(f), whole = n >> shift;
        if (n != a.ctx_len[f]) flags |= LORA_DEV_BAD_LENGTH;
        const bool served = need == 0 || place < left;
        int32_t *to = a.block_table + c * a.table_stride;
        const int32_t *from = a.block_table + f * a.table_stride;
        if (!served) flags |= LORA_DEV_NO_PAGE;
        for (int j = tid; j < whole && served; j += kThreads) {
            const int page = from[j];
            to[j] = page;
            if (page >= 0 && page < a.num_pages) atomicAdd(a.ref + page, 1);
            else flags |= LORA_DEV_BAD_PAGE;
        }
        if (tid == 0) {
            int old = -1, fresh = -1;
            if (need && served) {
                auto page_or_none = [&](int page) {
                    if (page >= 0 && page < a.num_pages) return page;
                    flags |= LORA_DEV_BAD_PAGE;
                    return -1;
                };
                old = page_or_none(from[whole]);
                to[whole] = fresh = page_or_none(a.free_pages[head + place]);
            }
            const bool pair = old >= 0 && fresh >= 0;
            p.src[i] = pair ? old : -1;
            p.dst[i] = pair ? fresh : -1;
            a.ctx_len[c] = served ? n : 0;
        }
    }
    flags |= head != head0 ? LORA_DEV_BAD_LENGTH : 0;
    if (flags) atomicOr(p.counters, flags);
    // every CTA reads the old head; the last one done writes the new one
    __syncthreads();
    if (tid == 0 && atom_acq_rel_gpu_add(p.counters + kPagesArrived, 1) == static_cast<int>(gridDim.x) - 1) {
        p.counters[kPagesArrived] = 0;
        *a.free_head = head + static_cast<int>(total < left ? total : left);
    }
}

// ---------------------------------------------------------------------------
// lora_kv_compact
// ---------------------------------------------------------------------------
// Four launches: mark the pages held and free; count, a chunk of pages a CTA, the free ones
// below the limit (holes), the held ones from it on (movers) and the free ones from it on;
// list: with the counts before a chunk, every page's place among its kind is known, so
// the pairs and the new free list are written in one pass; and the tables follow.
__global__ void __launch_bounds__(kThreads) compact_mark_kernel(const KvPagesParams p)
{
    pdl_launch_dependents();
    const lora_kv_pages_t &a = p.a;
    pdl_wait();
    int flags = 0;
    for (int r = blockIdx.x; r < a.num_rows; r += gridDim.x) {
        const int n = held_pages(a, a.ctx_len[r], &flags);
        for (int j = threadIdx.x; j < n; j += kThreads) {
            const int page = a.block_table[r * a.table_stride + j];
            if (page >= 0 && page < a.num_pages) *p.used(page) = 1;
            else flags |= LORA_DEV_BAD_PAGE;
        }
    }
    const int head0 = *a.free_head, head = max(0, min(head0, a.num_free));
    flags |= head != head0 ? LORA_DEV_BAD_LENGTH : 0;
    for (int64_t i = head + static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < a.num_free;
         i += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int page = a.free_pages[i];
        if (page >= 0 && page < a.num_pages) *p.free(page) = 1;
        else flags |= LORA_DEV_BAD_PAGE;
    }
    if (flags) atomicOr(p.counters, flags);
}

// What a page is, of its marks: bit 0 a hole, bit 8 a mover, bit 16 free from the limit on (so that 16 of a thread add up without carries).
__device__ __forceinline__ uint32_t kind_of(bool held, bool listed, bool high, int *both)
{
    *both |= held && listed;
    return held ? (high ? 1u << 8 : 0u) : listed ? (high ? 1u << 16 : 1u) : 0u;
}

__global__ void __launch_bounds__(kThreads) compact_count_kernel(const KvPagesParams p)
{
    pdl_launch_dependents();
    __shared__ int sum[3];
    if (threadIdx.x < 3) sum[threadIdx.x] = 0;
    __syncthreads();
    pdl_wait();
    const int64_t base = static_cast<int64_t>(blockIdx.x) * kPageChunk + threadIdx.x;
    const uint8_t *used = p.used(base), *free = p.free(base);   // a chunk's marks are consecutive
    uint32_t n = 0;
    int both = 0;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int64_t page = base + i * kThreads;
        if (page < p.a.num_pages) n += kind_of(used[i * kThreads], free[i * kThreads], page >= p.limit, &both);
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const int w = __reduce_add_sync(0xffffffffu, static_cast<int>(n >> (8 * i) & 0xFF));
        if ((threadIdx.x & 31) == 0 && w) atomicAdd(sum + i, w);
    }
    __syncthreads();
    if (threadIdx.x == 0) *p.counts(blockIdx.x) = make_int4(sum[0], sum[1], sum[2], 0);
    if (both) atomicOr(p.counters, LORA_DEV_BAD_PAGE);
}

__global__ void __launch_bounds__(kThreads) compact_list_kernel(const KvPagesParams p)
{
    pdl_launch_dependents();
    __shared__ int4 sm[2];
    __shared__ int64_t scan[32];
    const lora_kv_pages_t &a = p.a;
    pdl_wait();
    int4 all;
    const int4 before = sum_counts(p, gridDim.x, blockIdx.x, &all, sm);
    const int moved = min(min(all.x, all.y), p.max_copies);
    const int first = a.num_free - (all.x + all.z);          // the new head: as many are free as before
    const int64_t base = static_cast<int64_t>(blockIdx.x) * kPageChunk + threadIdx.x * kPerThread;
    uint8_t *used = p.used(base), *free = p.free(base);
    int32_t *map = p.map(base);
    uint32_t kind[kPerThread], n = 0;
    int both = 0;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        kind[i] = base + i < a.num_pages ? kind_of(used[i], free[i], base + i >= p.limit, &both) : 0u;
        n += kind[i];
    }
    int64_t total;
    const int64_t packed = (n & 0xFF) | static_cast<int64_t>(n >> 8 & 0xFF) << 20 | static_cast<int64_t>(n >> 16 & 0xFF) << 40;
    const int64_t at = block_scan_i64(packed, scan, &total);
    int hole = before.x + static_cast<int>(at & 0xFFFFF), mover = before.y + static_cast<int>(at >> 20 & 0xFFFFF);
    int high = before.z + static_cast<int>(at >> 40);
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int64_t page = base + i;
        if (page >= a.num_pages) break;
        const int32_t id = static_cast<int32_t>(page);
        int32_t to = 0;
        bool pair = false;                                   // its count is the other one's, or 0
        if (kind[i] & 1) {
            pair = hole < moved;
            if (pair) p.dst[hole] = id;
            else p.free_out[first + hole - moved] = id;
            ++hole;
        } else if (kind[i] & (1u << 8)) {
            pair = mover < moved;
            if (pair) {
                p.src[mover] = id;
                to = mover + 1;
                p.free_out[first + (all.x - moved) + high + mover] = id;
            }
            ++mover;
        } else if (kind[i]) {
            p.free_out[first + (all.x - moved) + high + min(mover, moved)] = id;
            ++high;
        }
        map[i] = to;
        if (!pair && p.ref_out != a.ref) p.ref_out[page] = a.ref[page];
        used[i] = free[i] = 0;
    }
    for (int64_t i = moved + static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < p.max_copies;
         i += static_cast<int64_t>(gridDim.x) * kThreads)
        p.src[i] = p.dst[i] = -1;
}

__global__ void __launch_bounds__(kThreads) compact_tables_kernel(const KvPagesParams p)
{
    pdl_launch_dependents();
    __shared__ int4 sm[2];
    const lora_kv_pages_t &a = p.a;
    pdl_wait();
    int4 all;
    const int chunks = (a.num_pages + kPageChunk - 1) / kPageChunk;
    sum_counts(p, chunks, 0, &all, sm);
    const int moved = min(min(all.x, all.y), p.max_copies), first = a.num_free - (all.x + all.z);
    const bool in_place = p.table_out == a.block_table;
    int flags = 0;
    for (int r = blockIdx.x; r < a.num_rows; r += gridDim.x) {
        const int n = held_pages(a, a.ctx_len[r], &flags);
        for (int j = threadIdx.x; j < (in_place ? n : a.table_width); j += kThreads) {
            int page = a.block_table[r * a.table_stride + j];
            if (j < n && page >= 0 && page < a.num_pages) {
                const int m = *p.map(page);
                if (m) page = p.dst[m - 1];
            }
            p.table_out[r * a.table_stride + j] = page;
        }
    }
    const int64_t gid = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads;
    for (int64_t i = gid; i < moved; i += stride) {
        const int src = p.src[i], n = a.ref[src];
        p.ref_out[p.dst[i]] = n;
        p.ref_out[src] = 0;
    }
    if (p.free_out != a.free_pages)
        for (int64_t i = gid; i < first; i += stride) p.free_out[i] = a.free_pages[i];
    if (gid == 0) *p.head_out = first;
}

// The same in one launch, for small caches: the CTAs of a cluster mark the pages in shared memory, every one takes
// all CTAs' marks together and counts for itself, and they share what is to be written.  7554 pages of 90
// rows 8.7 us by eight CTAs, 12.3 by four launches; 94 pages of 5 rows 7 by eight and 4.3 by one; with 32768 pages and
// as many entries eight CTAs and four launches take the same 14.
constexpr int64_t kClusterEntries = 1 << 15;
constexpr int32_t kSmallList = 4 * kSmallPages;   // longest lists: a CTA goes through them with 32-bit places
constexpr int kClusterCtas = 8;

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// *mine of CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t of_rank(const uint32_t *mine, uint32_t rank)
{
    uint32_t at, v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(mine)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

struct CompactShared {
    uint32_t used[kSmallThreads], free[kSmallThreads];                           // this CTA's marks, a bit a page
    uint32_t hole[kSmallThreads], mover[kSmallThreads], high[kSmallThreads];     // all CTAs'
    int64_t before[kSmallThreads], scan[32];   // holes, movers and high ones in the words before, 20 bits each
    uint16_t to[kSmallPages / 2];              // where a mover goes: no more than half of the pages do
};

template <int CTAS>
__global__ void __cluster_dims__(CTAS, 1, 1) __launch_bounds__(kSmallThreads) compact_small_kernel(const KvPagesParams p)
{
    pdl_launch_dependents();
    extern __shared__ __align__(16) uint8_t shared[];
    CompactShared &s = *reinterpret_cast<CompactShared *>(shared);
    const lora_kv_pages_t &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, rank = blockIdx.x, warp = (tid >> 5) * CTAS + rank;
    constexpr int kWarps = kSmallThreads / 32 * CTAS, kAll = kSmallThreads * CTAS;   // the cluster's
    s.used[tid] = s.free[tid] = 0;
    __syncthreads();
    pdl_wait();
    const int head0 = *a.free_head, head = max(0, min(head0, a.num_free));
    int flags = head != head0 ? LORA_DEV_BAD_LENGTH : 0;
    for (int r = warp; r < a.num_rows; r += kWarps) {
        const int n = held_pages(a, a.ctx_len[r], &flags);
#pragma unroll 4
        for (int j = lane; j < n; j += 32) {
            const int page = a.block_table[r * a.table_stride + j];
            if (page >= 0 && page < a.num_pages) atomicOr(s.used + page / 32, 1u << (page % 32));
            else flags |= LORA_DEV_BAD_PAGE;
        }
    }
    for (int i = head + rank * kSmallThreads + tid; i < a.num_free; i += kAll) {
        const int page = a.free_pages[i];
        if (page >= 0 && page < a.num_pages) atomicOr(s.free + page / 32, 1u << (page % 32));
        else flags |= LORA_DEV_BAD_PAGE;
    }
    uint32_t u = 0, f = 0;
    if (CTAS > 1) {
        cluster_arrive();
        cluster_wait();
#pragma unroll
        for (int c = 0; c < CTAS; ++c) {
            u |= of_rank(s.used + tid, c);
            f |= of_rank(s.free + tid, c);
        }
        cluster_arrive();   // until everybody has read the marks, nobody leaves
    } else {
        __syncthreads();
        u = s.used[tid];
        f = s.free[tid];
    }
    if (f & u) flags |= LORA_DEV_BAD_PAGE;
    f &= ~u;
    const int base = 32 * tid, below = max(0, min(32, p.limit - base));
    const uint32_t low = below == 32 ? ~0u : (1u << below) - 1, holes = f & low, movers = u & ~low, high = f & ~low;
    int64_t total;
    const int64_t before = block_scan_i64(
        __popc(holes) | static_cast<int64_t>(__popc(movers)) << 20 | static_cast<int64_t>(__popc(high)) << 40, s.scan, &total);
    const int all_holes = static_cast<int>(total & 0xFFFFF), all_movers = static_cast<int>(total >> 20 & 0xFFFFF);
    const int moved = min(min(all_holes, all_movers), p.max_copies);
    const int first = a.num_free - all_holes - static_cast<int>(total >> 40);
    s.hole[tid] = holes;
    s.mover[tid] = movers;
    s.high[tid] = high;
    s.before[tid] = before;
    int n = static_cast<int>(before & 0xFFFFF);
    for (uint32_t left = holes; left && n < moved; left &= left - 1, ++n) s.to[n] = static_cast<uint16_t>(base + __ffs(left) - 1);
    __syncthreads();

    // the list's old entries have all been read
    for (int w = warp; w < (a.num_pages + 31) / 32; w += kWarps) {
        const int page = 32 * w + lane;
        const uint32_t bit = 1u << lane, less = bit - 1;
        const int64_t at = s.before[w];
        const int hole = static_cast<int>(at & 0xFFFFF) + __popc(s.hole[w] & less);
        const int mover = static_cast<int>(at >> 20 & 0xFFFFF) + __popc(s.mover[w] & less);
        int32_t *high_out = p.free_out + first + (all_holes - moved) + static_cast<int>(at >> 40) + __popc(s.high[w] & less);
        bool pair = false;                                   // its count is the other one's, or 0
        if (s.hole[w] & bit) {
            pair = hole < moved;
            if (pair) p.dst[hole] = page;
            else p.free_out[first + hole - moved] = page;
        } else if (s.mover[w] & bit) {
            pair = mover < moved;
            if (pair) {
                p.src[mover] = page;
                high_out[mover] = page;
                p.ref_out[s.to[mover]] = a.ref[page];
                p.ref_out[page] = 0;
            }
        } else if (s.high[w] & bit) {
            high_out[min(mover, moved)] = page;
        }
        if (!pair && p.ref_out != a.ref && page < a.num_pages) p.ref_out[page] = a.ref[page];
    }
    for (int i = moved + rank * kSmallThreads + tid; i < p.max_copies; i += kAll) p.src[i] = p.dst[i] = -1;
    if (p.free_out != a.free_pages)
        for (int i = rank * kSmallThreads + tid; i < first; i += kAll) p.free_out[i] = a.free_pages[i];
    const bool in_place = p.table_out == a.block_table;
    for (int r = warp; r < a.num_rows; r += kWarps) {
        int ignored = 0;
        const int held = held_pages(a, a.ctx_len[r], &ignored);
#pragma unroll 4
        for (int j = lane; j < (in_place ? held : a.table_width); j += 32) {
            int page = a.block_table[r * a.table_stride + j];
            if (j < held && page >= 0 && page < a.num_pages && s.mover[page / 32] >> (page % 32) & 1) {
                const int i = static_cast<int>(s.before[page / 32] >> 20 & 0xFFFFF) +
                              __popc(s.mover[page / 32] & ((1u << (page % 32)) - 1));
                if (i < moved) page = s.to[i];
            }
            p.table_out[r * a.table_stride + j] = page;
        }
    }
    if (rank == 0 && tid == 0) *p.head_out = first;
    if (flags) atomicOr(p.counters, flags);
    if (CTAS > 1) cluster_wait();
}

// ---------------------------------------------------------------------------
// lora_kv_copy, lora_kv4_copy
// ---------------------------------------------------------------------------
// 16-byte units, a block a run of one page's; HBM bounds it, so a thread has eight
// loads in flight.  Lists may be mostly empty pairs (compaction pads its own), so a
// block looks at the pairs of several rounds at once.  1040 pages of 131 KB among 3777 pairs: 45 us, 6.1 TB/s
// (57 with four loads, 47 without the streaming stores).
constexpr int kCopyUnits = 8, kCopyRounds = 4;

template <bool ROWS>   // ROWS: a page's units go by head and slot strides
__global__ void __launch_bounds__(kThreads) page_copy_kernel(const PageCopyParams p)
{
    pdl_launch_dependents();
    const int units = p.heads * p.rows * p.vecs;
    const uint32_t runs = (units + kCopyUnits * kThreads - 1) / (kCopyUnits * kThreads), each = runs * (p.base[1] ? 2 : 1);
    const int64_t work = static_cast<int64_t>(p.num) * each, step = gridDim.x;
    pdl_wait();
    int bad = 0;
    for (int64_t w0 = blockIdx.x; w0 < work; w0 += kCopyRounds * step) {
        int src[kCopyRounds], dst[kCopyRounds];
        uint32_t rest[kCopyRounds];
#pragma unroll
        for (int q = 0; q < kCopyRounds; ++q) {
            const int64_t w = w0 + q * step;
            src[q] = dst[q] = -1;
            if (w >= work) continue;
            const int64_t i = work < (int64_t(1) << 32) ? static_cast<uint32_t>(w) / each : w / each;
            rest[q] = static_cast<uint32_t>(w - i * each);
            src[q] = p.src[i];
            dst[q] = p.dst[i];
        }
#pragma unroll
        for (int q = 0; q < kCopyRounds; ++q) {
            if (src[q] < 0 || dst[q] < 0 || src[q] >= p.num_pages || dst[q] >= p.num_pages) {
                bad |= src[q] != -1 || dst[q] != -1;
                continue;
            }
            const uint32_t part = rest[q] >= runs, run = rest[q] - part * runs;
            const uint4 *from = p.base[part] + src[q] * p.page_stride;
            uint4 *to = p.base[part] + dst[q] * p.page_stride;
            uint4 v[kCopyUnits];
            int64_t at[kCopyUnits];
#pragma unroll
            for (int u = 0; u < kCopyUnits; ++u) {
                const int k = (run * kCopyUnits + u) * kThreads + threadIdx.x;
                at[u] = -1;
                if (k >= units) continue;
                at[u] = k;
                if (ROWS) {
                    const int row = k / p.vecs, h = row / p.rows;
                    at[u] = h * p.head_stride + (row - h * p.rows) * p.slot_stride + (k - row * p.vecs);
                }
                v[u] = __ldcs(from + at[u]);
            }
#pragma unroll
            for (int u = 0; u < kCopyUnits; ++u)
                if (at[u] >= 0) __stcs(to + at[u], v[u]);
        }
    }
    if (bad) atomicOr(p.status, LORA_DEV_BAD_PAGE);
}

int64_t capped(int64_t n, int64_t per_sm)
{
    const int64_t cap = per_sm * num_sms_current_device();
    return n < 1 ? 1 : n < cap ? n : cap;
}

template <int CTAS>
cudaError_t launch_compact_small(const KvPagesParams &p, cudaStream_t stream)
{
    static bool configured[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
    if (dev >= 64 || !configured[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(compact_small_kernel<CTAS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   sizeof(CompactShared));
        if (e != cudaSuccess) return e;
        if (dev < 64) configured[dev] = true;
    }
    return launch_pdl(compact_small_kernel<CTAS>, CTAS, kSmallThreads, sizeof(CompactShared), p, stream);
}

}  // namespace

cudaError_t launch_kv_release(const KvPagesParams &p, cudaStream_t stream)
{
    const bool small = p.a.num_pages <= kSmallPages;
    if (small && static_cast<int64_t>(p.num) * p.a.table_width <= kSmallEntries)
        return launch_pdl(release_small_kernel<true>, 1, kSmallThreads, 0, p, stream);
    cudaError_t e = launch_pdl(release_rows_kernel, capped(p.num, 8), kThreads, 0, p, stream);
    if (small) return e == cudaSuccess ? launch_pdl(release_small_kernel<false>, 1, kSmallThreads, 0, p, stream) : e;
    const int chunks = (p.a.num_pages + kPageChunk - 1) / kPageChunk;
    if (e == cudaSuccess) e = launch_pdl(release_count_kernel, chunks, kThreads, 0, p, stream);
    if (e == cudaSuccess) e = launch_pdl(release_list_kernel, chunks, kThreads, 0, p, stream);
    return e;
}

cudaError_t launch_kv_fork(const KvPagesParams &p, cudaStream_t stream)
{
    const size_t smem = fork_shared(p.num, p.a.num_rows);   // at most 33.5 KB
    return launch_pdl(fork_kernel, capped(p.num, 1), kThreads, smem, p, stream);
}

cudaError_t launch_kv_compact(const KvPagesParams &p, cudaStream_t stream)
{
    const int64_t entries = static_cast<int64_t>(p.a.num_rows) * p.a.table_width;
    const bool small = p.a.num_pages <= kSmallPages && p.a.num_free <= kSmallList && p.max_copies <= kSmallList;
    if (small && entries <= kSmallEntries) return launch_compact_small<1>(p, stream);
    if (small && entries <= kClusterEntries) return launch_compact_small<kClusterCtas>(p, stream);
    const int chunks = (p.a.num_pages + kPageChunk - 1) / kPageChunk;
    const int64_t lists = (static_cast<int64_t>(p.a.num_free) + kThreads - 1) / kThreads;
    const int64_t rows = p.a.num_rows > lists ? p.a.num_rows : lists;
    cudaError_t e = launch_pdl(compact_mark_kernel, capped(rows, 4), kThreads, 0, p, stream);
    if (e == cudaSuccess) e = launch_pdl(compact_count_kernel, chunks, kThreads, 0, p, stream);
    if (e == cudaSuccess) e = launch_pdl(compact_list_kernel, chunks, kThreads, 0, p, stream);
    if (e == cudaSuccess) e = launch_pdl(compact_tables_kernel, capped(rows, 4), kThreads, 0, p, stream);
    return e;
}

cudaError_t launch_page_copy(const PageCopyParams &p, cudaStream_t stream)
{
    const int units = p.heads * p.rows * p.vecs, runs = (units + kCopyUnits * kThreads - 1) / (kCopyUnits * kThreads);
    const int64_t work = static_cast<int64_t>(p.num) * runs * (p.base[1] ? 2 : 1);
    const bool dense = p.heads == 1 && p.rows == 1;
    return launch_pdl(dense ? page_copy_kernel<false> : page_copy_kernel<true>, capped(work, 8), kThreads, 0, p, stream);
}

}  // namespace lora
