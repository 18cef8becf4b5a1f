// A block-wide scan and a search, for the kernels that turn lengths into
// offsets.
#pragma once
#include <cstdint>

namespace lora {

// Exclusive sum over the block's threads in thread order (blockDim a multiple
// of 32, up to 1024); *total is the whole block's.  wsum: 32 shared words.
__device__ __forceinline__ int64_t block_scan_i64(int64_t v, int64_t *wsum, int64_t *total)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) wsum[w] = x;
    __syncthreads();
    if (w == 0) {
        int64_t s = lane < nw ? wsum[lane] : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += y;
        }
        wsum[lane] = s;
    }
    __syncthreads();
    const int64_t base = w ? wsum[w - 1] : 0;
    *total = wsum[nw - 1];
    __syncthreads();
    return base + x - v;
}

// Last index i in [0, n) with a[i] <= v (a ascending, a[0] <= v).
__device__ __forceinline__ int last_le(const int32_t *a, int n, int32_t v)
{
    int lo = 0, hi = n;   // a[lo] <= v, and v < a[hi] where hi < n
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= v) lo = mid;
        else hi = mid;
    }
    return lo;
}

}  // namespace lora
