// Attention over packed rows or a paged cache (include/lora_attn.h).
//
// A first kernel that is right for every case: a warp per (row, head), 32 keys
// at a time, a lane per key for the scores and a lane per column for p v, with
// the running maximum and sum of a softmax.
#include <cuda_runtime.h>

#include "attn.h"
#include "internal.h"
#include "ptx.cuh"

namespace lora {

constexpr int kAttnThreads = 128;

__global__ void __launch_bounds__(kAttnThreads) attn_kernel(const AttnParams p)
{
    pdl_launch_dependents();
    pdl_wait();
    __shared__ float qs[kAttnThreads / 32][LORA_MAX_HEAD_DIM];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nb = p.hdr->nblocks, D = p.head_dim;
    for (int64_t u = blockIdx.x; u < static_cast<int64_t>(nb) * p.kv_heads; u += gridDim.x) {
        const AttnBlock b = p.blocks[p.order[u / p.kv_heads]];
        const int kvh = static_cast<int>(u % p.kv_heads);
        const int base = p.cu[b.req];
        for (int row = warp; row < b.ntok * p.group; row += kAttnThreads / 32) {
            const int i = row / p.group, h = kvh * p.group + row % p.group;
            const int64_t t = b.tok0 + i;
            const int limit = max(0, min(b.kv_len, b.qpos0 + i + 1));
            __syncwarp();
            for (int d = lane; d < D; d += 32)
                qs[warp][d] = __uint_as_float(static_cast<uint32_t>(p.q[t * p.q_tok + h * p.q_head + d]) << 16);
            __syncwarp();
            float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
            for (int j0 = 0; j0 < limit; j0 += 32) {
                const int j = j0 + lane;
                int64_t ko = -1, vo = -1;
                bool zero = false;
                if (j < limit) {
                    if (p.block_table) {
                        const int pg = j >> p.page_shift;
                        const int page = pg < p.table_width ? p.block_table[b.req * p.table_stride + pg] : -1;
                        if (page < 0 || page >= p.num_pages) {
                            zero = true;
                            atomicOr(p.counters + CNT_STATUS, LORA_DEV_BAD_PAGE);
                        } else {
                            ko = vo = page * p.page_stride + kvh * p.head_stride +
                                      (j & ((1 << p.page_shift) - 1)) * p.slot_stride;
                        }
                    } else {
                        ko = (static_cast<int64_t>(base) + j) * p.k_tok + kvh * p.k_head;
                        vo = (static_cast<int64_t>(base) + j) * p.v_tok + kvh * p.v_head;
                    }
                }
                float s = -INFINITY;
                if (ko >= 0) {
                    s = 0.f;
                    for (int d = 0; d < D; d += 8) {
                        const uint4 k8 = *reinterpret_cast<const uint4 *>(p.k + ko + d);
                        const uint32_t w[4] = {k8.x, k8.y, k8.z, k8.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            s += qs[warp][d + 2 * e] * bf16_lo(w[e]) + qs[warp][d + 2 * e + 1] * bf16_hi(w[e]);
                    }
                    s *= p.scale;
                } else if (zero) {
                    s = 0.f;
                }
                float mx = s;
                for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                const float mn = fmaxf(m, mx), f = m == -INFINITY ? 0.f : expf(m - mn);
                const float pr = s == -INFINITY ? 0.f : expf(s - mn);
                m = mn;
                l = l * f + pr;
                const float pb = __uint_as_float(pack_bf16x2(pr, 0.f) << 16);
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[c] *= f;
                for (int e = 0; e < 32 && j0 + e < limit; ++e) {
                    const float pe = __shfl_sync(0xffffffffu, pb, e);
                    const int64_t ve = __shfl_sync(0xffffffffu, vo, e);
                    if (ve < 0) continue;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (c * 32 + lane < D)
                            acc[c] += pe * __uint_as_float(static_cast<uint32_t>(p.v[ve + c * 32 + lane]) << 16);
                }
            }
            for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
            const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (c * 32 + lane < D)
                    p.o[t * p.o_tok + h * p.o_head + c * 32 + lane] =
                        static_cast<uint16_t>(pack_bf16x2(limit ? acc[c] * inv : 0.f, 0.f) & 0xFFFFu);
            if (p.lse && lane == 0) p.lse[t * p.heads + h] = limit ? m + logf(l) : -INFINITY;
        }
    }
}

cudaError_t launch_attn(const AttnParams &p, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(8 * num_sms_current_device());
    cfg.blockDim = dim3(kAttnThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    pdl_attribute(cfg, at);
    return cudaLaunchKernelEx(&cfg, attn_kernel, p);
}

}  // namespace lora
