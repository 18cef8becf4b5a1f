// lora_qk_rope (include/lora_kv.h): norms of queries and keys for each head and
// the rotation by position, and the keys' and values' way into the paged cache.
#include <cuda_runtime.h>

#include "kv_ops.h"
#include "internal.h"
#include "ptx.cuh"

namespace lora {

// A row of D elements is D / 8 items of two runs of 4 elements, one item a lane: the
// two halves of four rotated pairs (runs at 4i and rot / 2 + 4i), or eight
// neighbours (interleaved pairs, and what is not rotated).  So a pair never leaves
// its lane, and a row's sum of squares is a few lane exchanges away.
//
// The angle of (position p, frequency w) in turns is p * w / 2pi modulo 1.  With
// w / 2pi modulo 1 as a 64-bit fixed-point fraction the product with p wraps as
// it should in integer arithmetic, exactly at any position; only its top 32 bits
// become an fp32 angle.  A CTA does that once for its tokens, into shared memory.
//
// HBM bounds large calls: every row is read and written once, U rows of a lane in
// flight.
constexpr int kRopeThreads = 256;

__device__ __forceinline__ float2 turn_of(float inv_freq, int32_t pos)
{
    const double t = static_cast<double>(inv_freq) * 0.15915494309189535;   // 1 / 2pi
    const unsigned long long step = __double2ull_rz((t - floor(t)) * 18446744073709551616.0);
    const unsigned long long at = step * static_cast<unsigned>(pos);
    // the top 32 bits as a signed fraction of a turn, [-1/2, 1/2)
    const float half_turns = static_cast<float>(static_cast<int32_t>(at >> 32)) * 4.656612873077393e-10f;   // 2^-31
    float2 r;
    sincospif(half_turns, &r.y, &r.x);
    return r;
}

template <int LANES, int TOKENS, int U>
__global__ void __launch_bounds__(kRopeThreads) qk_rope_kernel(const QkRopeParams p)
{
    pdl_launch_dependents();
    __shared__ __align__(16) float2 turn[TOKENS][LORA_MAX_HEAD_DIM / 2];
    __shared__ int32_t position[TOKENS], slot[TOKENS];
    constexpr int kGroups = kRopeThreads / LANES;   // rows at a time
    const lora_qk_rope_t &a = p.a;
    const int tid = threadIdx.x, lane = tid % LANES, group = tid / LANES;
    const int half = a.rot_dim / 2;
    const bool rotated = lane < a.rot_dim / 8, on = lane < a.head_dim / 8;
    const bool halves = rotated && !a.interleaved;
    const int off0 = halves ? 4 * lane : 8 * lane, off1 = halves ? half + 4 * lane : 8 * lane + 4;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * TOKENS;
    const int tokens = static_cast<int>(a.num_tokens - t0 < TOKENS ? a.num_tokens - t0 : TOKENS);
    const int heads = a.heads, k_end = heads + a.kv_heads, per = k_end + (p.kc ? a.kv_heads : 0);
    const int rows = tokens * per;
    const bool norm = a.q_weight || a.k_weight;
    pdl_wait();

    // weights of this lane's elements
    uint2 w[2][2] = {};
    if (on && a.q_weight) {
        w[0][0] = *reinterpret_cast<const uint2 *>(a.q_weight + off0);
        w[0][1] = *reinterpret_cast<const uint2 *>(a.q_weight + off1);
    }
    if (on && a.k_weight) {
        w[1][0] = *reinterpret_cast<const uint2 *>(a.k_weight + off0);
        w[1][1] = *reinterpret_cast<const uint2 *>(a.k_weight + off1);
    }

    uint2 x[U][2];
    auto load = [&](int base) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = base + u * kGroups + group;
            x[u][0] = x[u][1] = make_uint2(0, 0);
            if (i >= rows || !on) continue;
            const int tok = TOKENS == 1 ? 0 : i / per, r = i - tok * per;
            const int64_t t = t0 + tok;
            const uint16_t *row = r < heads ? a.q + t * a.q_token_stride + r * a.q_head_stride
                                  : r < k_end ? a.k + t * a.k_token_stride + (r - heads) * a.k_head_stride
                                              : a.v + t * a.v_token_stride + (r - k_end) * a.v_head_stride;
            x[u][0] = *reinterpret_cast<const uint2 *>(row + off0);
            x[u][1] = *reinterpret_cast<const uint2 *>(row + off1);
        }
    };
    load(0);

    if (tid < tokens) {
        position[tid] = a.position ? a.position[t0 + tid] : 0;
        slot[tid] = p.kc ? a.slot_map[t0 + tid] : -1;
    }
    for (int i = tid; i < tokens * half; i += kRopeThreads) {
        const int tok = TOKENS == 1 ? 0 : i / half, j = i - tok * half;
        turn[tok][j] = turn_of(a.inv_freq[j], a.position[t0 + tok]);
    }
    __syncthreads();
    if (tid < tokens && slot[tid] != -1 && position[tid] >= 0 && (slot[tid] < 0 || slot[tid] >= p.slots))
        atomicOr(p.status, LORA_DEV_BAD_PAGE);

    for (int base = 0; base < rows; base += U * kGroups) {
        if (base) load(base);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = base + u * kGroups + group;
            const bool row_on = i < rows;
            const int tok = TOKENS == 1 || !row_on ? 0 : i / per, r = i - tok * per;
            const bool is_q = r < heads, is_v = r >= k_end;
            float y[8] = {bf16_lo(x[u][0].x), bf16_hi(x[u][0].x), bf16_lo(x[u][0].y), bf16_hi(x[u][0].y),
                          bf16_lo(x[u][1].x), bf16_hi(x[u][1].x), bf16_lo(x[u][1].y), bf16_hi(x[u][1].y)};
            if (norm) {
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) sum += y[j] * y[j];
#pragma unroll
                for (int d = LANES / 2; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                if (is_q ? a.q_weight != nullptr : a.k_weight != nullptr) {
                    const float f = rsqrtf(sum / static_cast<float>(a.head_dim) + a.eps);
                    const uint2 w0 = is_q ? w[0][0] : w[1][0], w1 = is_q ? w[0][1] : w[1][1];
                    const float wf[8] = {bf16_lo(w0.x), bf16_hi(w0.x), bf16_lo(w0.y), bf16_hi(w0.y),
                                         bf16_lo(w1.x), bf16_hi(w1.x), bf16_lo(w1.y), bf16_hi(w1.y)};
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[j] *= f * wf[j];
                }
            }
            if (!row_on || !on || position[tok] < 0) continue;
            if (rotated) {
                const float4 c01 = *reinterpret_cast<const float4 *>(&turn[tok][4 * lane]);
                const float4 c23 = *reinterpret_cast<const float4 *>(&turn[tok][4 * lane + 2]);
                const float c[4] = {c01.x, c01.z, c23.x, c23.z}, s[4] = {c01.y, c01.w, c23.y, c23.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float a0 = a.interleaved ? y[2 * j] : y[j], b0 = a.interleaved ? y[2 * j + 1] : y[4 + j];
                    const float a1 = a0 * c[j] - b0 * s[j], b1 = b0 * c[j] + a0 * s[j];
                    if (a.interleaved) {
                        y[2 * j] = a1;
                        y[2 * j + 1] = b1;
                    } else {
                        y[j] = a1;
                        y[4 + j] = b1;
                    }
                }
            }
            uint2 o0 = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
            uint2 o1 = make_uint2(pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
            const int64_t t = t0 + tok;
            uint16_t *out = nullptr;
            if (is_q) {
                out = a.q_out + t * a.qo_token_stride + r * a.qo_head_stride;
            } else if (!is_v && a.k_out) {
                out = a.k_out + t * a.ko_token_stride + (r - heads) * a.ko_head_stride;
            }
            if (is_v) {   // copied as it is
                o0 = x[u][0];
                o1 = x[u][1];
            }
            if (out) {
                *reinterpret_cast<uint2 *>(out + off0) = o0;
                *reinterpret_cast<uint2 *>(out + off1) = o1;
            }
            if (!is_q && p.kc && slot[tok] >= 0 && slot[tok] < p.slots) {
                const int64_t page = slot[tok] >> p.page_shift, line = slot[tok] & ((1 << p.page_shift) - 1);
                const int64_t h = r - (is_v ? k_end : heads);
                uint16_t *to = (is_v ? p.vc : p.kc) + page * p.page_stride + h * p.head_stride + line * p.slot_stride;
                *reinterpret_cast<uint2 *>(to + off0) = o0;
                *reinterpret_cast<uint2 *>(to + off1) = o1;
            }
        }
    }
}

cudaError_t launch_qk_rope(const QkRopeParams &p, cudaStream_t stream)
{
    const int64_t T = p.a.num_tokens;
    const bool wide = p.a.head_dim > 64;
    if (T <= 4ll * num_sms_current_device())   // few tokens: spread over the SMs
        return launch_pdl(wide ? qk_rope_kernel<16, 1, 4> : qk_rope_kernel<8, 1, 4>, T, kRopeThreads, 0, p, stream);
    return launch_pdl(wide ? qk_rope_kernel<16, 4, 4> : qk_rope_kernel<8, 4, 4>, (T + 3) / 4, kRopeThreads, 0, p, stream);
}

}  // namespace lora
