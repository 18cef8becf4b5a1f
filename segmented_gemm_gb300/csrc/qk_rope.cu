// lora_qk_rope (include/lora_kv.h): norms of queries and keys for each head and
// the rotation by position, and the keys' and values' way into the paged cache.
#include <cuda_runtime.h>

#include "attn_ptx.cuh"
#include "kv_ops.h"
#include "internal.h"
#include "ptx.cuh"

namespace lora {

// A row of D elements is D / 8 items of two runs of 4 elements, one item a lane: the
// two halves of four rotated pairs (runs at 4i and rot / 2 + 4i), or eight
// neighbours (interleaved pairs, and what is not rotated).  So a pair never leaves
// its lane, and a row's sum of squares is a few lane exchanges away.
//
// A group of lanes has one head's row of each of the CTA's tokens, then the next head's
// that is its turn, so what goes by the head (addresses, weights, what is
// done) is settled once for all tokens, and four tokens' rows are in flight together.  Nothing in
// their way has a branch: lanes that do not rotate turn by an angle of 0, and values are
// chosen at the end.
//
// HBM bounds it.  8100 tokens of 32 + 8 + 8 heads of 128 into the cache, 199 MB: 38.5 us, 5.2 TB/s (64 us with
// branches and a division a row, 47 with branches alone, 44 with three CTAs an SM instead of four).  32 tokens: 2.6 us, the launch and two loads in a row.
constexpr int kRopeThreads = 256, kCtas = 4;   // of an SM

// inv_freq / 2pi, modulo 1, in units of 2^-64: what a position turns by.  inv_freq is m * 2^e, so it is
// m * (2^88 / 2pi) * 2^(e - 24), in integers: fp64 would cost more than the rest of the kernel.
__device__ __forceinline__ unsigned long long turns_of(float inv_freq)
{
    constexpr unsigned long long kHi = 0x28BE60ull, kLo = 0xDB9391054A7F09D5ull;   // 2^88 / 2pi
    const uint32_t bits = __float_as_uint(inv_freq), field = bits >> 23 & 0xFF;
    const unsigned long long m = (bits & 0x7FFFFF) | (field ? 0x800000 : 0);
    const int shift = 174 - static_cast<int>(field ? field : 1);     // 24 - e
    const unsigned long long lo = m * kLo, hi = m * kHi + __umul64hi(m, kLo);
    unsigned long long step;
    if (shift >= 128) step = 0;
    else if (shift >= 64) step = hi >> (shift - 64);
    else if (shift > 0) step = hi << (64 - shift) | lo >> shift;
    else {   // from 2^24 on: not what these frequencies are, and not exact
        const double w = static_cast<double>(fabsf(inv_freq)) * 0.15915494309189535;
        step = __double2ull_rz((w - floor(w)) * 18446744073709551616.0);
    }
    return bits >> 31 ? 0 - step : step;
}

// The cosine and sine of position * inv_freq.  The product wraps as an angle in turns should, exactly at
// any position; only its top 32 bits become an fp32 angle.
__device__ __forceinline__ float2 turn_of(unsigned long long step, int32_t pos)
{
    const unsigned long long at = step * static_cast<unsigned>(pos);
    // a signed fraction of a turn, [-1/2, 1/2), in half turns
    const float half_turns = static_cast<float>(static_cast<int32_t>(at >> 32)) * 4.656612873077393e-10f;   // 2^-31
    float2 r;
    sincospif(half_turns, &r.y, &r.x);
    return r;
}

// Two fp32 at a time.
__device__ __forceinline__ uint64_t mul_f2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t widen2(uint32_t v) { return pack_f2(bf16_lo(v), bf16_hi(v)); }
__device__ __forceinline__ uint32_t narrow2(uint64_t v)
{
    float lo, hi;
    unpack_f2(v, lo, hi);
    return pack_bf16x2(lo, hi);
}

// Up to TOKENS of a CTA (p.cta_tokens), up to four of them in flight at a time.  PARTIAL: rows have elements that are not rotated
// (an angle of 0 would do for them, but for an infinity among those beside them).
template <int LANES, int TOKENS, bool INTERLEAVED, bool PARTIAL>
__global__ void __launch_bounds__(kRopeThreads, kCtas) qk_rope_kernel(const QkRopeParams p)
{
    pdl_launch_dependents();
    constexpr int kGroups = kRopeThreads / LANES;   // rows at a time
    constexpr int U = TOKENS < 4 ? TOKENS : 4;
    constexpr int kPairs = LORA_MAX_HEAD_DIM / 2;
    // cosines and sines by quarters of pairs, as the lanes want them: (c, c, c, c), (s, s, s, s)
    __shared__ __align__(16) float turn[TOKENS][kPairs / 4][2][4];
    __shared__ int32_t position[TOKENS];
    __shared__ int64_t place[TOKENS];               // of the token in the cache, or -1
    const lora_qk_rope_t &a = p.a;
    const int tid = threadIdx.x, lane = tid % LANES, group = tid / LANES;
    const int half = a.rot_dim / 2;
    const bool rotated = lane < a.rot_dim / 8, on = lane < a.head_dim / 8;
    const bool halves = rotated && !INTERLEAVED;
    const int off0 = halves ? 4 * lane : 8 * lane, off1 = halves ? half + 4 * lane : 8 * lane + 4;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.cta_tokens;
    const int tokens = static_cast<int>(a.num_tokens - t0 < p.cta_tokens ? a.num_tokens - t0 : p.cta_tokens);
    const int heads = a.heads, k_end = heads + a.kv_heads, per = k_end + (p.kc ? a.kv_heads : 0);
    const bool norms = a.q_weight || a.k_weight;
    const float mean = 1.f / static_cast<float>(a.head_dim);
    pdl_wait();

    // row r of a token: a query head, a key head, or a value head that is only copied
    struct Row {
        const uint16_t *from;
        uint16_t *to, *cache;        // either may be NULL
        int64_t step, to_step;       // from token to token
        const uint16_t *weight;
        bool on, turned;
    };
    auto row = [&](int r) {
        Row w = {};
        w.on = r < per && on;
        w.turned = r < k_end;
        if (r < heads) {
            w.from = a.q + r * a.q_head_stride + t0 * a.q_token_stride;
            w.step = a.q_token_stride;
            w.to = a.q_out + r * a.qo_head_stride + t0 * a.qo_token_stride;
            w.to_step = a.qo_token_stride;
            w.weight = a.q_weight;
        } else {
            const int h = r - (w.turned ? heads : k_end);
            w.from = w.turned ? a.k + h * a.k_head_stride + t0 * a.k_token_stride : a.v + h * a.v_head_stride + t0 * a.v_token_stride;
            w.step = w.turned ? a.k_token_stride : a.v_token_stride;
            if (w.turned && a.k_out) w.to = a.k_out + h * a.ko_head_stride + t0 * a.ko_token_stride;
            w.to_step = a.ko_token_stride;
            if (p.kc) w.cache = (w.turned ? p.kc : p.vc) + h * p.head_stride;
            w.weight = w.turned ? a.k_weight : nullptr;
        }
        return w;
    };
    uint2 x[U][2];
    auto load = [&](const Row &w, int i0) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            x[i][0] = x[i][1] = make_uint2(0, 0);
            if (!w.on || i0 + i >= tokens) continue;
            const uint16_t *at = w.from + (i0 + i) * w.step;
            x[i][0] = *reinterpret_cast<const uint2 *>(at + off0);
            x[i][1] = *reinterpret_cast<const uint2 *>(at + off1);
        }
    };
    Row w = row(blockIdx.y * kGroups + group);
    load(w, 0);

    if (tid < tokens) {
        const int32_t at = a.position[t0 + tid], s = p.kc ? a.slot_map[t0 + tid] : -1;
        const bool known = s >= 0 && s < p.slots;
        if (at >= 0 && s != -1 && !known) atomicOr(p.status, LORA_DEV_BAD_PAGE);
        position[tid] = at;
        place[tid] = known ? (s >> p.page_shift) * p.page_stride + (s & ((1 << p.page_shift) - 1)) * p.slot_stride : -1;
    }
    static_assert(kRopeThreads % kPairs == 0, "a thread has one frequency");
    {   // what is not rotated turns by nothing, so that no lane has a branch
        const int j = tid % kPairs;
        const unsigned long long step = j < half ? turns_of(a.inv_freq[j]) : 0;
        for (int i = tid / kPairs; i < tokens; i += kRopeThreads / kPairs) {
            const float2 cs = turn_of(step, j < half ? a.position[t0 + i] : 0);
            turn[i][j / 4][0][j % 4] = cs.x;
            turn[i][j / 4][1][j % 4] = cs.y;
        }
    }
    __syncthreads();

    // the same rounds for a whole warp: rows are summed by lane exchanges
    for (int first = blockIdx.y * kGroups; first < per; first += gridDim.y * kGroups) {
        const bool again = first != static_cast<int>(blockIdx.y) * kGroups;
        if (again) w = row(first + group);
        const bool weighted = w.on && w.weight;
        uint64_t wt[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) wt[j] = pack_f2(1.f, 1.f);
        if (weighted) {
            const uint2 w0 = *reinterpret_cast<const uint2 *>(w.weight + off0), w1 = *reinterpret_cast<const uint2 *>(w.weight + off1);
            wt[0] = widen2(w0.x);
            wt[1] = widen2(w0.y);
            wt[2] = widen2(w1.x);
            wt[3] = widen2(w1.y);
        }
#pragma unroll 1
        for (int i0 = 0; i0 < tokens; i0 += U) {
            if (again || i0) load(w, i0);
            float f[U];
#pragma unroll
            for (int i = 0; i < U; ++i) f[i] = 1.f;
            if (norms) {
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    const uint64_t y0 = widen2(x[i][0].x), y1 = widen2(x[i][0].y), y2 = widen2(x[i][1].x), y3 = widen2(x[i][1].y);
                    const uint64_t s2 = fma_f2(y3, y3, fma_f2(y2, y2, fma_f2(y1, y1, mul_f2(y0, y0))));
                    float s0, s1;
                    unpack_f2(s2, s0, s1);
                    f[i] = s0 + s1;
                }
#pragma unroll
                for (int d = LANES / 2; d; d >>= 1)
#pragma unroll
                    for (int i = 0; i < U; ++i) f[i] += __shfl_xor_sync(0xffffffffu, f[i], d);
#pragma unroll
                for (int i = 0; i < U; ++i) f[i] = weighted ? rsqrtf(fmaf(f[i], mean, a.eps)) : 1.f;
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int tok = i0 + i;
                uint64_t y[4] = {widen2(x[i][0].x), widen2(x[i][0].y), widen2(x[i][1].x), widen2(x[i][1].y)};
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = mul_f2(mul_f2(y[j], wt[j]), pack_f2(f[i], f[i]));
                const float4 c = *reinterpret_cast<const float4 *>(turn[tok][lane][0]);
                const float4 s = *reinterpret_cast<const float4 *>(turn[tok][lane][1]);
                if (!INTERLEAVED) {   // pairs (y[0], y[2]) and (y[1], y[3])
                    const uint64_t c2[2] = {pack_f2(c.x, c.y), pack_f2(c.z, c.w)}, s2[2] = {pack_f2(s.x, s.y), pack_f2(s.z, s.w)};
                    const uint64_t n2[2] = {pack_f2(-s.x, -s.y), pack_f2(-s.z, -s.w)};
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint64_t u = y[j], v = y[2 + j];
                        y[j] = fma_f2(v, n2[j], mul_f2(u, c2[j]));
                        y[2 + j] = fma_f2(u, s2[j], mul_f2(v, c2[j]));
                        if (PARTIAL) {
                            y[j] = rotated ? y[j] : u;
                            y[2 + j] = rotated ? y[2 + j] : v;
                        }
                    }
                } else {              // each y[j] is a pair
                    const float cf[4] = {c.x, c.y, c.z, c.w}, sf[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float u, v;
                        unpack_f2(y[j], u, v);
                        const uint64_t z = pack_f2(fmaf(v, -sf[j], u * cf[j]), fmaf(u, sf[j], v * cf[j]));
                        y[j] = PARTIAL && !rotated ? y[j] : z;
                    }
                }
                uint2 o0 = x[i][0], o1 = x[i][1];   // values are copied as they are
                if (w.turned) {
                    o0 = make_uint2(narrow2(y[0]), narrow2(y[1]));
                    o1 = make_uint2(narrow2(y[2]), narrow2(y[3]));
                }
                const bool ok = w.on && tok < tokens && position[tok] >= 0;
                if (ok && w.to) {
                    uint16_t *to = w.to + tok * w.to_step;
                    *reinterpret_cast<uint2 *>(to + off0) = o0;
                    *reinterpret_cast<uint2 *>(to + off1) = o1;
                }
                if (ok && w.cache && place[tok] >= 0) {
                    uint16_t *to = w.cache + place[tok];
                    *reinterpret_cast<uint2 *>(to + off0) = o0;
                    *reinterpret_cast<uint2 *>(to + off1) = o1;
                }
            }
        }
    }
}

template <int LANES, bool INTERLEAVED, bool PARTIAL>
static cudaError_t launch_rope(QkRopeParams &p, cudaStream_t stream)
{
    const int64_t T = p.a.num_tokens;
    constexpr int kGroups = kRopeThreads / LANES, kTokens = 8;
    const int per = p.a.heads + (p.kc ? 2 : 1) * p.a.kv_heads;
    // few tokens: a CTA for each group of heads too, one token each (400 tokens 5.5 us so, 6.0 without; 600 7.4 and 6.6)
    const int64_t sms = num_sms_current_device();
    const bool few = T <= 3 * sms;
    // CTAs of 8 tokens from a wave and a half of them on (8100 tokens: 38.6 us, 40.1 with 4), else of 4 (600: 6.6 us, 9.0
    // with 8; 2000: 13.5 and 18.2; 6000: 31.3 and 33.1)
    p.cta_tokens = few ? 1 : T < 12 * kCtas * sms ? 4 : kTokens;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = few ? dim3(static_cast<unsigned>(T), (per + kGroups - 1) / kGroups)
                      : dim3(static_cast<unsigned>((T + p.cta_tokens - 1) / p.cta_tokens));
    cfg.blockDim = dim3(kRopeThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    pdl_attribute(cfg, at);
    return cudaLaunchKernelEx(
        &cfg, few ? qk_rope_kernel<LANES, 1, INTERLEAVED, PARTIAL> : qk_rope_kernel<LANES, kTokens, INTERLEAVED, PARTIAL>, p);
}

template <int LANES>
static cudaError_t launch_lanes(QkRopeParams &p, cudaStream_t stream)
{
    const bool partial = p.a.rot_dim < p.a.head_dim;
    if (p.a.interleaved) return partial ? launch_rope<LANES, true, true>(p, stream) : launch_rope<LANES, true, false>(p, stream);
    return partial ? launch_rope<LANES, false, true>(p, stream) : launch_rope<LANES, false, false>(p, stream);
}

// Runs of 4 elements: with 8, for rows that allow it, 8100 tokens of 128 took 55 to 62 us instead of 38.5.
cudaError_t launch_qk_rope(QkRopeParams &p, cudaStream_t stream)
{
    return p.a.head_dim <= 64 ? launch_lanes<8>(p, stream) : launch_lanes<16>(p, stream);
}

}  // namespace lora
