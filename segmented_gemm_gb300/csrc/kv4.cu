// Writes into and reads of the 4-bit cache (include/lora_kv.h): lora_kv4_store
// and lora_kv4_load.
#include <cuda_runtime.h>

#include "attn_ptx.cuh"
#include "kv4.cuh"
#include "kv_ops.h"
#include "internal.h"
#include "ptx.cuh"

namespace lora {

constexpr int kKv4Threads = 256;

// The scale byte of 16 elements whose largest magnitude is amax (finite): amax / 6
// rounded to 3 fraction bits.  Ties can be told in fp32: amax has 8 significant bits, so
// a quotient that is not halfway between two scales is at least 2^-13 (relative) off.
__device__ __forceinline__ uint32_t scale_byte(float amax)
{
    const float a = __fdiv_rn(amax, 6.f);
    if (a < 6.103515625e-05f) return __float2uint_rn(a * 131072.f);   // below 2^-14: multiples of 2^-17
    const uint32_t bits = __float_as_uint(a);
    const uint32_t r = (bits + 0x7FFFFu + ((bits >> 20) & 1)) >> 20;  // exponent (bias 127) and 3 bits
    return min(r - (112u << 3), 226u);                                // 226: 10240
}

__device__ __forceinline__ float scale_value(uint32_t byte)
{
    return __half2float(__ushort_as_half(static_cast<unsigned short>(byte << 7)));
}

// Eight codes of four pairs of fp32, the first in the lowest bits; nearest, ties to even, saturating.
__device__ __forceinline__ uint32_t e2m1x8(const uint64_t (&y)[4])
{
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t.reg .f32 lo, hi;\n\t"
        "mov.b64 {lo, hi}, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b0, hi, lo;\n\t"
        "mov.b64 {lo, hi}, %2;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, hi, lo;\n\t"
        "mov.b64 {lo, hi}, %3;\n\tcvt.rn.satfinite.e2m1x2.f32 b2, hi, lo;\n\t"
        "mov.b64 {lo, hi}, %4;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, hi, lo;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "l"(y[0]), "l"(y[1]), "l"(y[2]), "l"(y[3]));
    return r;
}

// For two elements x (bf16): x * inv to a multiple of 2^-12 (for |x * inv| < 1024; a larger one keeps what precision
// there is), with the sign of x where that is 0 (of 0 itself a positive one).
__device__ __forceinline__ uint64_t rounded_products(uint32_t x, uint64_t inv)
{
    constexpr float kRound = 1.5f * 2048.f;   // fp32 numbers around it, from 2^11 to 2^12, are 2^-12 apart
    const uint64_t x2 = pack_f2(bf16_lo(x), bf16_hi(x)), y2 = add_f2(fma_f2(x2, inv, pack_f2(kRound, kRound)), pack_f2(-kRound, -kRound));
    float x0, x1, y0, y1;
    unpack_f2(add_f2(x2, 0), x0, x1);  // -0 becomes 0
    unpack_f2(y2, y0, y1);
    return pack_f2(copysignf(y0, x0), copysignf(y1, x1));
}

// 16 bf16 elements -> 16 codes (8 bytes) and the scale byte.
__device__ __forceinline__ uint2 quantise(const uint4 &x0, const uint4 &x1, uint32_t *scale)
{
    const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
    uint32_t top2 = 0;   // the largest magnitudes' bits, which order as the magnitudes do, NaN above all
#pragma unroll
    for (int i = 0; i < 8; ++i) asm("max.u16x2 %0, %0, %1;" : "+r"(top2) : "r"(w[i] & 0x7FFF7FFFu));
    const uint32_t top = max(top2 & 0xFFFFu, top2 >> 16) << 16;
    if (top > 0x7F800000u) {
        *scale = 0xFF;
        return make_uint2(0, 0);
    }
    // an infinity counts as the largest bf16: the scale saturates, and x / s does
    const uint32_t b = scale_byte(__uint_as_float(min(top, 0x7F7F0000u)));
    *scale = b;
    if (b == 0) return make_uint2(0, 0);
    // x / s as x * (1 / s), rounded to a multiple of 2^-12 on the way.  A quotient halfway
    // between two values is x = half * s: the product is within 2^-22 of it and rounds to it.  Any
    // other one is at least 2^-8 (relative) from there, x having 8 and half * s 7
    // significant bits, and stays on its side.
    const float inv = __frcp_rn(scale_value(b));
    const uint64_t inv2 = pack_f2(inv, inv);
    uint32_t c[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint64_t y[4] = {rounded_products(w[4 * i], inv2), rounded_products(w[4 * i + 1], inv2),
                               rounded_products(w[4 * i + 2], inv2), rounded_products(w[4 * i + 3], inv2)};
        c[i] = e2m1x8(y);
    }
    return make_uint2(c[0], c[1]);
}

// A thread takes 16 elements of a head's key row and of its value row, consecutive
// threads consecutive elements.  Memory bounds it, and the arithmetic of 32 elements a thread: 7300 tokens
// of 8 heads of 128, 38 MB, 10.3 us (13.9 with divisions, 11.4 without packed arithmetic); 32 tokens 2.6 us.
template <int DP>
__global__ void __launch_bounds__(kKv4Threads) kv4_store_kernel(const Kv4StoreParams p)
{
    pdl_launch_dependents();
    using Tile = Kv4Tile<DP>;
    const uint32_t per = static_cast<uint32_t>(p.kv_heads) * Tile::kGroups;
    const int64_t total = p.T * per;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kKv4Threads;
    pdl_wait();
    int bad = 0;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kKv4Threads + threadIdx.x; i < total; i += stride) {
        const int64_t t = total < (int64_t(1) << 32) ? static_cast<uint32_t>(i) / per : i / per;
        const int u = static_cast<int>(i - t * per), h = u / Tile::kGroups, g = u % Tile::kGroups;
        const int32_t slot = p.slot_map[t];
        uint4 k[2] = {}, v[2] = {};
        const uint16_t *kr = p.k + t * p.k_tok + h * p.k_head + 16 * g, *vr = p.v + t * p.v_tok + h * p.v_head + 16 * g;
        if (p.sectors) {
            if (16 * g < p.head_dim) {
                load32(kr, k);
                load32(vr, v);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (16 * g + 8 * e >= p.head_dim) continue;   // padding
                k[e] = *reinterpret_cast<const uint4 *>(kr + 8 * e);
                v[e] = *reinterpret_cast<const uint4 *>(vr + 8 * e);
            }
        }
        if (slot < 0 || slot >= p.slots) {
            bad |= slot != -1;
            continue;
        }
        const int64_t page = slot >> p.page_shift;
        const int line = slot & ((1 << p.page_shift) - 1), j = line & 15;
        uint8_t *tile = p.data + page * p.page_stride + h * p.head_stride + (line >> 4) * Tile::kBytes;
        uint32_t scale;
        uint2 c = quantise(k[0], k[1], &scale);
        *reinterpret_cast<uint2 *>(tile + j * (DP / 2) + g * 8) = c;
        tile[Tile::kKeyScales + j * Tile::kGroups + g] = static_cast<uint8_t>(scale);
        c = quantise(v[0], v[1], &scale);
        *reinterpret_cast<uint32_t *>(tile + Tile::value_word(j, 16 * g)) = c.x;
        *reinterpret_cast<uint32_t *>(tile + Tile::value_word(j, 16 * g + 8)) = c.y;
        tile[Tile::value_scale(j, g)] = static_cast<uint8_t>(scale);
    }
    if (bad) atomicOr(p.status, LORA_DEV_BAD_PAGE);
}

// The reverse, the same split; memory bounds it, three quarters of it the writes: 8192 slots of 8 heads of
// 128, 43 MB, 9.0 us (12.0 with 16-byte stores, half sectors each).
template <int DP>
__global__ void __launch_bounds__(kKv4Threads) kv4_load_kernel(const Kv4LoadParams p)
{
    pdl_launch_dependents();
    using Tile = Kv4Tile<DP>;
    const uint32_t groups = (p.head_dim + 15) / 16, per = static_cast<uint32_t>(p.kv_heads) * groups;
    const int64_t total = p.n * per;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kKv4Threads;
    pdl_wait();
    int bad = 0;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kKv4Threads + threadIdx.x; i < total; i += stride) {
        const int64_t t = total < (int64_t(1) << 32) ? static_cast<uint32_t>(i) / per : i / per;
        const int u = static_cast<int>(i - t * per), h = u / groups, g = u - h * groups;
        const int32_t slot = p.slot_list[t];
        const bool on = slot >= 0 && slot < p.slots;
        bad |= !on && slot != -1;
        uint2 kw = {}, vw = {};
        uint32_t ks = 0, vs = 0;
        if (on) {
            const int64_t page = slot >> p.page_shift;
            const int line = slot & ((1 << p.page_shift) - 1), j = line & 15;
            const uint8_t *tile = p.data + page * p.page_stride + h * p.head_stride + (line >> 4) * Tile::kBytes;
            kw = *reinterpret_cast<const uint2 *>(tile + j * (DP / 2) + g * 8);
            ks = tile[Tile::kKeyScales + j * Tile::kGroups + g];
            vw.x = *reinterpret_cast<const uint32_t *>(tile + Tile::value_word(j, 16 * g));
            vw.y = *reinterpret_cast<const uint32_t *>(tile + Tile::value_word(j, 16 * g + 8));
            vs = tile[Tile::value_scale(j, g)];
        }
        const bool second = 16 * g + 8 < p.head_dim;
        uint16_t *const rows[2] = {p.k ? p.k + t * p.k_tok + h * p.k_head + 16 * g : nullptr,
                                   p.v ? p.v + t * p.v_tok + h * p.v_head + 16 * g : nullptr};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (!rows[e]) continue;
            const uint4 lo = kv4_values(e ? vw.x : kw.x, e ? vs : ks), hi = kv4_values(e ? vw.y : kw.y, e ? vs : ks);
            if (p.sectors) {
                store32(rows[e], lo, hi);
            } else {
                *reinterpret_cast<uint4 *>(rows[e]) = lo;
                if (second) *reinterpret_cast<uint4 *>(rows[e] + 8) = hi;
            }
        }
    }
    if (bad) atomicOr(p.status, LORA_DEV_BAD_PAGE);
}

static int64_t kv4_ctas(int64_t total)
{
    const int64_t ctas = (total + kKv4Threads - 1) / kKv4Threads, cap = 16ll * num_sms_current_device();
    return ctas < cap ? ctas : cap;
}

cudaError_t launch_kv4_store(const Kv4StoreParams &p, cudaStream_t stream)
{
    const int dp = kv4_padded(p.head_dim);
    return launch_pdl(dp == 64 ? kv4_store_kernel<64> : kv4_store_kernel<128>,
                      kv4_ctas(p.T * p.kv_heads * (dp / 16)), kKv4Threads, 0, p, stream);
}

cudaError_t launch_kv4_load(const Kv4LoadParams &p, cudaStream_t stream)
{
    return launch_pdl(p.head_dim <= 64 ? kv4_load_kernel<64> : kv4_load_kernel<128>,
                      kv4_ctas(p.n * p.kv_heads * ((p.head_dim + 15) / 16)), kKv4Threads, 0, p, stream);
}

}  // namespace lora
