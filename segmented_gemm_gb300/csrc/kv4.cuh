// The 4-bit cache's number formats and tile layout (include/lora_kv.h).
#pragma once
#include <cuda_fp16.h>

#include <cstdint>

#include "ptx.cuh"

namespace lora {

// Eight 4-bit codes -> four pairs of fp16 values; codes 2i and 2i + 1 (byte i) give o[i].
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t codes, uint32_t (&o)[4])
{
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
        : "r"(codes));
}

// The product of a code's value (2 significant bits) and a scale (4) is exact in fp16.
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Scale bytes i and j of v as a pair of fp16: a scale is an fp16's bits 14 to 7.
template <int I, int J>
__device__ __forceinline__ uint32_t scale_pair(uint32_t v)
{
    return __byte_perm(v, 0u, I | 0x40 | (J << 8) | 0x4000) << 7;
}

// 8 codes and their scale -> 8 bf16 values (exact: 6 significant bits).
__device__ __forceinline__ uint4 kv4_values(uint32_t codes, uint32_t scale)
{
    uint32_t f[4];
    e2m1x8_to_f16(codes, f);
    const uint32_t s = scale_pair<0, 0>(scale);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t two = mul_f16x2(f[i], s);
        const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&two));
        o[i] = pack_bf16x2(x.x, x.y);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// Offsets in a tile.
template <int DP>
struct Kv4Tile {
    static constexpr int kBytes = 18 * DP, kKeyScales = 8 * DP, kValues = 9 * DP, kValueScales = 17 * DP;
    static constexpr int kGroups = DP / 16;

    // 8 codes of the values of key j, elements d .. d + 7 (d a multiple of 8)
    static __device__ __forceinline__ int value_word(int j, int d)
    {
        return kValues + ((((j >> 3) * 8 + d / (DP / 8)) * 4 + (j & 7) / 2) * (DP / 64) + d % (DP / 8) / 8) * 8 + (j & 1) * 4;
    }
    static __device__ __forceinline__ int value_scale(int j, int group)
    {
        return kValueScales + (group * 4 + (j & 7) / 2) * 4 + (j >> 3) * 2 + (j & 1);
    }
};

}  // namespace lora
