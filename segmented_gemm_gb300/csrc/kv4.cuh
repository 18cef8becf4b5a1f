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

// 8 codes and their scale -> 8 fp16 values (exact).
__device__ __forceinline__ uint4 kv4_values_f16(uint32_t codes, uint32_t scale)
{
    uint32_t f[4];
    e2m1x8_to_f16(codes, f);
    const uint32_t s = scale_pair<0, 0>(scale);
    return make_uint4(mul_f16x2(f[0], s), mul_f16x2(f[1], s), mul_f16x2(f[2], s), mul_f16x2(f[3], s));
}

// 8 codes and their scale -> 8 bf16 values (exact: 6 significant bits).
__device__ __forceinline__ uint4 kv4_values(uint32_t codes, uint32_t scale)
{
    const uint4 v = kv4_values_f16(codes, scale);
    const uint32_t two[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&two[i]));
        o[i] = pack_bf16x2(x.x, x.y);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// 32 bytes at once, a whole sector, where rows start on 32 bytes and are whole groups.
__device__ __forceinline__ void load32(const uint16_t *from, uint4 (&x)[2])
{
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(x[0].x), "=r"(x[0].y), "=r"(x[0].z), "=r"(x[0].w), "=r"(x[1].x), "=r"(x[1].y), "=r"(x[1].z), "=r"(x[1].w)
                 : "l"(from));
}
__device__ __forceinline__ void store32(uint16_t *to, const uint4 &a, const uint4 &b)
{
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w),
                 "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
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
