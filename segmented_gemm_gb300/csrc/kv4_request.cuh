// A request of a step over the 4-bit cache, as the kernels of lora_kv4_attn see it.
#pragma once
#include "kv_ops.h"

namespace lora {

// Packed tokens of request r and its keys, clamped.
struct Kv4Request {
    int tok0, n, keys;
};

__device__ __forceinline__ Kv4Request kv4_request(const Kv4AttnParams &p, int r, int *bad)
{
    const int a0 = p.cu[r], b0 = p.cu[r + 1], k0 = p.kv_len[r];
    const int a = max(0, min(a0, p.T)), b = max(0, min(b0, p.T));
    Kv4Request q;
    q.tok0 = a;
    q.n = max(0, b - a);
    q.keys = static_cast<int>(k0 < 0 ? 0 : k0 > p.max_kv ? p.max_kv : k0);
    *bad |= (a != a0) | (b != b0) | (b < a) | (q.keys != k0);
    return q;
}

}  // namespace lora
