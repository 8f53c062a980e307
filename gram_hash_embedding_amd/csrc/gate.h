// Pieces of the gate shared by its kernels (gate_dot.hip, gate_grad.hip, checkpoint.hip, wkv_mx4.hip): pairs of bf16, sums over a
// wave, the gate of a dot, and the residual.
#pragma once

#include "common.h"

namespace engram {

__device__ inline float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ inline float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ inline float wave_sum(float v) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}

__device__ inline uint32_t pack2_bf16(float lo, float hi) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 v = {static_cast<__bf16>(lo), static_cast<__bf16>(hi)};  // round to nearest even
    return __builtin_bit_cast(uint32_t, v);
}

// h + gate * v as two fp32 roundings (the product, then the sum), then bf16: the pages form the
// gated value first and add it to the stream, so no fused multiply-add here
__device__ inline u32x4 residual(const u32x4 h, const u32x4 v, float gate) {
#pragma clang fp contract(off)
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float g0 = gate * lo_bf16(v[i]);
        const float g1 = gate * hi_bf16(v[i]);
        o[i] = pack2_bf16(lo_bf16(h[i]) + g0, hi_bf16(h[i]) + g1);
    }
    return o;
}

// sigmoid of the signed square root; |dot| is clamped from below at 1e-6 first
__device__ inline float gate_of(float d) {
    const float z = copysignf(sqrtf(fmaxf(fabsf(d), 1e-6f)), d);
    return 1.0f / (1.0f + expf(-z));
}

}  // namespace engram
