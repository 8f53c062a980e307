// OCP MX fp8 block encoding (E4M3 elements, one E8M0 scale per 32 elements), shared by the quantiser of bf16
// rows (engram_mx_quant) and the gather that writes MX fp8 rows directly (engram_gather_mx): both encode the
// same bf16 values, so their bytes agree.  And MXINT8 (elements of 64ths), the checkpoints' format.
#pragma once

#include "common.h"

namespace engram {

// The block's shared exponent from its amax (a bf16 value held in fp32, normal or subnormal, so fp32 holds it
// exactly): floor(log2 amax) - 8 (8 is E4M3's largest exponent), clamped to E8M0's [-127, 127], read off the
// exponent field (or, for a subnormal, the leading one of the fraction); -127 for an all-zero block.  Its E8M0
// code is shared + 127.
__device__ inline int mx_shared_exp(float amax) {
    if (!(amax > 0.f)) return -127;
    const uint32_t au = __float_as_uint(amax);
    const int ef = static_cast<int>(au >> 23);
    const int fl = ef != 0 ? ef - 127 : 31 - __builtin_clz(au & 0x7FFFFFu) - 149;  // floor(log2 amax)
    return max(-127, min(127, fl - 8));
}

// Four elements times 2^-shared (exact: a power of two; results below fp32's normal range round to 0 in E4M3
// either way), clamped to +-448 so that the conversion cannot overflow, rounded to E4M3 (nearest even,
// subnormals included) by v_cvt_pk_fp8_f32 -- OCP E4M3 on gfx950: the saturating conversion.  Bytes in
// element order.
__device__ inline uint32_t mx_encode4(float f0, float f1, float f2, float f3, int shared) {
    auto g = [shared](float f) { return __builtin_amdgcn_fmed3f(__builtin_ldexpf(f, -shared), -448.0f, 448.0f); };
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(g(f0), g(f1), 0, false);
    return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(g(f2), g(f3), lo, true));
}

// Byte offset of the E8M0 scale of (row r, 32-column block b) in the scale layout [K/128][rows4][4].
__device__ inline int64_t mx_scale_offset(int64_t r, int b, int64_t rows4) {
    return (static_cast<int64_t>(b >> 2) * rows4 + r) * 4 + (b & 3);
}

// ---- MXINT8: an element is an integer in [-127, 127] times 2^(code - 127) / 64.  With code the exponent field of the block's
// largest magnitude, integers reach 64 .. 127 (rounded values past 127 saturate); a value is exact in bf16 again.
typedef uint32_t mx_u32x2 __attribute__((ext_vector_type(2)));

// the largest magnitude of eight bf16 values, as its bit pattern (the patterns' order is the magnitudes')
__device__ inline uint32_t bf16_top8(const u32x4& v) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, max(v[i] & 0x7FFFu, (v[i] >> 16) & 0x7FFFu));
    return top;
}
// the same over the four lanes 4 b .. 4 b + 3 of a block of 32 (every lane of the wave takes part)
__device__ inline uint32_t block_top(uint32_t top) {
    top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 1, 64)));
    return max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 2, 64)));
}
// Eight bf16 values as MXINT8 with the scale code `code`, bytes in element order: times 2^(133 - code) (exact, by exponent:
// the factor itself may pass fp32's range), clamped, and rounded to nearest even by adding 1.5 * 2^23, which leaves the
// integer in the sum's low bits.  A block with an infinity or a NaN (code 255, the NaN scale) holds zeros.
__device__ inline mx_u32x2 mxint8_encode8(const u32x4& v, uint32_t code) {
    mx_u32x2 o;
    const int shift = 133 - static_cast<int>(code);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t b[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t w = v[2 * h + e / 2];
            const float f = __uint_as_float(e % 2 ? w & 0xFFFF0000u : w << 16);
            b[e] = __float_as_uint(__builtin_amdgcn_fmed3f(__builtin_ldexpf(f, shift), -127.0f, 127.0f) + 12582912.0f);
        }
        const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u), hi = __builtin_amdgcn_perm(b[3], b[2], 0x0C0C0400u);
        o[h] = code == 255 ? 0u : lo | (hi << 16);
    }
    return o;
}
// what a unit of a block with this code stands for (NaN for the NaN scale)
__device__ inline float mxint8_unit(uint32_t code) {
    return code == 255 ? __uint_as_float(0x7FC00000u) : __builtin_ldexpf(1.0f, static_cast<int>(code) - 133);
}
// element e of eight, in units (cut out of its word: as shifted bytes the eight of a row are made 64-bit shifts that hold a
// register pair each, and the gradient that reads eight rows spilled 86 registers)
__device__ inline float mxint8_at(const mx_u32x2& q, int e) {
    return static_cast<float>(static_cast<int>(__builtin_amdgcn_sbfe(q[e / 4], 8 * (e % 4), 8)));
}
// eight elements as floats (exact)
__device__ inline void mxint8_decode8(const mx_u32x2& q, float unit, float (&f)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = mxint8_at(q, e) * unit;
}

}  // namespace engram
