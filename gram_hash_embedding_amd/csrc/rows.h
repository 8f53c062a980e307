// Pieces shared by the training kernels: 8 consecutive row elements as fp32, from and to bf16 or fp32 memory.
#pragma once

#include "common.h"

namespace engram {

// element types of the training entry points (ENGRAM_BF16, ENGRAM_F32)
struct Bf16 {
    static constexpr int kBytes = 2;
};
struct F32 {
    static constexpr int kBytes = 4;
};

// zeros over `bytes` (a multiple of 16) at a 16-byte aligned address
int launch_zero(void* p, int64_t bytes, hipStream_t stream, const char* what);

inline bool known_dtype(int32_t d) { return d == ENGRAM_BF16 || d == ENGRAM_F32; }

// eight elements as they lie in memory: one 16-byte vector (bf16) or two (fp32)
template <class T>
struct Piece;
template <>
struct Piece<Bf16> {
    u32x4 v;
    __device__ inline void load(const void* row, int64_t piece) { v = reinterpret_cast<const u32x4*>(row)[piece]; }
    __device__ inline void load_nt(const void* row, int64_t piece) {
        v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(row) + piece);
    }
    __device__ inline void to(float (&f)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(v[i] << 16);
            f[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
        }
    }
    // round to nearest even
    __device__ inline void from(const float (&f)[8]) {
        typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bf16x2_t p = {static_cast<__bf16>(f[2 * i]), static_cast<__bf16>(f[2 * i + 1])};
            v[i] = __builtin_bit_cast(uint32_t, p);
        }
    }
    __device__ inline void store(void* row, int64_t piece) const { reinterpret_cast<u32x4*>(row)[piece] = v; }
    __device__ inline void store_nt(void* row, int64_t piece) const {
        __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(row) + piece);
    }
};
template <>
struct Piece<F32> {
    u32x4 a, b;
    __device__ inline void load(const void* row, int64_t piece) {
        a = reinterpret_cast<const u32x4*>(row)[2 * piece];
        b = reinterpret_cast<const u32x4*>(row)[2 * piece + 1];
    }
    __device__ inline void load_nt(const void* row, int64_t piece) {
        a = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(row) + 2 * piece);
        b = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(row) + 2 * piece + 1);
    }
    __device__ inline void to(float (&f)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = __uint_as_float(a[i]);
            f[4 + i] = __uint_as_float(b[i]);
        }
    }
    __device__ inline void from(const float (&f)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = __float_as_uint(f[i]);
            b[i] = __float_as_uint(f[4 + i]);
        }
    }
    __device__ inline void store(void* row, int64_t piece) const {
        reinterpret_cast<u32x4*>(row)[2 * piece] = a;
        reinterpret_cast<u32x4*>(row)[2 * piece + 1] = b;
    }
    __device__ inline void store_nt(void* row, int64_t piece) const {
        __builtin_nontemporal_store(a, reinterpret_cast<u32x4*>(row) + 2 * piece);
        __builtin_nontemporal_store(b, reinterpret_cast<u32x4*>(row) + 2 * piece + 1);
    }
};

}  // namespace engram
