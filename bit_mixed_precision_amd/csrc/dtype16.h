// The two 16-bit activation types of the decoder-layer operators and the
// forms in which 4-bit codes u = 0..15 enter their dot products and matrix
// instructions.
//
// fp16: the nibble is left where a mask finds it, as the bits of a subnormal
// fp16 (bits 0..3: u 2^-24, bits 4..7: u 2^-20; the dot product and the
// matrix instructions of gfx950 keep subnormal inputs), so a dword of eight
// codes costs one shift and four masks; the two positions' sums are kept
// apart or brought to one position by three shifts.
// bf16: a product with a bf16 subnormal would leave the fp32 range, so the
// nibble becomes the mantissa of 128: 0x4300 | u = 128 + u, exactly; the sum
// of the other operand, times the bias, is subtracted per group.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bq {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));

struct F16 {
    static constexpr bool kBf16 = false;
    static constexpr uint32_t kOnes = 0x3c003c00u;  // (1, 1)
    static __device__ __forceinline__ float to_f32(uint32_t bits16)
    {
        return (float)__builtin_bit_cast(_Float16, (uint16_t)bits16);
    }
    static __device__ __forceinline__ uint16_t from_f32(float v)
    {
        return __builtin_bit_cast(uint16_t, (_Float16)v);
    }
    static __device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c)
    {
        return __builtin_amdgcn_fdot2(__builtin_bit_cast(h2, a), __builtin_bit_cast(h2, b), c, false);
    }
    static __device__ __forceinline__ f4 mma(u4 a, u4 b, f4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
    }
};

struct BF16 {
    static constexpr bool kBf16 = true;
    static constexpr uint32_t kOnes = 0x3f803f80u;
    static __device__ __forceinline__ float to_f32(uint32_t bits16) { return __uint_as_float(bits16 << 16); }
    static __device__ __forceinline__ uint16_t from_f32(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
    static __device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c)
    {
        return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(b2, a), __builtin_bit_cast(b2, b), c, false);
    }
    static __device__ __forceinline__ f4 mma(u4 a, u4 b, f4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, a), __builtin_bit_cast(b8, b), c, 0, 0, 0);
    }
};

// Two 16-bit values in one dword: the low halves of a and b, or the high ones.
__device__ __forceinline__ uint32_t pack_lo(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x05040100u); }
__device__ __forceinline__ uint32_t pack_hi(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }

__device__ __forceinline__ float half_bits(uint32_t b) { return F16::to_f32(b); }

}  // namespace bq
