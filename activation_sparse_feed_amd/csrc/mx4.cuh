// The 4-bit form of cached keys and values: OCP MX FP4 in blocks of 32 elements of a
// head, E2M1 elements (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives) and one E8M0 scale
// byte b for 2^(b - 127) or NaN.  A byte holds the element 2 i in its low and
// 2 i + 1 in its high four bits.
//
// Taken because gfx950 converts it both ways two elements at a time with the scale
// applied, and because every value it stands for is a bfloat16 number: attention over the
// 4-bit cache is attention over that bfloat16 cache, with nothing rounded on the way.
// The instructions agree with the format for all 256 scales and all codes (subnormal
// results and overflow to infinity included), and round ties to the even code on encoding
// with larger values saturated, for scales 2^-124 .. 2^125 and any finite float32.
#pragma once

#include <hip/hip_runtime.h>

#include "common.cuh"

namespace sffn {

constexpr int kMxBlock = 32;
constexpr int mx_blocks(int head_dim) { return (head_dim + kMxBlock - 1) / kMxBlock; }

// The scale of a byte.  253 and 254, whose largest elements no type here holds, are never
// written and read as NaN like 255, so that a block is finite or NaN as a whole.
constexpr uint32_t kMxBad = 253;
__device__ __forceinline__ float mx_scale(uint32_t byte) {
  return __uint_as_float((byte >= kMxBad ? 255u : byte) << 23);
}

// The scale byte of a block whose largest magnitude has the float32 bits `top`: the
// smallest exponent e in -124 .. 125 with top < 7 * 2^e, so that no element is off by more
// than half a step of the largest binade (above 7 * 2^125, which has no such e, up to a
// quarter), 255 where an element is not finite.  From -124 on values below 2^-126 are
// under half the smallest element, and the instruction's treatment of subnormals
// does not matter; up to 125 the largest element is finite in float32 and bfloat16.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t top) {
  const int e = (int)(top >> 23) - 2 + ((top & 0x7fffffu) >= 0x600000u ? 1 : 0);
  return top >= 0x7f800000u ? 255u : (uint32_t)min(max(e, 3), 252);
}

// Eight elements in one word.
__device__ __forceinline__ uint32_t mx_encode8(const float (&x)[8], float scale) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], scale, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], scale, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], scale, 3);
}

// The elements of a word as T: 16 bytes of bfloat16 or 32 of float32.
template <typename T> struct Mx;
template <> struct Mx<uint16_t> {
  static constexpr int kChunks = 1;
  __device__ static __forceinline__ void decode8(uint32_t w, float scale, u32x4_t (&o)[1]) {
    o[0][0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
    o[0][1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
    o[0][2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
    o[0][3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
  }
};
template <> struct Mx<float> {
  static constexpr int kChunks = 2;
  __device__ static __forceinline__ void decode8(uint32_t w, float scale, u32x4_t (&o)[2]) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    const f2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 0);
    const f2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 1);
    const f2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 2);
    const f2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 3);
    o[0] = u32x4_t{__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y)};
    o[1] = u32x4_t{__float_as_uint(c.x), __float_as_uint(c.y), __float_as_uint(d.x), __float_as_uint(d.y)};
  }
};

}  // namespace sffn
