// Shared device helpers of the 8-bit (E4M3) operators: one float32 scale for 128 values along K.
//
// A group with largest magnitude a is stored as the codes of x * inv, inv = fl32(448 / a'), under the
// scale s = fl32(a' * fl32(1 / 448)), a' = max(a, 2^-100): 448 is the largest E4M3 number, so the
// group's maximum takes the top code, and the floor gives a group of zeros a finite scale and a finite
// inv. fl(a' inv) is at most 448 (1 + 2^-23), which rounds to 448: nothing has to be clamped.
// Magnitudes are compared as the bit patterns of |x|, whose unsigned order is that of the numbers with
// infinity and then NaN above them: a NaN anywhere makes its whole group NaN, an infinity gives the
// scale infinity (codes 0, and NaN at the infinity), so no group comes out finite that was not.
#pragma once

#include "operators.hpp"

namespace fp4 {

typedef unsigned v2u __attribute__((ext_vector_type(2)));

// The same at any even address, as rows of an N that is no multiple of 8 begin: global memory takes wide stores there.
typedef v2u v2u_any __attribute__((aligned(2)));
typedef v4u v4u_any __attribute__((aligned(2)));

constexpr int kF8Group = 128;
constexpr unsigned kF8FloorBits = 0x0D800000u;  // 2^-100

__device__ __forceinline__ unsigned abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Maximum over the 16 lanes of a DPP row (lanes 16 i .. 16 i + 15), in every one of them.
__device__ __forceinline__ unsigned row16_max(unsigned m) {
  m = max(m, (unsigned)__builtin_amdgcn_update_dpp(0, (int)m, 0x128, 0xF, 0xF, false));  // row_ror:8
  m = max(m, (unsigned)__builtin_amdgcn_update_dpp(0, (int)m, 0x124, 0xF, 0xF, false));  // row_ror:4
  m = max(m, (unsigned)__builtin_amdgcn_update_dpp(0, (int)m, 0x122, 0xF, 0xF, false));  // row_ror:2
  m = max(m, (unsigned)__builtin_amdgcn_update_dpp(0, (int)m, 0x121, 0xF, 0xF, false));  // row_ror:1
  return m;
}

// Sum over the 64 lanes, the same bits in every one of them (a butterfly of commutative additions).
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int h = 32; h > 0; h >>= 1) v += __shfl_xor(v, h);
  return v;
}

__device__ __forceinline__ float f8_scale(unsigned amax) {
  return __uint_as_float(max(amax, kF8FloorBits)) * (1.0f / 448.0f);
}
__device__ __forceinline__ float f8_inverse(unsigned amax) {
  return 448.0f / __uint_as_float(max(amax, kF8FloorBits));
}

// Eight float32 values times inv -> eight E4M3 codes (round to nearest, ties to even), element i in byte i.
__device__ __forceinline__ v2u f8_codes8(const float* v, float inv) {
  int a = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * inv, v[1] * inv, 0, false);
  a = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * inv, v[3] * inv, a, true);
  int b = __builtin_amdgcn_cvt_pk_fp8_f32(v[4] * inv, v[5] * inv, 0, false);
  b = __builtin_amdgcn_cvt_pk_fp8_f32(v[6] * inv, v[7] * inv, b, true);
  return v2u{(unsigned)a, (unsigned)b};
}

// Eight bf16 values (16 bytes) -> float32, exact.
__device__ __forceinline__ void widen8(v4u w, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(w[i]);
    v[2 * i + 1] = bf16_hi(w[i]);
  }
}

// Four.
__device__ __forceinline__ void widen4(v2u w, float v[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v[2 * i] = bf16_lo(w[i]);
    v[2 * i + 1] = bf16_hi(w[i]);
  }
}

// Eight float32 values -> bf16 (round to nearest even).
__device__ __forceinline__ v4u narrow8(const float* v) {
  v4u w;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = (unsigned)__builtin_bit_cast(uint16_t, (__bf16)v[2 * i]) |
           ((unsigned)__builtin_bit_cast(uint16_t, (__bf16)v[2 * i + 1]) << 16);
  return w;
}

}  // namespace fp4
