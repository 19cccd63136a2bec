// Device helpers that the attention kernels share: matrix operands from cache values, and maxima and sums across a wave.
#pragma once

#include "paged.hpp"

namespace fp4 {

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kNever = -__builtin_inff();  // the score of a token that a row does not see

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// Both halves of the wave (lane ^ 32), and both halves of each half (lane ^ 16), side by side.
template <int X>
__device__ __forceinline__ void lane_swap(unsigned v, unsigned& a, unsigned& b) {
  static_assert(X == 16 || X == 32, "the two swaps there are");
  const auto r = X == 32 ? __builtin_amdgcn_permlane32_swap(v, v, false, false) : __builtin_amdgcn_permlane16_swap(v, v, false, false);
  a = r[0];
  b = r[1];
}
template <int X>
__device__ __forceinline__ float max_across(float v) {
  unsigned a, b;
  lane_swap<X>(__float_as_uint(v), a, b);
  return fmaxf(__uint_as_float(a), __uint_as_float(b));
}
template <int X>
__device__ __forceinline__ float sum_across(float v) {
  unsigned a, b;
  lane_swap<X>(__float_as_uint(v), a, b);
  return __uint_as_float(a) + __uint_as_float(b);
}

// Four E4M3 codes -> two words of bf16 (exact).
__device__ __forceinline__ v2u bf16_of_codes(unsigned c) {
  const v2bf lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, false), hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, true);
  return v2u{__builtin_bit_cast(unsigned, lo), __builtin_bit_cast(unsigned, hi)};
}

// Two floats -> a word of bf16, a in the low half (to nearest even).
__device__ __forceinline__ unsigned bf16_pair(float a, float b) {
  const v2bf v{(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(unsigned, v);
}

// Both halves of a word of bf16 and c, in float32.
__device__ __forceinline__ float add_pair(unsigned w, float c) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(v2bf, w), v2bf{(__bf16)1.f, (__bf16)1.f}, c, false);
}

// What a load brought, waited for here: its first use inside a loop would wait there in every round, and for all loads since.
template <class T>
__device__ __forceinline__ void arrived(T& x) {
  v4u w = __builtin_bit_cast(v4u, x);
  asm volatile("" : "+v"(w));
  x = __builtin_bit_cast(T, w);
}

// The same number, from here on as far as the compiler knows: what follows from it is computed where it is needed and holds no registers
// from before. An offset of 32 bits goes into a load with its scalar address so; addresses made ahead of the loop took 64 bits each.
__device__ __forceinline__ unsigned here(unsigned x) {
  asm volatile("" : "+v"(x));
  return x;
}

// A word that all lanes read alike and that no kernel running now writes, into scalar registers.
__device__ __forceinline__ int uniform_load(const int* p) {
  return *(const __attribute__((address_space(4))) int*)(reinterpret_cast<uintptr_t>(p));
}

// Partial results in the workspace: n outputs of D over their own maxima, then n maxima and sums.
struct Parts {
  float* o;
  v2f* ml;
};
__device__ __forceinline__ Parts parts_of(void* workspace, size_t n, int dim) {
  float* o = static_cast<float*>(workspace);
  return {o, reinterpret_cast<v2f*>(o + n * dim)};
}
// What a partial result counts under the common maximum m. Without a maximum its sum is 0, or NaN where a score was.
__device__ __forceinline__ float share_of(v2f ml, float m) { return ml[0] == kNever ? (ml[1] == 0.f ? 0.f : 1.f) : exp2_hw(ml[0] - m); }

// Another partial result (x, y) into (ml, o).
__device__ __forceinline__ void join_parts(v2f& ml, v4f& o, v2f x, v4f y) {
  const float m = fmaxf(ml[0], x[0]), keep = share_of(ml, m), more = share_of(x, m);
  ml = v2f{m, ml[1] * keep + x[1] * more};
#pragma unroll
  for (int k = 0; k < 4; ++k) o[k] = o[k] * keep + y[k] * more;
}

// The low or the high halves of two words, a's in the low half.
__device__ __forceinline__ unsigned low_halves(unsigned a, unsigned b) { return __builtin_amdgcn_perm(b, a, 0x05040100u); }
__device__ __forceinline__ unsigned high_halves(unsigned a, unsigned b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }

// Partial results first .. last of outputs joined by the 256 threads of a workgroup: `wide` outputs side by side, D / 4 lanes hold one
// of them, the other lanes go over the partial results in turn with them. True for the lanes that have the sum in the end.
template <int D, class Place>
__device__ __forceinline__ bool join_all(const Parts& parts, int wide, int first, int last, Place place, v2f& ml, v4f& o) {
  constexpr int LANES = D / 4, GROUPS = 256 / LANES;
  constexpr int kAtOnce = 4;  // whose loads are in flight together
  __shared__ v4f red[GROUPS][LANES];
  __shared__ v2f red_ml[GROUPS];
  const int g = threadIdx.x / LANES, lane = threadIdx.x % LANES, turns = GROUPS / wide;
  ml = v2f{kNever, 0.f};
  o = v4f{0.f, 0.f, 0.f, 0.f};
  for (int w = first + g / wide; w <= last; w += kAtOnce * turns) {
    v2f x[kAtOnce];
    v4f y[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const size_t at = place(min(w + i * turns, last));
      x[i] = parts.ml[at];
      y[i] = *reinterpret_cast<const v4f*>(parts.o + at * D + 4 * lane);
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
      if (w + i * turns <= last) join_parts(ml, o, x[i], y[i]);
  }
  if (turns == 1) return true;
  red[g][lane] = o;
  if (lane == 0) red_ml[g] = ml;
  __syncthreads();
  if (g >= wide) return false;
  for (int i = g + wide; i < GROUPS; i += wide) join_parts(ml, o, red_ml[i], red[i][lane]);
  return true;
}

}  // namespace fp4
