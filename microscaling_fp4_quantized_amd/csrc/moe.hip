// Mixture-of-experts layer for a few tokens over MXFP4 experts (gfx950).
//
//   route    p = softmax(x Wr^T) in float32, the k largest of a token, ties to the lowest index
//   experts  y_t = sum_j p_tj W2[e] H (silu(G[e] H x_t) * (U[e] H x_t)),  e = ids_tj,  H the block Hadamard rotation
//
// The experts are bound by reading the used experts' weights, 3 D I (1/2 + 1/32) bytes each, so the kernels
// stream those once and multiply them as they lie in memory, by v_mfma_scale_f32_16x16x128_f8f6f4 with E2M1 codes and
// their E8M0 scales as the row operand. Its column operand may be E4M3, and a few tokens leave most of
// its 16 columns free, so an activation is not rounded to 8 bits: it is stored as a sum of THREE E4M3 terms,
//   v / s = q0 + q1 / 16 + q2 / 256,  q_i = e4m3(what is left * 16^i),  s a power of two per 32 values,
// each rounding leaving at most 2^-4 of what it rounds, so at most 2^-12 of v (or 2^-18 of the group's largest) is
// lost, where bf16 would lose 2^-9. The three terms are three columns of one instruction, 5 tokens to
// 16 columns, and are added in float32 at the end. The factors 16^-i ride in the E8M0 scale operand.
//
// Steps of a call (each a launch; every sum in a fixed order):
//   split x    rotate (float32), split into terms                  [T, 3, D]
//   up         per expert and 16 features of h: gate and up rows, silu(g) * u in float32   [T k, I]
//   split h    rotate, split                                       [T k, 3, I]
//   down       per expert and 32 output features                   [T k, D] float32
//   combine    y_t = sum_j p_tj * down, over the slots in order, rounded once to bf16
// Workgroup (a, tile) finds the a-th used expert from the ids itself: a bit per expert in LDS.
#include <atomic>
#include <type_traits>

#include "fp8_device.hpp"
#include "quant_device.hpp"
#include "../../include/fp4.h"

namespace fp4 {
namespace {

typedef __attribute__((address_space(3))) void lds_void;

// ---- route -----------------------------------------------------------------------------------------------------------

constexpr int kRouteWaves = 8;

// Logits of 16 experts x 16 tokens: v_mfma_f32_16x16x32_bf16, products of bf16 exact in float32, the waves
// taking slices of 128 along D. Lane group g takes 32 consecutive elements of the slice for both operands.
__global__ __launch_bounds__(kRouteWaves * 64) void route_logits(const uint16_t* __restrict__ X, int64_t ldx,
                                                                 const uint16_t* __restrict__ Wr, int T, int E, int D,
                                                                 float* __restrict__ logits) {
  __shared__ v4f red[kRouteWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
  const int e0 = blockIdx.x * 16, t0 = blockIdx.y * 16;
  const uint16_t* w = Wr + (size_t)min(e0 + r, E - 1) * D + 32 * g;
  const uint16_t* x = X + (size_t)min(t0 + r, T - 1) * ldx + 32 * g;
  v4f acc = {0.f, 0.f, 0.f, 0.f};
  for (int s = wave; s < D / 128; s += kRouteWaves) {
    v4u a[4], b[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      a[u] = *reinterpret_cast<const v4u*>(w + (size_t)s * 128 + 8 * u);
      b[u] = *reinterpret_cast<const v4u*>(x + (size_t)s * 128 + 8 * u);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a[u]), __builtin_bit_cast(v8bf, b[u]), acc, 0,
                                                    0, 0);
  }
  red[wave][lane] = acc;
  __syncthreads();
  if (wave != 0) return;
  v4f sum = red[0][lane];
#pragma unroll
  for (int i = 1; i < kRouteWaves; ++i) sum += red[i][lane];
  // lane holds experts e0 + 4 g + i of token t0 + r
  if (t0 + r >= T) return;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (e0 + 4 * g + i < E) logits[(size_t)(t0 + r) * E + e0 + 4 * g + i] = sum[i];
}

constexpr int kMaxExperts = 1024;
constexpr int kRouteRegs = kMaxExperts / 64;

// Unsigned order of float values: larger value, larger key; NaN below every number, and 0 below all.
__device__ __forceinline__ unsigned order_key(float v) {
  const unsigned b = __float_as_uint(v);
  if ((b & 0x7FFFFFFFu) > 0x7F800000u) return 1u;
  if (b == 0x80000000u) return 0x80000001u;  // -0 equals +0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u) + 1u;
}

// One wave per token: softmax over E logits, then k rounds of the largest remaining logit (lowest index first).
__global__ __launch_bounds__(256) void route_topk(const float* __restrict__ logits, int T, int E, int k, int renorm,
                                                  int* __restrict__ ids, float* __restrict__ weights) {
  const int lane = threadIdx.x & 63, t = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= T) return;
  float v[kRouteRegs];
  unsigned key[kRouteRegs];
  float m = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < kRouteRegs; ++i) {
    const int e = i * 64 + lane;
    v[i] = e < E ? logits[(size_t)t * E + e] : -__builtin_inff();
    key[i] = e < E ? order_key(v[i]) : 0u;
    m = fmaxf(m, v[i]);
  }
#pragma unroll
  for (int h = 32; h > 0; h >>= 1) m = fmaxf(m, __shfl_xor(m, h));
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kRouteRegs; ++i)
    if (i * 64 + lane < E) sum += expf(v[i] - m);
  sum = wave_sum(sum);
  float mine = 0.f, chosen = 0.f;
  int my_id = 0;
  for (int j = 0; j < k; ++j) {
    unsigned best = 0, at = 0;
#pragma unroll
    for (int i = 0; i < kRouteRegs; ++i)
      if (key[i] > best) best = key[i], at = i * 64 + lane;
#pragma unroll
    for (int h = 32; h > 0; h >>= 1) {
      const unsigned ob = __shfl_xor(best, h), oa = __shfl_xor(at, h);
      if (ob > best || (ob == best && oa < at)) best = ob, at = oa;
    }
    float p = 0.f;
#pragma unroll
    for (int i = 0; i < kRouteRegs; ++i)
      if ((unsigned)(i * 64 + lane) == at) {
        p = expf(v[i] - m) / sum;
        key[i] = 0;
      }
    p = __shfl(p, at & 63);
    chosen += p;
    if (lane == j) mine = p, my_id = at;
  }
  if (lane < k) {
    ids[(size_t)t * k + lane] = my_id;
    weights[(size_t)t * k + lane] = renorm ? mine / chosen : mine;
  }
}

// ---- experts ---------------------------------------------------------------------------------------------------------

constexpr int kTerms = 3;
constexpr int kTokens = 5;           // tokens per fragment of 16 columns
constexpr int kMaxFrags = 4;         // fragments per pass over an expert's weights
constexpr int kWaves = 4;
constexpr int kThreads = kWaves * 64;
constexpr int kSlice = 256;          // bytes (512 elements) of a row per slice
constexpr int kSliceBytes = 16 * kSlice;
constexpr int kRing = 2;             // slices a wave holds or has in flight
constexpr int kMaxPairs = FP4_MOE_MAX_TOKENS * FP4_MOE_MAX_TOPK;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_rsrc(const void* base, unsigned bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00020000);
}

// Rotate 32 values (a chunk of the Hadamard block, see fwht) and write their terms and the group's E8M0
// code. The code puts the group's largest magnitude into (224, 448], and is at least 8, so that the terms'
// codes, 4 less each, stay codes. A group that is not finite gets NaN terms.
template <int B>
__device__ __forceinline__ void split_chunk(float v[32], uint8_t* q, int64_t term_stride, uint8_t* scale) {
  fwht<B>(v);
  const float c = __uint_as_float(hadamard_constant_bits(B));
  unsigned m = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    v[i] *= c;
    m = max(m, abs_bits(v[i]));
  }
  // |max| = 1.f * 2^(e - 127); 448 = 1.75 * 2^8
  const int e = (int)(m >> 23) - 8 + ((m & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  const int code = e < 8 ? 8 : e;
  const bool finite = m < 0x7F800000u;
  const float inv = __uint_as_float((unsigned)(254 - code) << 23);  // 2^(127 - code), code <= 247
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] *= inv;
#pragma unroll
  for (int t = 0; t < kTerms; ++t) {
    unsigned w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      int b = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i], v[4 * i + 1], 0, false);
      b = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2], v[4 * i + 3], b, true);
      const v2f lo = __builtin_amdgcn_cvt_pk_f32_fp8(b, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(b, true);
      v[4 * i] = (v[4 * i] - lo[0]) * 16.f;
      v[4 * i + 1] = (v[4 * i + 1] - lo[1]) * 16.f;
      v[4 * i + 2] = (v[4 * i + 2] - hi[0]) * 16.f;
      v[4 * i + 3] = (v[4 * i + 3] - hi[1]) * 16.f;
      w[i] = finite ? (unsigned)b : 0x7F7F7F7Fu;
    }
    v4u* dst = reinterpret_cast<v4u*>(q + t * term_stride);
    dst[0] = v4u{w[0], w[1], w[2], w[3]};
    dst[1] = v4u{w[4], w[5], w[6], w[7]};
  }
  *scale = (uint8_t)(finite ? code : 127);
}

// Rows of `cpr` chunks of 32 values -> terms [row][3][32 cpr] and scales [row][cpr]; one lane a chunk. The
// 2 or 4 chunks of a Hadamard block of 64 or 128 sit in adjacent lanes (cpr % 4 == 0).
template <int B, bool F32>
__global__ __launch_bounds__(256) void split_rows(const void* __restrict__ V, int64_t ld, int rows, int cpr,
                                                  uint8_t* __restrict__ q, uint8_t* __restrict__ scales) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= rows * cpr) return;  // whole quads: rows * cpr % 4 == 0
  const int row = c / cpr, at = c - row * cpr;
  float v[32];
  if constexpr (F32) {
    const v4f* p = reinterpret_cast<const v4f*>(reinterpret_cast<const float*>(V) + row * ld + at * 32);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const v4f w = p[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * i + j] = w[j];
    }
  } else {
    const v4u* p = reinterpret_cast<const v4u*>(reinterpret_cast<const uint16_t*>(V) + row * ld + at * 32);
#pragma unroll
    for (int i = 0; i < 4; ++i) widen8(p[i], v + 8 * i);
  }
  const int64_t K = 32 * (int64_t)cpr;
  split_chunk<B>(v, q + row * kTerms * K + at * 32, K, scales + c);
}

// The a-th used expert (in index order) and its pairs (t k + slot, in order) into list[]; the number of pairs,
// 0 if fewer than a + 1 experts are used. Ids outside [0, E) name no expert. Every thread calls this.
__device__ __forceinline__ int find_expert(const int* __restrict__ ids, int pairs, int E, int a, int* used,
                                           int* list, int* found, int& expert) {
  const int tid = threadIdx.x, lane = tid & 63;
  for (int i = tid; i < kMaxExperts / 32; i += kThreads) used[i] = 0;
  __syncthreads();
  for (int p = tid; p < pairs; p += kThreads) {
    const int e = ids[p];
    if (e >= 0 && e < E) atomicOr(&used[e >> 5], 1 << (e & 31));
  }
  __syncthreads();
  if (tid < 64) {
    unsigned bits = lane < kMaxExperts / 32 ? (unsigned)used[lane] : 0u;
    const int mine = __popc(bits);
    int before = mine;
#pragma unroll
    for (int h = 1; h < 64; h <<= 1) {
      const int o = __shfl_up(before, h);
      if (lane >= h) before += o;
    }
    before -= mine;
    if (lane == 0) found[0] = -1;
    __builtin_amdgcn_wave_barrier();
    if (a >= before && a < before + mine) {
      for (int j = before; j < a; ++j) bits &= bits - 1;
      found[0] = lane * 32 + __ffs(bits) - 1;
    }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);
    const int e = *(volatile int*)found;
    int n = 0;
    if (e >= 0) {
      for (int p0 = 0; p0 < pairs; p0 += 64) {
        const bool hit = p0 + lane < pairs && ids[p0 + lane] == e;
        const uint64_t mask = __ballot(hit);
        if (hit) list[n + __popcll(mask & ((1ull << lane) - 1))] = p0 + lane;
        n += __popcll(mask);
      }
    }
    if (lane == 0) found[1] = n;
  }
  __syncthreads();
  expert = found[0];
  return found[1];
}

// Two tiles of 16 rows of one expert's matrix by MF fragments of 5 tokens: the slices of 512 elements along K
// go to the waves in turn, each through its own LDS ring by the LDS DMA; the waves' sums meet in LDS in order.
// xq [row][3][K], xs [row][K / 32]; rowof[j]: the row of xq that token j of this pass has, n tokens.
// Afterwards sums[tile][f][col][feature] (float32) is in LDS for all threads.
template <int MF>
__device__ __forceinline__ void expert_tiles(uint8_t* lds, const uint8_t* __restrict__ w0, const uint8_t* __restrict__ w1,
                                             const uint8_t* __restrict__ s0, const uint8_t* __restrict__ s1, int K,
                                             const uint8_t* __restrict__ xq, const uint8_t* __restrict__ xs,
                                             const int* rowof, int n) {
  constexpr int area_bytes = kRing * 2 * kSliceBytes;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const unsigned KB = (unsigned)K / 2, KS = (unsigned)K / 32;
  const int steps = K / 128, nsl = (steps + 3) / 4;
  const int mine = nsl > wave ? (nsl - wave + kWaves - 1) / kWaves : 0;
  uint8_t* area = lds + wave * area_bytes;
  auto fetch = [&](int j) {
    const unsigned at = (unsigned)(wave + kWaves * j) * kSlice;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const __amdgpu_buffer_rsrc_t rw = buffer_rsrc(t ? w1 : w0, 16u * KB);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 4 * i + g;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)(area + ((j % kRing) * 2 + t) * kSliceBytes + i * 1024), 16,
                                                 (unsigned)row * KB + at + 16u * (unsigned)(r ^ row), 0, 0, 0);
      }
    }
  };
  const uint8_t* xp[MF];
  const uint8_t* xsp[MF];
  const int term = r % kTerms;  // column 15 repeats a term and is not read
#pragma unroll
  for (int f = 0; f < MF; ++f) {
    const int row = rowof[min(kTokens * f + r / kTerms, n - 1)];
    xp[f] = xq + ((size_t)row * kTerms + term) * K + 16 * g;
    xsp[f] = xs + (size_t)row * KS;
  }
  v4f acc[2][MF];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int f = 0; f < MF; ++f) acc[t][f] = v4f{0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < kRing && j < mine; ++j) fetch(j);
  for (int j = 0; j < mine; ++j) {
    const int sl = wave + kWaves * j;
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): the slice has landed
    asm volatile("" ::: "memory");
    const uint8_t* sp0 = s0 + (size_t)r * KS + 16 * sl;
    const uint8_t* sp1 = s1 + (size_t)r * KS + 16 * sl;
    const uint8_t* wa = area + (j % kRing) * 2 * kSliceBytes + r * kSlice;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int step = 4 * sl + u;
      if (step >= steps) break;  // wave-uniform
      const v4u a0 = *reinterpret_cast<const v4u*>(wa + 16 * ((4 * u + g) ^ r));
      const v4u a1 = *reinterpret_cast<const v4u*>(wa + kSliceBytes + 16 * ((4 * u + g) ^ r));
      const v8i A0 = {(int)a0[0], (int)a0[1], (int)a0[2], (int)a0[3], 0, 0, 0, 0};
      const v8i A1 = {(int)a1[0], (int)a1[1], (int)a1[2], (int)a1[3], 0, 0, 0, 0};
      const int sa0 = sp0[4 * u + g], sa1 = sp1[4 * u + g];
#pragma unroll
      for (int f = 0; f < MF; ++f) {
        // E4M3 operand: a lane group's 32 bytes are elements 16 g .. and 64 + 16 g .. of the step's 128
        // (measured); block b of 32 elements is scaled by the byte of lane group b for either operand
        const v4u x0 = *reinterpret_cast<const v4u*>(xp[f] + (size_t)step * 128);
        const v4u x1 = *reinterpret_cast<const v4u*>(xp[f] + (size_t)step * 128 + 64);
        const v8i B = {(int)x0[0], (int)x0[1], (int)x0[2], (int)x0[3], (int)x1[0], (int)x1[1], (int)x1[2], (int)x1[3]};
        const int sb = xsp[f][4 * step + g] - 4 * term;
        acc[0][f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A0, B, acc[0][f], 4, 0, 0, sa0, 0, sb);
        acc[1][f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A1, B, acc[1][f], 4, 0, 0, sa1, 0, sb);
      }
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);  // the slice has been read before its slot is refilled
    asm volatile("" ::: "memory");
    if (j + kRing < mine) fetch(j + kRing);
  }
  v4f* red = reinterpret_cast<v4f*>(area);
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int f = 0; f < MF; ++f) red[(t * MF + f) * 64 + 4 * r + g] = acc[t][f];
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * MF * 64; i += kThreads) {
    v4f sum = reinterpret_cast<const v4f*>(lds)[i];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) sum += reinterpret_cast<const v4f*>(lds + w * area_bytes)[i];
    reinterpret_cast<v4f*>(lds)[i] = sum;  // its own element of wave 0's area
  }
  __syncthreads();
}

// Sum of the three terms of token j (of a pass) and feature i of tile t.
template <int MF>
__device__ __forceinline__ float term_sum(const uint8_t* lds, int t, int j, int i) {
  const float* s = reinterpret_cast<const float*>(lds) + ((t * MF + j / kTokens) * 16 + (j % kTokens) * kTerms) * 16 + i;
  return (s[0] + s[16]) + s[32];
}

struct ExpertArgs {
  const int* ids;
  int pairs, k, E, D, I;
  const uint8_t *wq, *ws;  // the experts' matrices
  const uint8_t *xq, *xs;  // terms and scales of the rows
  float* out;
};

// UP: h[pair][f0 .. f0 + 15] = silu(gate) * up.  Not UP: out[pair][n0 .. n0 + 31].
template <bool UP, int MF>
__device__ __forceinline__ void expert_pass(uint8_t* lds, const ExpertArgs& A, int e, int tile, const int* list, int* rowof,
                                            int n) {
  const int K = UP ? A.D : A.I;
  const size_t KB = K / 2, KS = K / 32, base = (size_t)e * (UP ? 2 * A.I : A.D);
  const size_t r0 = base + (UP ? 16 * tile : 32 * tile), r1 = r0 + (UP ? A.I : 16);
  for (int j = threadIdx.x; j < n; j += kThreads) rowof[j] = UP ? list[j] / A.k : list[j];
  __syncthreads();
  expert_tiles<MF>(lds, A.wq + r0 * KB, A.wq + r1 * KB, A.ws + r0 * KS, A.ws + r1 * KS, K, A.xq, A.xs, rowof, n);
  if constexpr (UP) {
    for (int i = threadIdx.x; i < n * 16; i += kThreads) {
      const int j = i >> 4, c = i & 15;
      const float gate = term_sum<MF>(lds, 0, j, c), up = term_sum<MF>(lds, 1, j, c);
      A.out[(size_t)list[j] * A.I + 16 * tile + c] = gate / (1.0f + expf(-gate)) * up;
    }
  } else {
    for (int i = threadIdx.x; i < n * 32; i += kThreads) {
      const int j = i >> 5, c = i & 31;
      A.out[(size_t)list[j] * A.D + 32 * tile + c] = term_sum<MF>(lds, c >> 4, j, c & 15);
    }
  }
  __syncthreads();  // the sums and rowof are read before the next pass
}

template <bool UP>
__global__ __launch_bounds__(kThreads) void expert_gemm(ExpertArgs A, int tiles) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ int used[kMaxExperts / 32], list[kMaxPairs], rowof[kTokens * kMaxFrags], found[2];
  const int a = blockIdx.x / tiles, tile = blockIdx.x % tiles;
  int e;
  const int n = find_expert(A.ids, A.pairs, A.E, a, used, list, found, e);
  if (n == 0) return;
  for (int j = 0; j < n; j += kTokens * kMaxFrags) {
    const int m = min(n - j, kTokens * kMaxFrags);
    if (m <= kTokens) expert_pass<UP, 1>(lds, A, e, tile, list + j, rowof, m);
    else if (m <= 2 * kTokens) expert_pass<UP, 2>(lds, A, e, tile, list + j, rowof, m);
    else expert_pass<UP, kMaxFrags>(lds, A, e, tile, list + j, rowof, m);
  }
}

// y[t][d .. d + 3] = sum over the slots in order of p * out; slots without an expert add nothing.
__global__ __launch_bounds__(256) void combine(const int* __restrict__ ids, const float* __restrict__ p,
                                               const float* __restrict__ out, int T, int k, int E, int D,
                                               uint16_t* __restrict__ Y) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)T * (D / 4)) return;
  const int t = (int)(i / (D / 4)), d = (int)(i % (D / 4)) * 4;
  v4f y = {0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < k; ++j) {
    const int pair = t * k + j, e = ids[pair];
    if (e < 0 || e >= E) continue;
    const v4f o = *reinterpret_cast<const v4f*>(out + (size_t)pair * D + d);
    const float w = p[pair];
#pragma unroll
    for (int q = 0; q < 4; ++q) y[q] = __builtin_fmaf(w, o[q], y[q]);
  }
  unsigned b[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) b[q] = __builtin_bit_cast(uint16_t, (__bf16)y[q]);
  *reinterpret_cast<v2u*>(Y + (size_t)t * D + d) = v2u{b[0] | b[1] << 16, b[2] | b[3] << 16};
}

template <bool F32>
hipError_t launch_split(int block, const void* V, int64_t ld, int rows, int K, uint8_t* q, uint8_t* s, hipStream_t st) {
  const int cpr = K / 32;
  const dim3 grid((unsigned)(((int64_t)rows * cpr + 255) / 256));
  switch (block) {
    case 16: hipLaunchKernelGGL((split_rows<16, F32>), grid, dim3(256), 0, st, V, ld, rows, cpr, q, s); break;
    case 32: hipLaunchKernelGGL((split_rows<32, F32>), grid, dim3(256), 0, st, V, ld, rows, cpr, q, s); break;
    case 64: hipLaunchKernelGGL((split_rows<64, F32>), grid, dim3(256), 0, st, V, ld, rows, cpr, q, s); break;
    default: hipLaunchKernelGGL((split_rows<128, F32>), grid, dim3(256), 0, st, V, ld, rows, cpr, q, s);
  }
  return hipGetLastError();
}

constexpr int kExpertLds = kWaves * kRing * 2 * kSliceBytes;
static_assert(2 * kMaxFrags * 1024 <= kRing * 2 * kSliceBytes, "the partial sums fit a wave's ring");

// The dynamic LDS limit of both expert kernels, raised once per device.
hipError_t raise_lds_limits() {
  static std::atomic<int> ready[64];
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const bool cached = dev >= 0 && dev < 64;
  if (cached && ready[dev].load(std::memory_order_acquire)) return hipSuccess;
  for (const void* k : {(const void*)expert_gemm<true>, (const void*)expert_gemm<false>}) {
    e = hipFuncSetAttribute(k, hipFuncAttributeMaxDynamicSharedMemorySize, kExpertLds);
    if (e != hipSuccess) return e;
  }
  if (cached) ready[dev].store(1, std::memory_order_release);
  return hipSuccess;
}

}  // namespace
}  // namespace fp4

hipError_t fp4_launch_moe_route(const uint16_t* X, int64_t T, int64_t D, int64_t ldx, const uint16_t* Wr, int64_t E, int k,
                                int renorm, float* logits, int* ids, float* weights, hipStream_t st) {
  using namespace fp4;
  const dim3 grid((unsigned)((E + 15) / 16), (unsigned)((T + 15) / 16));
  hipLaunchKernelGGL(route_logits, grid, dim3(kRouteWaves * 64), 0, st, X, ldx, Wr, (int)T, (int)E, (int)D, logits);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(route_topk, dim3((unsigned)((T + 3) / 4)), dim3(256), 0, st, logits, (int)T, (int)E, k, renorm, ids,
                     weights);
  return hipGetLastError();
}

hipError_t fp4_launch_moe_experts(const uint16_t* X, int64_t T, int64_t D, int64_t ldx, const int* ids,
                                  const float* weights, int k, int64_t E, int64_t I, int block, const uint8_t* W13q,
                                  const uint8_t* W13s, const uint8_t* W2q, const uint8_t* W2s, uint16_t* Y, uint8_t* ws,
                                  hipStream_t st) {
  using namespace fp4;
  const int pairs = (int)T * k, slots = pairs < E ? pairs : (int)E;
  uint8_t* xq = ws;
  uint8_t* xs = ws + FP4_MOE_WS_XS(T, k, D, I);
  float* h = reinterpret_cast<float*>(ws + FP4_MOE_WS_H(T, k, D, I));
  uint8_t* hq = ws + FP4_MOE_WS_HQ(T, k, D, I);
  uint8_t* hs = ws + FP4_MOE_WS_HS(T, k, D, I);
  float* out = reinterpret_cast<float*>(ws + FP4_MOE_WS_OUT(T, k, D, I));
  hipError_t e = raise_lds_limits();
  if (e != hipSuccess) return e;
  e = launch_split<false>(block, X, ldx, (int)T, (int)D, xq, xs, st);
  if (e != hipSuccess) return e;
  ExpertArgs up{ids, pairs, k, (int)E, (int)D, (int)I, W13q, W13s, xq, xs, h};
  hipLaunchKernelGGL(expert_gemm<true>, dim3((unsigned)(slots * (I / 16))), dim3(kThreads), kExpertLds, st, up,
                     (int)(I / 16));
  e = hipGetLastError();
  if (e == hipSuccess) e = launch_split<true>(block, h, I, pairs, (int)I, hq, hs, st);
  if (e != hipSuccess) return e;
  ExpertArgs down{ids, pairs, k, (int)E, (int)D, (int)I, W2q, W2s, hq, hs, out};
  hipLaunchKernelGGL(expert_gemm<false>, dim3((unsigned)(slots * (D / 32))), dim3(kThreads), kExpertLds, st, down,
                     (int)(D / 32));
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(combine, dim3((unsigned)((T * (D / 4) + 255) / 256)), dim3(256), 0, st, ids, weights, out, (int)T, k,
                     (int)E, (int)D, Y);
  return hipGetLastError();
}
