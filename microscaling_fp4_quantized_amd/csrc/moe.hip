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
// lost, where bf16 would lose 2^-9. The three terms are three columns of one instruction, and are added in float32
// at the end. The factors 16^-i ride in the E8M0 scale operand. A token takes four columns (the fourth is zero), 4
// tokens to 16: a quad of lanes then reads 64 bytes that lie together. The cache serves a quad's line per clock, and
// 16-byte pieces of four different rows four times slower (38 against 150 B/ns a CU).
//
// Steps of a call (each a launch; every sum in a fixed order):
//   split x    rotate (float32), split into terms   [T, 4, D]; one more workgroup sorts the pairs by expert
//   up         per used expert and 32 features of h: gate and up rows, silu(g) * u in float32   [T k, I]
//   split h    rotate, split                                                                    [T k, 4, I]
//   down       per used expert and 64 output features, float32                                  [T k, D]
//   combine    y_t = sum_j p_tj * down, over the slots in order, rounded once to bf16
// Few pairs take two launches instead (few_experts below).
//
// 64 tokens, 6 of 64 experts of 4096 x 1408 (588 MB of weights): 143 us; up 79 us (5.0 TB/s), down 52 (3.8), the other
// three 5 each. The same workgroups without products, tokens and scales, streaming W alone, take 69 and 43: what is
// left to a plain read of the weights (98 us) is mostly the starts and ends of workgroups.
#include <atomic>
#include <type_traits>

#include "fp8_device.hpp"
#include "quant_device.hpp"
#include "../../include/fp4.h"

namespace fp4 {
namespace {

typedef __attribute__((address_space(3))) void lds_void;

// ---- route -----------------------------------------------------------------------------------------------------------

// Two launches: the logits, bound by the latency of reading Wr, and the choice, bound by that of k rounds of a wave.
// D is split over kRouteSplit workgroups of kRouteWaves waves each, so that a wave has one or two loads of 16 experts'
// rows to wait for even for one token; the choice adds the splits' sums in order. (8 of 128 experts, D 2048, 1 token:
// 4.6 + 9.2 us with D in one workgroup and all of k rounds over 1024 experts' registers, now 3.0 + 3.0 us.)
constexpr int kRouteWaves = 4, kRouteSplit = FP4_MOE_ROUTE_SPLIT;

// Partial logits of 16 experts x 16 tokens: v_mfma_f32_16x16x32_bf16, products of bf16 exact in float32, the waves
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
  for (int s = blockIdx.z * kRouteWaves + wave; s < D / 128; s += kRouteSplit * kRouteWaves) {
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
  float* dst = logits + ((size_t)blockIdx.z * T + t0 + r) * E + e0 + 4 * g;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (e0 + 4 * g + i < E) dst[i] = sum[i];
}

constexpr int kMaxExperts = 1024;

// Unsigned order of float values: larger value, larger key; NaN below every number, and 0 below all.
__device__ __forceinline__ unsigned order_key(float v) {
  const unsigned b = __float_as_uint(v);
  if ((b & 0x7FFFFFFFu) > 0x7F800000u) return 1u;
  if (b == 0x80000000u) return 0x80000001u;  // -0 equals +0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u) + 1u;
}

// Maximum over the 64 lanes, uniform: rows of 16 by DPP rotations, then the four rows' by v_readlane.
__device__ __forceinline__ unsigned wave_max(unsigned m) {
  m = row16_max(m);
  const unsigned a = __builtin_amdgcn_readlane(m, 0), b = __builtin_amdgcn_readlane(m, 16);
  const unsigned c = __builtin_amdgcn_readlane(m, 32), d = __builtin_amdgcn_readlane(m, 48);
  return max(max(a, b), max(c, d));
}

// One wave per token: softmax over E <= 64 R logits, then k rounds of the largest remaining logit (lowest index
// first). Expert i * 64 + lane is in register i.
template <int R>
__global__ __launch_bounds__(256) void route_topk(const float* __restrict__ logits, int T, int E, int k, int renorm,
                                                  int* __restrict__ ids, float* __restrict__ weights) {
  const int lane = threadIdx.x & 63, t = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= T) return;
  float v[R];
  unsigned key[R], top = 0;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int e = min(i * 64 + lane, E - 1);
    float z[kRouteSplit];
#pragma unroll
    for (int s = 0; s < kRouteSplit; ++s) z[s] = logits[((size_t)s * T + t) * E + e];
    v[i] = z[0];
#pragma unroll
    for (int s = 1; s < kRouteSplit; ++s) v[i] += z[s];
  }
  // the largest number: keys of numbers are above 1
#pragma unroll
  for (int i = 0; i < R; ++i) {
    key[i] = i * 64 + lane < E ? order_key(v[i]) : 0u;
    top = max(top, key[i]);
  }
  top = wave_max(top);
  const float m = top <= 1u ? 0.f  // NaN throughout
                  : top > 0x80000000u ? __uint_as_float((top - 1u) & 0x7FFFFFFFu) : __uint_as_float(~top);
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    v[i] = expf(v[i] - m);
    if (i * 64 + lane < E) sum += v[i];
  }
  sum = wave_sum(sum);
  float mine = 0.f, chosen = 0.f;
  int my_id = 0;
  for (int j = 0; j < k; ++j) {
    unsigned best = key[0];
#pragma unroll
    for (int i = 1; i < R; ++i) best = max(best, key[i]);
    best = wave_max(best);
    bool found = false;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const uint64_t mask = __ballot(key[i] == best);
      if (!found && mask != 0) {  // uniform: the lowest register, then the lowest lane
        found = true;
        const int at = __ffsll((unsigned long long)mask) - 1;
        const float p = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v[i]), at)) / sum;
        chosen += p;
        if (lane == j) mine = p, my_id = i * 64 + at;
        if (lane == at) key[i] = 0;
      }
    }
  }
  if (lane < k) {
    ids[(size_t)t * k + lane] = my_id;
    weights[(size_t)t * k + lane] = renorm ? mine / chosen : mine;
  }
}

// ---- experts ---------------------------------------------------------------------------------------------------------

constexpr int kTerms = 3;
constexpr int kCols = 4;             // columns of a token: its terms, and zeros
constexpr int kTokens = 16 / kCols;  // tokens per fragment of 16 columns
constexpr int kMaxFrags = 4;         // fragments per pass over an expert's weights
constexpr int kTiles = 4;            // tiles of 16 rows per wave
constexpr int kHalf = 128;           // bytes (256 elements) of a row per half slice
constexpr int kHalfBytes = kTiles * 16 * kHalf;
constexpr int kRing = 2;             // half slices a wave holds or has in flight
constexpr int kScaleRow = 128;       // scale bytes of a row in LDS at once: 4096 elements
constexpr int kScaleBytes = kTiles * 16 * kScaleRow;

// The pairs (t k + slot) of one used expert: list[first .. first + n - 1], and the first of them here, so that a
// workgroup has them with its first load; n = 0 past the last used expert.
constexpr int kSlotPairs = 16;
struct Slot {
  int expert, n, first, pad, pairs[kSlotPairs];
};
static_assert(sizeof(Slot) + 4 == FP4_MOE_WS_PLAN_PAIR, "the plan's bytes per pair");

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_rsrc(const void* base, unsigned bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00020000);
}

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 0xF) | (0x7 << 4) | (0xF << 8) | (((N >> 4) & 3) << 14));
}

// Where the 16 bytes of elements 128 step + 64 half + 16 g .. + 15 and column c of a row of K elements lie, from the
// row's start (4 K bytes a row): the order in which lane (4 token + c, g) reads them as the product's operand. (An
// E4M3 operand's lane group g takes elements 16 g .. and 64 + 16 g .. of an instruction's 128: measured.)
__device__ __forceinline__ int term_offset(int step, int half, int g, int c) {
  return ((step * 2 + half) * 4 + g) * (kCols * 16) + c * 16;
}

// The value of lane l ^ X, X = 1, 2, 4, 8 or 16.
template <int X>
__device__ __forceinline__ unsigned lane_xor(unsigned v) {
  if constexpr (X == 1) return __builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false);  // quad_perm 1 0 3 2
  if constexpr (X == 2) return __builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false);  // quad_perm 2 3 0 1
  if constexpr (X == 4) {  // ^ 7, then ^ 3
    const int w = __builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false);  // row_half_mirror
    return __builtin_amdgcn_update_dpp(0, w, 0x1B, 0xF, 0xF, false);               // quad_perm 3 2 1 0
  }
  if constexpr (X == 8) return __builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xF, 0xF, false);  // row_ror:8
  return __builtin_amdgcn_ds_swizzle((int)v, 0x401F);
}

// A butterfly stage over lanes: the lower lane keeps the sum, the upper one the lower's value minus its own.
template <int X>
__device__ __forceinline__ void butterfly(float v[4], int lane) {
  const unsigned flip = lane & X ? 0x80000000u : 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = __uint_as_float(lane_xor<X>(__float_as_uint(v[i]))) + __uint_as_float(__float_as_uint(v[i]) ^ flip);
}

// Rotate 256 values, 4 l .. 4 l + 3 of them in lane l, and split them: lane l returns the 16 bytes of term l % 4 (zeros
// for the fourth) of values 16 (l / 4) .. + 15, which belong at byte 16 l of the 1 KB that term_offset gives them, and
// the E8M0 code of its chunk of 32 values. The code puts the chunk's largest magnitude into (224, 448], and is at
// least 12, so that the columns' codes, 4 less each, stay codes. A chunk that is not finite gets NaN terms.
// Four values a lane keep all 64 lanes at work where a wave has one such piece (a chunk of 32 a lane, eight lanes
// of 64, took 31.8 us for 4 tokens of 8 of 128 experts of 2048 x 768, this 25.1).
// The lanes of a half wave (128 values) take part together.
template <int B>
__device__ __forceinline__ v4u split_terms(float v[4], int lane, uint8_t& scale) {
  const float s0 = v[0] + v[1], s1 = v[0] - v[1], s2 = v[2] + v[3], s3 = v[2] - v[3];
  v[0] = s0 + s2, v[1] = s1 + s3, v[2] = s0 - s2, v[3] = s1 - s3;
  butterfly<1>(v, lane);
  butterfly<2>(v, lane);
  if constexpr (B >= 32) butterfly<4>(v, lane);
  if constexpr (B >= 64) butterfly<8>(v, lane);
  if constexpr (B >= 128) butterfly<16>(v, lane);
  const float c = __uint_as_float(hadamard_constant_bits(B));
  unsigned m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] *= c;
    m = max(m, abs_bits(v[i]));
  }
  m = max(m, lane_xor<1>(m));
  m = max(m, lane_xor<2>(m));
  m = max(m, lane_xor<4>(m));
  // |max| = 1.f * 2^(e - 127); 448 = 1.75 * 2^8
  const int e = (int)(m >> 23) - 8 + ((m & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  const int code = e < 12 ? 12 : e;
  const bool finite = m < 0x7F800000u;
  const float inv = __uint_as_float((unsigned)(254 - code) << 23);  // 2^(127 - code), code <= 247
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] *= inv;
  unsigned w[kCols] = {0, 0, 0, 0};
#pragma unroll
  for (int t = 0; t < kTerms; ++t) {
    int b = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], b, true);
    const v2f lo = __builtin_amdgcn_cvt_pk_f32_fp8(b, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(b, true);
    v[0] = (v[0] - lo[0]) * 16.f;
    v[1] = (v[1] - lo[1]) * 16.f;
    v[2] = (v[2] - hi[0]) * 16.f;
    v[3] = (v[3] - hi[1]) * 16.f;
    w[t] = finite ? (unsigned)b : 0x7F7F7F7Fu;
  }
  scale = (uint8_t)(finite ? code : 127);
  // transpose over the quad: lane q has word t of its four values, and wants term q of the quad's sixteen
  const bool odd = lane & 1, upper = lane & 2;
  const unsigned r0 = lane_xor<1>(odd ? w[0] : w[1]), r1 = lane_xor<1>(odd ? w[2] : w[3]);
  const unsigned a0 = odd ? r0 : w[0], a1 = odd ? w[1] : r0, b0 = odd ? r1 : w[2], b1 = odd ? w[3] : r1;
  const unsigned c0 = lane_xor<2>(upper ? a0 : b0), c1 = lane_xor<2>(upper ? a1 : b1);
  return upper ? v4u{c0, c1, b0, b1} : v4u{a0, a1, c0, c1};
}

// Sort the pairs by expert: one workgroup of 256 threads. Ids outside [0, E) name no expert. The order of an
// expert's pairs in list[] is that of the counter's updates and decides only which column a token has, never a bit
// of a result.
__device__ __forceinline__ void plan_experts(const int* __restrict__ ids, int pairs, int E, int slots, Slot* slot,
                                             int* list) {
  __shared__ int count[kMaxExperts], first[kMaxExperts], start[kMaxExperts], rank_of[kMaxExperts], total[2][4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int e = tid; e < kMaxExperts; e += 256) count[e] = 0;
  __syncthreads();
  for (int p = tid; p < pairs; p += 256) {
    const int e = ids[p];
    if (e >= 0 && e < E) atomicAdd(&count[e], 1);
  }
  __syncthreads();
  // thread tid takes experts 4 tid .. 4 tid + 3: pairs and used experts before them
  int n[4], pairs_mine = 0, used_mine = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    n[i] = count[4 * tid + i];
    pairs_mine += n[i];
    used_mine += n[i] > 0;
  }
  int at = pairs_mine, rank = used_mine;  // inclusive sums over the wave, then the waves before
#pragma unroll
  for (int h = 1; h < 64; h <<= 1) {
    const int x = __shfl_up(at, h), y = __shfl_up(rank, h);
    if (lane >= h) at += x, rank += y;
  }
  if (lane == 63) total[0][wave] = at, total[1][wave] = rank;
  __syncthreads();
  at -= pairs_mine;
  rank -= used_mine;
  int used = 0;
  for (int w = 0; w < 4; ++w) {
    if (w < wave) at += total[0][w], rank += total[1][w];
    used += total[1][w];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    first[4 * tid + i] = at;
    if (n[i] > 0) {
      slot[rank].expert = 4 * tid + i;
      slot[rank].n = n[i];
      slot[rank].first = at;
      rank_of[4 * tid + i] = rank++;
      start[4 * tid + i] = at;
    }
    at += n[i];
  }
  for (int i = used + tid; i < slots; i += 256) slot[i].n = 0;
  __syncthreads();
  for (int p = tid; p < pairs; p += 256) {
    const int e = ids[p];
    if (e < 0 || e >= E) continue;
    const int j = atomicAdd(&first[e], 1);
    list[j] = p;
    if (j - start[e] < kSlotPairs) slot[rank_of[e]].pairs[j - start[e]] = p;
  }
}

struct PlanArgs {
  const int* ids;
  int pairs, E, slots;
  Slot* slot;
  int* list;
};

// Rows of `quads` groups of 4 values -> terms (16 bytes a group) and scales [row][quads / 8], a group a lane. A row is
// whole half waves (K % 128 == 0). With PLAN, the first workgroup sorts the pairs instead.
template <int B, bool PLAN>
__global__ __launch_bounds__(256) void split_rows(const void* __restrict__ V, int64_t ld, int rows, int quads,
                                                  uint8_t* __restrict__ q, uint8_t* __restrict__ scales, PlanArgs P) {
  if (PLAN && blockIdx.x == 0) {
    plan_experts(P.ids, P.pairs, P.E, P.slots, P.slot, P.list);
    return;
  }
  const unsigned c = (blockIdx.x - (PLAN ? 1 : 0)) * 256 + threadIdx.x;
  if (c >= (unsigned)rows * quads) return;
  const unsigned row = c / quads, at = c - row * quads;
  float v[4];
  if constexpr (!PLAN) {  // h, float32
    const v4f w = *reinterpret_cast<const v4f*>(reinterpret_cast<const float*>(V) + row * ld + at * 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = w[i];
  } else {  // x, bf16
    widen4(*reinterpret_cast<const v2u*>(reinterpret_cast<const uint16_t*>(V) + row * ld + at * 4), v);
  }
  uint8_t scale;
  const v4u terms = split_terms<B>(v, threadIdx.x & 63, scale);
  *reinterpret_cast<v4u*>(q + (size_t)c * 16) = terms;
  if (threadIdx.x % 8 == 0) scales[c / 8] = scale;
}

// The three terms of token j are columns 4 j .. 4 j + 2 of a DPP row: lane (4 j, g) ends with their sums for features
// 4 g .. 4 g + 3.
__device__ __forceinline__ v4f term_sums(v4f v) {
  v4f y;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int b = __float_as_int(v[i]);
    y[i] = (v[i] + __int_as_float(__builtin_amdgcn_update_dpp(0, b, 0x101, 0xF, 0xF, false))) +  // row_shl:1
           __int_as_float(__builtin_amdgcn_update_dpp(0, b, 0x102, 0xF, 0xF, false));             // row_shl:2
  }
  return y;
}

struct ExpertArgs {
  const Slot* slot;
  const int* list;
  int k, D, I;
  const uint8_t *wq, *ws;  // the experts' matrices
  const uint8_t *xq, *xs;  // terms and scales of the rows
  float* out;
};

// W's scale bytes of a workgroup's 64 rows in LDS, up to 128 of a row at a time, so that each line of them is read
// from memory once (read 16 bytes a slice, a third of them came from HBM again, W having pushed them out of the L2
// between slices). Rows of up to 128 bytes lie back to back in memory (32 or 64 of them) and are copied whole; of
// longer rows one window of 128 bytes (4096 elements) is held, the last one ending with the row. Where a row is
// whole 16-byte chunks, chunk q of row r sits at slot (q + r) % chunks: rows 0 .. 7 read the same byte of
// different banks.
struct ScaleWindow {
  int KS, chunks;  // chunks 0: rows as they lie in memory
  __device__ __forceinline__ explicit ScaleWindow(int ks) : KS(ks), chunks(ks > kScaleRow ? 8 : ks % 16 ? 0 : ks / 16) {}
  // First byte of a row in window c.
  __device__ __forceinline__ int start(int c) const { return KS > kScaleRow ? min(c * kScaleRow, KS - kScaleRow) : 0; }

  // Request window c: rows 0 .. 31 and skip .. skip + 31 of the `rows` rows at mat; wave w of S takes its part.
  __device__ __forceinline__ void fetch(uint8_t* lds, const uint8_t* mat, unsigned rows, unsigned skip, int c, int w,
                                        int S) const {
    const int lane = threadIdx.x & 63;
    const __amdgpu_buffer_rsrc_t rs = buffer_rsrc(mat, rows * (unsigned)KS);
    const int units = KS > kScaleRow ? kTiles * 16 * 8 : 4 * KS;  // of 16 bytes
    for (int u0 = 64 * w; u0 < units; u0 += 64 * S) {
      const unsigned u = u0 + lane;
      unsigned off;
      if (chunks == 0) {
        off = 16 * u + (u >= 2u * KS ? (skip - 32) * (unsigned)KS : 0u);
      } else {
        const unsigned r = u / chunks, slot = u - r * chunks, q = (slot + chunks * 64u - r) % chunks;
        off = (r < 32 ? r : r - 32 + skip) * (unsigned)KS + (unsigned)start(c) + 16 * q;
      }
      if (u >= (unsigned)units) off = 0xFFFFFFF0u;  // reads as zero
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(lds + u0 * 16), 16, off, 0, 0, 0);
    }
  }

  // Where byte `at` (uniform) of row r's window lies; rm = r % chunks.
  __device__ __forceinline__ int where(int r, int rm, int at) const {
    if (chunks == 0) return r * KS + at;
    const int slot = (at >> 4) + rm;
    return (r * chunks + (slot >= chunks ? slot - chunks : slot)) * 16 + (at & 15);
  }
};

// 16-byte chunk q of row r of a tile's half slice sits at slot q ^ swz(r): the lanes that ds_read_b128 serves together
// (0-3, 12-15 and 20-27, ...) then read distinct banks.
__device__ __forceinline__ int swz(int r) { return r & 7; }

// Four tiles of 16 rows of an expert's matrix by up to 4 MF tokens, all of K, by a workgroup of S waves. UP: the gate
// and up rows of features 32 tile .. + 31 of h (two tiles each), h[pair] = silu(gate) * up. Not UP: output
// features 64 tile .. + 63.
// Half slice i of 256 elements along K goes to wave i % S, which streams W through its own LDS ring by the LDS DMA, 8
// rows x 128 bytes an instruction; the tokens' terms go to registers, requested two half slices ahead (one, with
// more than two fragments). Four
// tiles share what is read of the tokens (with two, reading it from L2 took a third more time). The waves' sums meet
// once, through LDS, in the order of the waves.
template <bool UP, int S, int MF>
__device__ __forceinline__ void expert_tile(uint8_t* lds, const ExpertArgs& A, const Slot* slot, int tile, int j0, int n) {
  const int K = UP ? A.D : A.I, expert = slot->expert;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const unsigned KB = (unsigned)K / 2, KS = (unsigned)K / 32;
  const int steps = K / 128, nhalf = (steps + 1) / 2;
  const int mine = nhalf > wave ? (nhalf - wave + S - 1) / S : 0;  // this wave's half slices
  const size_t base = (size_t)expert * (UP ? 2 * A.I : A.D) + (UP ? 32 : 64) * (size_t)tile;
  uint8_t* ring = lds + wave * (kRing * kHalfBytes);
  uint8_t* wscl = lds + S * (kRing * kHalfBytes);
  const ScaleWindow win((int)KS);
  auto fetch_scales = [&](int c) {
    win.fetch(wscl, A.ws + base * KS, UP ? A.I + 32u : 64u, UP ? (unsigned)A.I : 32u, c, wave, S);
  };
  auto fetch = [&](int j) {
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      const size_t row0 = base + (UP ? (t >> 1) * A.I + 16 * (t & 1) : 16 * t);
      const __amdgpu_buffer_rsrc_t rw = buffer_rsrc(A.wq + row0 * KB, 16u * KB);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int row = 8 * q + (lane >> 3);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)(ring + (j % kRing) * kHalfBytes + t * 2048 + q * 1024), 16,
                                                 (unsigned)row * KB + (unsigned)(wave + S * j) * kHalf +
                                                     16u * (unsigned)((lane & 7) ^ swz(row)),
                                                 0, 0, 0);
      }
    }
  };
  // DMA loads of a fetch. The counted waits below count these alone: loads return in order, every one of these is issued, and
  // loads to registers, which the compiler may merge, drop or move, can only make such a wait longer than it has to be.
  constexpr int kDma = 2 * kTiles;
  fetch_scales(0);
  if (mine > 0) fetch(0);
  const int col = r % kCols;
  const int* list = A.list + slot->first;
  auto pair_of = [&](int j) { return j < kSlotPairs ? slot->pairs[j] : list[j]; };
  const uint8_t *xp[MF], *xsp[MF];
#pragma unroll
  for (int f = 0; f < MF; ++f) {
    const int pair = pair_of(j0 + min(kTokens * f + r / kCols, n - 1)), row = UP ? pair / A.k : pair;
    xp[f] = A.xq + (size_t)row * K * kCols + term_offset(0, 0, g, col);
    xsp[f] = A.xs + (size_t)row * KS;
  }
  constexpr int XB = MF <= 2 ? 2 : 1;  // half slices of the tokens in registers
  v4u x[XB][MF][2][2];                 // [half slice % XB][fragment][step of it][16 bytes]
  unsigned xs[XB][MF][2];
  auto load_tokens = [&](int j, int h) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int step = min(2 * (wave + S * j) + u, steps - 1);
#pragma unroll
      for (int f = 0; f < MF; ++f) {
        // block b of 32 elements is scaled by the byte of lane group b, for either operand (measured)
        x[h % XB][f][u][0] = *reinterpret_cast<const v4u*>(xp[f] + (size_t)step * (128 * kCols));
        x[h % XB][f][u][1] = *reinterpret_cast<const v4u*>(xp[f] + (size_t)step * (128 * kCols) + 64 * kCols);
        xs[h % XB][f][u] = *reinterpret_cast<const unsigned*>(xsp[f] + 4 * step);
      }
    }
  };
  if (mine > 0) load_tokens(0, 0);
  if (mine > 1) {
    if constexpr (XB == 2) load_tokens(1, 1);
    fetch(1);
  }
  // window 0 has landed: it was requested before both fetches
  if (mine > 1) wait_vmcnt<2 * kDma>();
  else wait_vmcnt<0>();
  __syncthreads();
  v4f acc[kTiles][MF];
#pragma unroll
  for (int t = 0; t < kTiles; ++t)
#pragma unroll
    for (int f = 0; f < MF; ++f) acc[t][f] = v4f{0.f, 0.f, 0.f, 0.f};
  const int rm = win.chunks ? r % win.chunks : 0, rm16 = win.chunks ? 16 % win.chunks : 0;
  constexpr int kWindow = kScaleRow / 8 / S;  // half slices of a wave per window (of rows longer than one)
  const int windows = KS > kScaleRow ? (int)((KS + kScaleRow - 1) / kScaleRow) : 1;
  static_assert(kWindow % 2 == 0, "windows hold whole pairs of half slices");
  for (int c = 0; c < windows; ++c) {
    if (c > 0) {
      __syncthreads();  // every wave has read the window before
      fetch_scales(c);
      wait_vmcnt<0>();
      __syncthreads();
    }
    const int start = win.start(c), end = c + 1 < windows ? (c + 1) * kWindow : mine;
    for (int jj = c * kWindow; jj < end; jj += 2) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int j = jj + h, i = wave + S * j;
        if (j >= mine) break;  // uniform in the wave
        // the half slice has landed: the next one's W was requested after it
        if (j + 1 < mine) wait_vmcnt<kDma>();
        else wait_vmcnt<0>();
        asm volatile("" ::: "memory");
        const uint8_t* wa = ring + (j % kRing) * kHalfBytes + r * kHalf;
        v4u a[2][kTiles];
        unsigned wb[2][kTiles];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          int rt = rm;
#pragma unroll
          for (int t = 0; t < kTiles; ++t) {
            a[u][t] = *reinterpret_cast<const v4u*>(wa + t * 2048 + 16 * ((4 * u + g) ^ swz(r)));
            wb[u][t] = wscl[win.where(16 * t + r, rt, 8 * i + 4 * u - start) + g];
            rt += rm16;
            rt -= rt >= win.chunks ? win.chunks : 0;
          }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (2 * i + u < steps) {  // uniform
#pragma unroll
            for (int f = 0; f < MF; ++f) {
              const v4u x0 = x[h % XB][f][u][0], x1 = x[h % XB][f][u][1];
              const v8i B = {(int)x0[0], (int)x0[1], (int)x0[2], (int)x0[3], (int)x1[0], (int)x1[1], (int)x1[2], (int)x1[3]};
              const int xb = (int)((xs[h % XB][f][u] >> (8 * g)) & 0xFFu) - 4 * col;
#pragma unroll
              for (int t = 0; t < kTiles; ++t) {
                const v8i W = {(int)a[u][t][0], (int)a[u][t][1], (int)a[u][t][2], (int)a[u][t][3], 0, 0, 0, 0};
                acc[t][f] =
                    __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(W, B, acc[t][f], 4, 0, 0, (int)wb[u][t], 0, xb);
              }
            }
          }
        }
        if (j + XB < mine) load_tokens(j + XB, h);
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the half slice has been read before its slot is refilled
        asm volatile("" ::: "memory");
        if (j + kRing < mine) fetch(j + kRing);
      }
    }
  }
  // Partial sums into the wave's own ring, then sum them in the order of the waves.
  v4f* red = reinterpret_cast<v4f*>(ring);
#pragma unroll
  for (int t = 0; t < kTiles; ++t)
#pragma unroll
    for (int f = 0; f < MF; ++f) red[(t * MF + f) * 64 + lane] = acc[t][f];
  __syncthreads();
  auto sum_of = [&](int t, int f) {
    const uint8_t* at = lds + ((t * MF + f) * 64 + lane) * 16;
    v4f v = *reinterpret_cast<const v4f*>(at);
#pragma unroll
    for (int w = 1; w < S; ++w) v += *reinterpret_cast<const v4f*>(at + w * (kRing * kHalfBytes));
    return term_sums(v);
  };
  constexpr int kItems = (UP ? 2 : kTiles) * MF;
  for (int q = wave; q < kItems; q += S) {
    const int t = q / MF, f = q % MF, j = kTokens * f + r / kCols;
    const v4f y = sum_of(t, f);
    v4f up = y;
    if constexpr (UP) up = sum_of(t + 2, f);
    if (col != 0 || j >= n) continue;
    const size_t pair = pair_of(j0 + j);
    if constexpr (UP) {
      v4f h;
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = y[i] / (1.0f + expf(-y[i])) * up[i];
      *reinterpret_cast<v4f*>(A.out + pair * A.I + 32 * tile + 16 * t + 4 * g) = h;
    } else {
      *reinterpret_cast<v4f*>(A.out + pair * A.D + 64 * tile + 16 * t + 4 * g) = y;
    }
  }
}

template <bool UP, int S>
__global__ __launch_bounds__(64 * S) __attribute__((amdgpu_waves_per_eu(2, 8))) void expert_gemm(ExpertArgs A, int tiles) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  const Slot* s = A.slot + blockIdx.x / tiles;
  const int tile = blockIdx.x % tiles, n = s->n;
  for (int j = 0; j < n; j += kTokens * kMaxFrags) {
    if (j > 0) __syncthreads();  // the sums of the pass before have been read
    const int m = min(n - j, kTokens * kMaxFrags);
    if (m <= kTokens) expert_tile<UP, S, 1>(lds, A, s, tile, j, m);
    else if (m <= 2 * kTokens) expert_tile<UP, S, 2>(lds, A, s, tile, j, m);
    else if (m <= 3 * kTokens) expert_tile<UP, S, 3>(lds, A, s, tile, j, m);
    else expert_tile<UP, S, 4>(lds, A, s, tile, j, m);
  }
}

template <bool UP, int S>
hipError_t launch_gemm(const ExpertArgs& A, int slots, int tiles, hipStream_t st) {
  static std::atomic<int> ready[64];
  const int scale_row = (UP ? A.D : A.I) / 32;
  const int lds = S * kRing * kHalfBytes + (scale_row > kScaleRow ? kScaleBytes : (64 * scale_row + 1023) / 1024 * 1024);
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  auto kern = expert_gemm<UP, S>;
  const bool cached = dev >= 0 && dev < 64;
  if (!cached || !ready[dev].load(std::memory_order_acquire)) {
    e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, S * kRing * kHalfBytes + kScaleBytes);
    if (e != hipSuccess) return e;
    if (cached) ready[dev].store(1, std::memory_order_release);
  }
  hipLaunchKernelGGL(kern, dim3((unsigned)(slots * tiles)), dim3(64 * S), lds, st, A, tiles);
  return hipGetLastError();
}

template <bool UP>
hipError_t launch_experts(const ExpertArgs& A, int slots, hipStream_t st) {
  const int tiles = UP ? A.I / 32 : A.D / 64;
  switch (expert_waves(UP ? A.D : A.I, slots * tiles)) {
    case 1: return launch_gemm<UP, 1>(A, slots, tiles, st);
    case 2: return launch_gemm<UP, 2>(A, slots, tiles, st);
    default: return launch_gemm<UP, 8>(A, slots, tiles, st);
  }
}

// ---- a few pairs: two launches ------------------------------------------------------------------------------------------

// Where the pairs are few, five launches cost more than the work: here every pair reads its expert's matrices itself, a
// workgroup of eight waves rotates and splits what it needs of x or of h while its first weights are on their way, and
// the second launch takes all of a token's experts, so that their weighted sum is y.
//   UP      workgroup (pair, 16 features of h): item = half slice (256 elements) of D, of the gate and the up rows
//   not UP  workgroup (token, 16 output features): item = (slot, half slice of I), its product times the slot's weight
// Items go to the waves in turn. A wave splits the vectors of two or four items at a time
// into its own LDS, and streams each item's 32 or 16 rows x 128 bytes of W through its own ring; a single token's columns
// are repeated over the instruction's 16. 8 of 128 experts of 2048 x 768, one token: 25 us
// in five launches, 13 in two; four tokens 41 and 25, eight tokens 47 and 50. 16 waves for the second launch: no faster.
constexpr int kFewWaves = 8;
constexpr int kHalfTerms = 256 * kCols;  // bytes of the terms of a half slice
template <bool UP>
struct Few {
  static constexpr int kTiles = UP ? 2 : 1;  // of 16 rows
  static constexpr int kSlot = kTiles * 2048;
  static constexpr int kItems = UP ? 2 : 4;     // split at once
  static constexpr int kWave = kRing * kSlot + kItems * kHalfTerms;  // LDS of a wave
  static constexpr int kLds = kFewWaves * kWave;
};
static_assert(Few<true>::kLds <= 80 * 1024 && Few<false>::kLds <= 80 * 1024, "two workgroups on a CU");

struct FewArgs {
  const void* v;  // x (bf16) or h (float32)
  int64_t ld;
  const int* ids;
  const float* weights;
  int k, E, D, I;
  const uint8_t *wq, *ws;
  void* out;  // h (float32) or y (bf16)
};

template <bool UP, int B>
__device__ __forceinline__ void few_items(uint8_t* lds, const FewArgs& A, int tiles) {
  constexpr int kTiles = Few<UP>::kTiles, kSlot = Few<UP>::kSlot, kWave = Few<UP>::kWave, kItems = Few<UP>::kItems;
  const int K = UP ? A.D : A.I;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4, col = r % kCols;
  const int who = blockIdx.x / tiles, tile = blockIdx.x % tiles;  // pair or token
  const unsigned KB = (unsigned)K / 2, KS = (unsigned)K / 32;
  const int steps = K / 128, nhalf = (steps + 1) / 2, items = UP ? nhalf : A.k * nhalf;
  const int mine = items > wave ? (items - wave + kFewWaves - 1) / kFewWaves : 0;
  uint8_t* ring = lds + wave * kWave;
  uint8_t* terms = ring + kRing * kSlot;
  uint8_t* tscl = terms + term_offset(0, 0, 0, kTerms);  // scale bytes, in an item's unused column
  auto used = [&](int e) { return e >= 0 && e < A.E; };
  auto pair_of = [&](int m) { return UP ? who : who * A.k + (wave + kFewWaves * m) / nhalf; };
  auto half_of = [&](int m) { return UP ? wave + kFewWaves * m : (wave + kFewWaves * m) % nhalf; };
  auto row0 = [&](int e, int t) {
    return UP ? (size_t)e * 2 * A.I + t * A.I + 16 * (size_t)tile : (size_t)e * A.D + 16 * (size_t)tile;
  };
  using Slot0 = std::integral_constant<int, 0>;
  using Slot1 = std::integral_constant<int, 1>;
  static_assert(kRing == 2 && kItems % kRing == 0, "an item's slot goes by its place in the group");
  unsigned sw[kRing][kTiles][2];
  // W of item m into ring slot m % kRing (`slot`), two DMA loads a tile, also for an unused slot, which reads nothing of W;
  // its scale bytes to registers.
  auto fetch = [&](int m, auto slot) {
    constexpr int b = decltype(slot)::value;
    const int id = A.ids[pair_of(m)], i = half_of(m), e = used(id) ? id : 0;
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int u = 0; u < 2; ++u)
        sw[b][t][u] = *reinterpret_cast<const unsigned*>(A.ws + (row0(e, t) + r) * KS + 4 * min(2 * i + u, steps - 1));
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      const __amdgpu_buffer_rsrc_t rw = buffer_rsrc(A.wq + row0(e, t) * KB, 16u * KB);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int row = 8 * q + (lane >> 3);
        const unsigned off = (unsigned)row * KB + (unsigned)i * kHalf + 16u * (unsigned)((lane & 7) ^ swz(row));
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)(ring + b * kSlot + t * 2048 + q * 1024), 16,
                                                 used(id) ? off : 0xFFFFFFF0u, 0, 0, 0);
      }
    }
  };
  constexpr int kDma = 2 * kTiles;  // DMA loads of a fetch; as in expert_tile, no counted wait counts others

  v4f acc[kTiles];
#pragma unroll
  for (int t = 0; t < kTiles; ++t) acc[t] = v4f{0.f, 0.f, 0.f, 0.f};
  for (int m0 = 0; m0 < mine; m0 += kItems) {
    // The items' values are requested before the ids are known; those of an unused slot's h (whatever lies there) and
    // those past K (of an odd number of steps; the row's last) are split too, and go nowhere.
    typename std::conditional<UP, v2u, v4f>::type raw[kItems];
#pragma unroll
    for (int n = 0; n < kItems; ++n) {
      const int m = min(m0 + n, mine - 1), pair = pair_of(m), at = min(256 * half_of(m) + 4 * lane, K - 4);
      if constexpr (UP) raw[n] = *reinterpret_cast<const v2u*>(static_cast<const uint16_t*>(A.v) + (pair / A.k) * A.ld + at);
      else raw[n] = *reinterpret_cast<const v4f*>(static_cast<const float*>(A.v) + (size_t)pair * K + at);
    }
    if (m0 == 0) {
      if (UP && !used(A.ids[who])) return;  // the whole workgroup
      fetch(0, Slot0{});
      if (mine > 1) fetch(1, Slot1{});
    }
#pragma unroll
    for (int n = 0; n < kItems; ++n) {
      if (m0 + n >= mine) break;  // uniform in the wave
      float v[4];
      if constexpr (UP) {
        widen4(raw[n], v);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = raw[n][j];
      }
      uint8_t scale;
      *reinterpret_cast<v4u*>(terms + n * kHalfTerms + lane * 16) = split_terms<B>(v, lane, scale);
      if (lane % 8 == 0) tscl[n * kHalfTerms + lane / 8] = scale;
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the wave's own LDS
    asm volatile("" ::: "memory");
    auto item = [&](auto slot, int n) __attribute__((always_inline)) {  // item n of the group
      constexpr int b = decltype(slot)::value;
      const int m = m0 + n;
      if (m >= mine) return;  // uniform in the wave
      // the item has landed: the next one's DMA is younger
      if (m + 1 < mine) wait_vmcnt<kDma>();
      else wait_vmcnt<0>();
      asm volatile("" ::: "memory");
      if (used(A.ids[pair_of(m)])) {  // uniform in the wave
        const int i = half_of(m);
        const float weight = UP ? 1.f : A.weights[pair_of(m)];
        v4f p[kTiles];
#pragma unroll
        for (int t = 0; t < kTiles; ++t) p[t] = UP ? acc[t] : v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (2 * i + u < steps) {
            const uint8_t* xt = terms + n * kHalfTerms;
            const v4u x0 = *reinterpret_cast<const v4u*>(xt + term_offset(u, 0, g, col));
            const v4u x1 = *reinterpret_cast<const v4u*>(xt + term_offset(u, 1, g, col));
            const v8i Bv = {(int)x0[0], (int)x0[1], (int)x0[2], (int)x0[3], (int)x1[0], (int)x1[1], (int)x1[2], (int)x1[3]};
            const int xb = (int)tscl[n * kHalfTerms + 4 * u + g] - 4 * col;
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
              const v4u a = *reinterpret_cast<const v4u*>(ring + b * kSlot + t * 2048 + r * kHalf +
                                                          16 * ((4 * u + g) ^ swz(r)));
              const v8i W = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
              p[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(W, Bv, p[t], 4, 0, 0, (int)(sw[b][t][u] >> (8 * g)), 0, xb);
            }
          }
        }
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          if constexpr (UP) {
            acc[t] = p[t];
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[t][j] = __builtin_fmaf(weight, p[t][j], acc[t][j]);
          }
        }
      }
      __builtin_amdgcn_s_waitcnt(0xC07F);  // the item has been read before its slot is refilled
      asm volatile("" ::: "memory");
      if (m + kRing < mine) fetch(m + kRing, slot);
    };
#pragma unroll
    for (int n = 0; n < kItems; n += kRing) {
      item(Slot0{}, n);
      item(Slot1{}, n + 1);
    }
  }
  // The waves' sums in their order, then the terms'; lane (0, g) ends with features 4 g .. + 3 of the tile.
#pragma unroll
  for (int t = 0; t < kTiles; ++t) *reinterpret_cast<v4f*>(ring + t * 1024 + lane * 16) = acc[t];
  __syncthreads();
  if (wave != 0) return;
  auto sum_of = [&](int t) {
    v4f v = *reinterpret_cast<const v4f*>(lds + t * 1024 + lane * 16);
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) v += *reinterpret_cast<const v4f*>(lds + w * kWave + t * 1024 + lane * 16);
    return term_sums(v);
  };
  const v4f y = sum_of(0);
  if constexpr (UP) {
    const v4f up = sum_of(1);
    if (r != 0) return;
    v4f h;
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = y[j] / (1.0f + expf(-y[j])) * up[j];
    *reinterpret_cast<v4f*>(static_cast<float*>(A.out) + (size_t)who * A.I + 16 * tile + 4 * g) = h;
  } else {
    if (r != 0) return;
    unsigned b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = __builtin_bit_cast(uint16_t, (__bf16)y[j]);
    *reinterpret_cast<v2u*>(static_cast<uint16_t*>(A.out) + (size_t)who * A.D + 16 * tile + 4 * g) =
        v2u{b[0] | b[1] << 16, b[2] | b[3] << 16};
  }
}

template <bool UP, int B>
__global__ __launch_bounds__(kFewWaves * 64) void few_experts(FewArgs A, int tiles) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  few_items<UP, B>(lds, A, tiles);
}

template <bool UP, int B>
hipError_t launch_few_block(const FewArgs& A, int blocks, int tiles, hipStream_t st) {
  static std::atomic<int> ready[64];
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  auto kern = few_experts<UP, B>;
  const bool cached = dev >= 0 && dev < 64;
  if (!cached || !ready[dev].load(std::memory_order_acquire)) {
    e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, Few<UP>::kLds);
    if (e != hipSuccess) return e;
    if (cached) ready[dev].store(1, std::memory_order_release);
  }
  hipLaunchKernelGGL(kern, dim3((unsigned)(blocks * tiles)), dim3(kFewWaves * 64), Few<UP>::kLds, st, A, tiles);
  return hipGetLastError();
}

template <bool UP>
hipError_t launch_few(int block, const FewArgs& A, int blocks, hipStream_t st) {
  const int tiles = (UP ? A.I : A.D) / 16;
  switch (block) {
    case 16: return launch_few_block<UP, 16>(A, blocks, tiles, st);
    case 32: return launch_few_block<UP, 32>(A, blocks, tiles, st);
    case 64: return launch_few_block<UP, 64>(A, blocks, tiles, st);
    default: return launch_few_block<UP, 128>(A, blocks, tiles, st);
  }
}

// y[t][d .. d + 3] = sum over the slots in order of p * out, four slots' loads in flight at once; slots without an expert
// add nothing.
constexpr int kCombine = 4;
__global__ __launch_bounds__(256) void combine(const int* __restrict__ ids, const float* __restrict__ p,
                                               const float* __restrict__ out, int T, int k, int E, int D,
                                               uint16_t* __restrict__ Y) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)T * (D / 4)) return;
  const int t = (int)(i / (D / 4)), d = (int)(i % (D / 4)) * 4;
  v4f y = {0.f, 0.f, 0.f, 0.f};
  for (int j0 = 0; j0 < k; j0 += kCombine) {
    int e[kCombine];
    float w[kCombine];
    v4f o[kCombine];
#pragma unroll
    for (int j = 0; j < kCombine; ++j) {
      const int pair = t * k + min(j0 + j, k - 1);
      e[j] = ids[pair];
      w[j] = p[pair];
      o[j] = *reinterpret_cast<const v4f*>(out + (size_t)pair * D + d);  // of an unused slot: whatever lies there
    }
#pragma unroll
    for (int j = 0; j < kCombine; ++j) {
      const bool used = j0 + j < k && e[j] >= 0 && e[j] < E;
#pragma unroll
      for (int q = 0; q < 4; ++q) y[q] = used ? __builtin_fmaf(w[j], o[j][q], y[q]) : y[q];
    }
  }
  unsigned b[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) b[q] = __builtin_bit_cast(uint16_t, (__bf16)y[q]);
  *reinterpret_cast<v2u*>(Y + (size_t)t * D + d) = v2u{b[0] | b[1] << 16, b[2] | b[3] << 16};
}

template <bool PLAN>
hipError_t launch_split(int block, const void* V, int64_t ld, int rows, int K, uint8_t* q, uint8_t* s, const PlanArgs& P,
                        hipStream_t st) {
  const int quads = K / 4;
  const dim3 grid((unsigned)(((int64_t)rows * quads + 255) / 256 + (PLAN ? 1 : 0)));
  switch (block) {
    case 16: hipLaunchKernelGGL((split_rows<16, PLAN>), grid, dim3(256), 0, st, V, ld, rows, quads, q, s, P); break;
    case 32: hipLaunchKernelGGL((split_rows<32, PLAN>), grid, dim3(256), 0, st, V, ld, rows, quads, q, s, P); break;
    case 64: hipLaunchKernelGGL((split_rows<64, PLAN>), grid, dim3(256), 0, st, V, ld, rows, quads, q, s, P); break;
    default: hipLaunchKernelGGL((split_rows<128, PLAN>), grid, dim3(256), 0, st, V, ld, rows, quads, q, s, P);
  }
  return hipGetLastError();
}

}  // namespace
}  // namespace fp4

hipError_t fp4_launch_moe_route(const uint16_t* X, int64_t T, int64_t D, int64_t ldx, const uint16_t* Wr, int64_t E, int k,
                                int renorm, float* logits, int* ids, float* weights, hipStream_t st) {
  using namespace fp4;
  const dim3 grid((unsigned)((E + 15) / 16), (unsigned)((T + 15) / 16), kRouteSplit);
  hipLaunchKernelGGL(route_logits, grid, dim3(kRouteWaves * 64), 0, st, X, ldx, Wr, (int)T, (int)E, (int)D, logits);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  auto topk = E <= 64 ? route_topk<1> : E <= 128 ? route_topk<2> : E <= 256 ? route_topk<4> : route_topk<kMaxExperts / 64>;
  hipLaunchKernelGGL(topk, dim3((unsigned)((T + 3) / 4)), dim3(256), 0, st, logits, (int)T, (int)E, k, renorm, ids,
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
  Slot* slot = reinterpret_cast<Slot*>(ws + FP4_MOE_WS_PLAN(T, k, D, I));
  int* list = reinterpret_cast<int*>(slot + pairs);
  if (few_pairs((int)T, k, E, D, I)) {
    const FewArgs up{X, ldx, ids, weights, k, (int)E, (int)D, (int)I, W13q, W13s, h};
    const hipError_t e = launch_few<true>(block, up, pairs, st);
    if (e != hipSuccess) return e;
    const FewArgs down{h, I, ids, weights, k, (int)E, (int)D, (int)I, W2q, W2s, Y};
    return launch_few<false>(block, down, (int)T, st);
  }
  const PlanArgs plan{ids, pairs, (int)E, slots, slot, list};
  hipError_t e = launch_split<true>(block, X, ldx, (int)T, (int)D, xq, xs, plan, st);
  if (e != hipSuccess) return e;
  const ExpertArgs up{slot, list, k, (int)D, (int)I, W13q, W13s, xq, xs, h};
  e = launch_experts<true>(up, slots, st);
  if (e == hipSuccess) e = launch_split<false>(block, h, I, pairs, (int)I, hq, hs, plan, st);
  if (e != hipSuccess) return e;
  const ExpertArgs down{slot, list, k, (int)D, (int)I, W2q, W2s, hq, hs, out};
  e = launch_experts<false>(down, slots, st);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(combine, dim3((unsigned)((T * (D / 4) + 255) / 256)), dim3(256), 0, st, ids, weights, out, (int)T, k,
                     (int)E, (int)D, Y);
  return hipGetLastError();
}
