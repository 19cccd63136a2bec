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
//   split x    rotate (float32), split into terms   [T, 3, D]; one more workgroup sorts the pairs by expert
//   up         per used expert and 32 features of h: gate and up rows, silu(g) * u in float32   [T k, I]
//   split h    rotate, split                        [T k, 3, I]
//   down       per used expert and 64 output features                                           [T k, D] float32
//   combine    y_t = sum_j p_tj * down, over the slots in order, rounded once to bf16
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
constexpr int kMaxFrags = 2;         // fragments per pass over an expert's weights
constexpr int kTiles = 4;            // tiles of 16 rows per wave
constexpr int kHalf = 128;           // bytes (256 elements) of a row per half slice
constexpr int kHalfBytes = kTiles * 16 * kHalf;
constexpr int kRing = 2;             // half slices a wave holds or has in flight
constexpr int kScaleRow = 128;       // scale bytes of a row in LDS at once: 4096 elements
constexpr int kScaleBytes = kTiles * 16 * kScaleRow;
constexpr int kExpertLds = kRing * kHalfBytes + kScaleBytes;  // 24 KB: six waves on a CU

// The pairs (t k + slot) of one used expert: list[first .. first + n - 1]; n = 0 past the last used expert.
struct Slot {
  int expert, first, n, pad;
};

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

// Sort the pairs by expert: one workgroup of 256 threads. Ids outside [0, E) name no expert. The order of an
// expert's pairs in list[] is that of the counter's updates and decides only which column a token has, never a bit
// of a result.
__device__ __forceinline__ void plan_experts(const int* __restrict__ ids, int pairs, int E, int slots, Slot* slot,
                                             int* list) {
  __shared__ int count[kMaxExperts], first[kMaxExperts], total[2][4];
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
    if (n[i] > 0) slot[rank++] = Slot{4 * tid + i, at, n[i], 0};
    at += n[i];
  }
  for (int i = used + tid; i < slots; i += 256) slot[i] = Slot{0, 0, 0, 0};
  __syncthreads();
  for (int p = tid; p < pairs; p += 256) {
    const int e = ids[p];
    if (e >= 0 && e < E) list[atomicAdd(&first[e], 1)] = p;
  }
}

struct PlanArgs {
  const int* ids;
  int pairs, E, slots;
  Slot* slot;
  int* list;
};

// Rows of `cpr` chunks of 32 values -> terms [row][3][32 cpr] and scales [row][cpr]; one lane a chunk. The
// 2 or 4 chunks of a Hadamard block of 64 or 128 sit in adjacent lanes (cpr % 4 == 0). With PLAN, the first
// workgroup sorts the pairs instead.
template <int B, bool PLAN>
__global__ __launch_bounds__(256) void split_rows(const void* __restrict__ V, int64_t ld, int rows, int cpr,
                                                  uint8_t* __restrict__ q, uint8_t* __restrict__ scales, PlanArgs P) {
  if (PLAN && blockIdx.x == 0) {
    plan_experts(P.ids, P.pairs, P.E, P.slots, P.slot, P.list);
    return;
  }
  const int c = (blockIdx.x - (PLAN ? 1 : 0)) * 256 + threadIdx.x;
  if (c >= rows * cpr) return;  // whole quads: rows * cpr % 4 == 0
  const int row = c / cpr, at = c - row * cpr;
  float v[32];
  if constexpr (!PLAN) {  // h, float32
    const v4f* p = reinterpret_cast<const v4f*>(reinterpret_cast<const float*>(V) + row * ld + at * 32);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const v4f w = p[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * i + j] = w[j];
    }
  } else {  // x, bf16
    const v4u* p = reinterpret_cast<const v4u*>(reinterpret_cast<const uint16_t*>(V) + row * ld + at * 32);
#pragma unroll
    for (int i = 0; i < 4; ++i) widen8(p[i], v + 8 * i);
  }
  const int64_t K = 32 * (int64_t)cpr;
  split_chunk<B>(v, q + row * kTerms * K + at * 32, K, scales + c);
}

struct ExpertArgs {
  const Slot* slot;
  const int* list;
  int k, D, I;
  const uint8_t *wq, *ws;  // the experts' matrices
  const uint8_t *xq, *xs;  // terms and scales of the rows
  float* out;
};

typedef v4u v4u_dword __attribute__((aligned(4)));

// The four E8M0 dwords (one per step of 128) of slice sl of a row of KS scale bytes; past the row's end the
// last dword again.
__device__ __forceinline__ v4u slice_scales(const uint8_t* row, int sl, int KS) {
  if (KS % 16 == 0) return *reinterpret_cast<const v4u_dword*>(row + 16 * sl);
  v4u s;
#pragma unroll
  for (int u = 0; u < 4; ++u) s[u] = *reinterpret_cast<const unsigned*>(row + min(16 * sl + 4 * u, KS - 4));
  return s;
}

// W's scale bytes of a wave's 64 rows in LDS, up to 128 of a row at a time, so that each line of them is read
// from memory once: read 16 bytes a slice, a third of them came from HBM again, W having pushed them out of the L2
// between slices. Rows of up to 128 bytes lie back to back in memory (32 or 64 of them) and are copied whole; of
// longer rows one 128-byte window is held, the last one ending with the row. Where a row is whole 16-byte
// chunks, chunk q of row r sits at slot (q + r) % chunks: rows 0 .. 7 read the same byte of different banks.
struct ScaleWindow {
  int KS, chunks;  // chunks 0: rows as they lie in memory
  __device__ __forceinline__ explicit ScaleWindow(int ks) : KS(ks), chunks(ks > kScaleRow ? 8 : ks % 16 ? 0 : ks / 16) {}
  __device__ __forceinline__ int start(int step) const { return KS > kScaleRow ? min(step / 32 * kScaleRow, KS - kScaleRow) : 0; }

  // Request the window that holds `step`: rows base .. + 31 and base + skip .. + 31.
  __device__ __forceinline__ void fetch(uint8_t* lds, const uint8_t* mat, unsigned rows, unsigned skip, int step) const {
    const int lane = threadIdx.x & 63;
    const __amdgpu_buffer_rsrc_t rs = buffer_rsrc(mat, rows * (unsigned)KS);
    auto row_at = [&](unsigned r) { return (r < 32 ? r : r - 32 + skip) * (unsigned)KS; };
    const int units = KS > kScaleRow ? kTiles * 16 * 8 : 4 * KS;  // of 16 bytes
    for (int u0 = 0; u0 < units; u0 += 64) {
      const unsigned u = u0 + lane;
      unsigned off;
      if (chunks == 0) {
        off = 16 * u + (u >= 2u * KS ? (skip - 32) * (unsigned)KS : 0u);
      } else {
        const unsigned r = u / chunks, slot = u - r * chunks, q = (slot + chunks * 64u - r) % chunks;
        off = row_at(r) + (unsigned)start(step) + 16 * q;
      }
      if (u >= (unsigned)units) off = 0xFFFFFFF0u;  // reads as zero
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(lds + u0 * 16), 16, off, 0, 0, 0);
    }
  }

  // Byte of row r, step and lane group g.
  __device__ __forceinline__ unsigned get(const uint8_t* lds, int r, int step, int g) const {
    const int at = 4 * step - start(step) + g;
    return chunks == 0 ? lds[r * KS + at] : lds[(r * chunks + ((at >> 4) + r) % chunks) * 16 + (at & 15)];
  }
};

// 16-byte chunk q of row r of a tile's half slice sits at slot q ^ swz(r): the 16 rows of a fragment read take
// every slot twice, once on even and once on odd rows.
__device__ __forceinline__ int swz(int r) { return (r ^ ((r >> 3) & 1)) & 7; }

// One wave: four tiles of 16 rows of an expert's matrix by up to 5 MF tokens, all of K. UP: the gate and up rows of
// features 32 tile .. + 31 of h (two tiles each), h[pair] = silu(gate) * up. Not UP: output features 64 tile .. + 63.
// W streams through the wave's own LDS ring by the LDS DMA in half slices of 256 elements, 8 rows x 128 bytes an
// instruction; the tokens' terms and every scale go to registers, the next ones requested while these are
// multiplied. Four tiles share what is read of the tokens (with two, reading it from L2 took a third more time).
// No barrier: waves share nothing.
template <bool UP, int MF>
__device__ __forceinline__ void expert_tile(uint8_t* lds, const ExpertArgs& A, int expert, int tile, const int* list, int n) {
  const int K = UP ? A.D : A.I;
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const unsigned KB = (unsigned)K / 2, KS = (unsigned)K / 32;
  const int steps = K / 128, nsl = (steps + 3) / 4, nhalf = (steps + 1) / 2;
  const size_t base = (size_t)expert * (UP ? 2 * A.I : A.D) + (UP ? 32 : 64) * (size_t)tile;
  auto row0 = [&](int t) { return base + (UP ? (t >> 1) * A.I + 16 * (t & 1) : 16 * t); };
  auto fetch = [&](int i) {
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      const __amdgpu_buffer_rsrc_t rw = buffer_rsrc(A.wq + row0(t) * KB, 16u * KB);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int row = 8 * q + (lane >> 3);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)(lds + (i % kRing) * kHalfBytes + t * 2048 + q * 1024), 16,
                                                 (unsigned)row * KB + (unsigned)i * kHalf +
                                                     16u * (unsigned)((lane & 7) ^ swz(row)),
                                                 0, 0, 0);
      }
    }
  };
  constexpr int kFetch = 2 * kTiles;  // loads of a fetch
  const ScaleWindow win((int)KS);
  uint8_t* wscl = lds + kRing * kHalfBytes;
  auto fetch_scales = [&](int step) {
    win.fetch(wscl, A.ws + base * KS, UP ? A.I + 32u : 64u, UP ? (unsigned)A.I : 32u, step);
  };
  fetch(0);
  fetch_scales(0);
  const int term = r % kTerms;  // column 15 repeats a term of the next token and is not read
  const uint8_t *xp[MF], *xsp[MF];
#pragma unroll
  for (int f = 0; f < MF; ++f) {
    const int pair = list[min(kTokens * f + r / kTerms, n - 1)], row = UP ? pair / A.k : pair;
    xp[f] = A.xq + ((size_t)row * kTerms + term) * K + 16 * g;
    xsp[f] = A.xs + (size_t)row * KS;
  }
  v4u x[MF][2][2], xs[MF];
  auto load_step = [&](int step, int u) {
    step = min(step, steps - 1);
#pragma unroll
    for (int f = 0; f < MF; ++f) {
      // E4M3 operand: a lane group's 32 bytes are elements 16 g .. and 64 + 16 g .. of the step's 128
      // (measured); block b of 32 elements is scaled by the byte of lane group b for either operand
      x[f][u][0] = *reinterpret_cast<const v4u*>(xp[f] + (size_t)step * 128);
      x[f][u][1] = *reinterpret_cast<const v4u*>(xp[f] + (size_t)step * 128 + 64);
    }
  };
  auto load_scales = [&](int sl) {
#pragma unroll
    for (int f = 0; f < MF; ++f) xs[f] = slice_scales(xsp[f], sl, KS);
  };
  load_scales(0);
#pragma unroll
  for (int u = 0; u < 2; ++u) load_step(u, u);
  if (nhalf > 1) fetch(1);
  v4f acc[kTiles][MF];
#pragma unroll
  for (int t = 0; t < kTiles; ++t)
#pragma unroll
    for (int f = 0; f < MF; ++f) acc[t][f] = v4f{0.f, 0.f, 0.f, 0.f};
  for (int sl = 0; sl < nsl; ++sl) {
    unsigned wb[kTiles][4], xb[MF][4];  // this slice's scale bytes of the lane's group, one per step
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = 2 * sl + h;
      if (i >= nhalf) break;  // uniform
      // the half slice has landed, and everything requested after it but the next one's loads
      if (i + 1 < nhalf) __builtin_amdgcn_s_waitcnt(0x0F70 | kFetch);
      else __builtin_amdgcn_s_waitcnt(0x0F70);
      asm volatile("" ::: "memory");
      if (h == 0) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
#pragma unroll
          for (int t = 0; t < kTiles; ++t) wb[t][u] = win.get(wscl, 16 * t + r, min(4 * sl + u, steps - 1), g);
#pragma unroll
          for (int f = 0; f < MF; ++f) xb[f][u] = ((xs[f][u] >> (8 * g)) & 0xFFu) - 4u * (unsigned)term;
        }
      }
      const uint8_t* wa = lds + (i % kRing) * kHalfBytes + r * kHalf;
      v4u a[2][kTiles];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
          a[u][t] = *reinterpret_cast<const v4u*>(wa + t * 2048 + 16 * ((4 * u + g) ^ swz(r)));
      if (h == 0 && sl % 8 == 7 && sl + 1 < nsl) {  // the last slice of a window: its bytes are in registers
        __builtin_amdgcn_s_waitcnt(0xC07F);
        asm volatile("" ::: "memory");
        fetch_scales(4 * sl + 4);
      }
      if (h == 1 && sl + 1 < nsl) load_scales(sl + 1);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (2 * i + u < steps) {  // uniform
#pragma unroll
          for (int f = 0; f < MF; ++f) {
            const v8i B = {(int)x[f][u][0][0], (int)x[f][u][0][1], (int)x[f][u][0][2], (int)x[f][u][0][3],
                           (int)x[f][u][1][0], (int)x[f][u][1][1], (int)x[f][u][1][2], (int)x[f][u][1][3]};
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
              const v8i W = {(int)a[u][t][0], (int)a[u][t][1], (int)a[u][t][2], (int)a[u][t][3], 0, 0, 0, 0};
              acc[t][f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(W, B, acc[t][f], 4, 0, 0, (int)wb[t][2 * h + u], 0,
                                                                           (int)xb[f][2 * h + u]);
            }
          }
        }
        if (i + 1 < nhalf) load_step(2 * i + 2 + u, u);
      }
      __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the half slice has been read before its slot is refilled
      asm volatile("" ::: "memory");
      if (i + kRing < nhalf) fetch(i + kRing);
    }
  }
  // The three terms of token j are columns 3 j .. 3 j + 2 of a DPP row; lane (3 j, g) ends with features 4 g .. + 3.
#pragma unroll
  for (int f = 0; f < MF; ++f) {
    v4f y[kTiles];
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float v = acc[t][f][i];
        const int b = __float_as_int(v);
        y[t][i] = (v + __int_as_float(__builtin_amdgcn_update_dpp(0, b, 0x101, 0xF, 0xF, false))) +  // row_shl:1
                  __int_as_float(__builtin_amdgcn_update_dpp(0, b, 0x102, 0xF, 0xF, false));         // row_shl:2
      }
    const int j = kTokens * f + r / kTerms;
    if (term != 0 || r == 15 || j >= n) continue;
    const size_t pair = list[j];
    if constexpr (UP) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        v4f h;
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = y[t][i] / (1.0f + expf(-y[t][i])) * y[t + 2][i];
        *reinterpret_cast<v4f*>(A.out + pair * A.I + 32 * tile + 16 * t + 4 * g) = h;
      }
    } else {
#pragma unroll
      for (int t = 0; t < kTiles; ++t) *reinterpret_cast<v4f*>(A.out + pair * A.D + 64 * tile + 16 * t + 4 * g) = y[t];
    }
  }
}

template <bool UP>
__global__ __launch_bounds__(64) void expert_gemm(ExpertArgs A, int tiles) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kExpertLds];
  const Slot s = A.slot[blockIdx.x / tiles];
  const int tile = blockIdx.x % tiles;
  for (int j = 0; j < s.n; j += kTokens * kMaxFrags) {
    const int m = min(s.n - j, kTokens * kMaxFrags);
    if (m <= kTokens) expert_tile<UP, 1>(lds, A, s.expert, tile, A.list + s.first + j, m);
    else expert_tile<UP, 2>(lds, A, s.expert, tile, A.list + s.first + j, m);
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

template <bool PLAN>
hipError_t launch_split(int block, const void* V, int64_t ld, int rows, int K, uint8_t* q, uint8_t* s, const PlanArgs& P,
                        hipStream_t st) {
  const int cpr = K / 32;
  const dim3 grid((unsigned)(((int64_t)rows * cpr + 255) / 256 + (PLAN ? 1 : 0)));
  switch (block) {
    case 16: hipLaunchKernelGGL((split_rows<16, PLAN>), grid, dim3(256), 0, st, V, ld, rows, cpr, q, s, P); break;
    case 32: hipLaunchKernelGGL((split_rows<32, PLAN>), grid, dim3(256), 0, st, V, ld, rows, cpr, q, s, P); break;
    case 64: hipLaunchKernelGGL((split_rows<64, PLAN>), grid, dim3(256), 0, st, V, ld, rows, cpr, q, s, P); break;
    default: hipLaunchKernelGGL((split_rows<128, PLAN>), grid, dim3(256), 0, st, V, ld, rows, cpr, q, s, P);
  }
  return hipGetLastError();
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
  Slot* slot = reinterpret_cast<Slot*>(ws + FP4_MOE_WS_PLAN(T, k, D, I));
  int* list = reinterpret_cast<int*>(slot + pairs);
  const PlanArgs plan{ids, pairs, (int)E, slots, slot, list};
  hipError_t e = launch_split<true>(block, X, ldx, (int)T, (int)D, xq, xs, plan, st);
  if (e != hipSuccess) return e;
  const ExpertArgs up{slot, list, k, (int)D, (int)I, W13q, W13s, xq, xs, h};
  hipLaunchKernelGGL(expert_gemm<true>, dim3((unsigned)(slots * (I / 32))), dim3(64), 0, st, up, (int)(I / 32));
  e = hipGetLastError();
  if (e == hipSuccess) e = launch_split<false>(block, h, I, pairs, (int)I, hq, hs, plan, st);
  if (e != hipSuccess) return e;
  const ExpertArgs down{slot, list, k, (int)D, (int)I, W2q, W2s, hq, hs, out};
  hipLaunchKernelGGL(expert_gemm<false>, dim3((unsigned)(slots * (D / 64))), dim3(64), 0, st, down, (int)(D / 64));
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(combine, dim3((unsigned)((T * (D / 4) + 255) / 256)), dim3(256), 0, st, ids, weights, out, (int)T, k,
                     (int)E, (int)D, Y);
  return hipGetLastError();
}
