// Attention of one new token of each sequence over a paged key-value cache.
//
//   o_h = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q_h k_j - m),  over the visible tokens j
//
// Bound by reading keys and values once. A workgroup takes a piece of a sequence for one key-value head and up to 16 of the query
// heads that share it; its four waves take tiles of 32 tokens in turn, each with a running maximum, sum and output of its own, and
// meet once at the end. Pieces of a longer sequence meet in a second launch (join).
//
// Both products run on the matrix cores with the tokens as rows and the heads as columns, so nothing has to change lanes:
//   S^T = K Q^T: a lane's K rows are 16-byte loads from the cache. Row r of half a of a tile is token 8 (r / 4) + 4 a + r % 4: the two
//   results then hold, in lane group q, the scores of tokens 8 q .. 8 q + 7 of one head.
//   O^T = V^T P^T: just those are the lane's part of P^T. Of V a lane loads the same dims of its 8 tokens, and a byte permute of each
//   pair of tokens turns them into rows of V^T, row r being dim 8 r + n of product n: no trip through LDS.
// The loads of the next tile and the page numbers of the one after it are in flight while a tile is worked on.
//
// 8-bit caches: codes are exact in bf16, so the matrix cores see codes and the scales are applied in float32, a key's to its score
// and a value's to its p. p is rounded to bf16 for the second product (2^-9 of each p, which averages out); its sum is not.
#include "../../include/fp4.h"
#include "attention_device.hpp"

namespace fp4 {
namespace {

constexpr int kWaves = 4;
constexpr int kTile = 32;
constexpr int kMinTiles = 4;   // of a piece: one for each wave
constexpr float kSlack = 8.f;  // the running maximum may lag behind by this many powers of two: p stays below 2^8

// The visible tokens of a sequence, as granules of 16: ga of them from token 0 on, then more from granule gb on.
struct Span {
  int n, lo, sinks, ga, gb, granules;
  __device__ int first_of(int g) const { return (g < ga ? g : g - ga + gb) * kGranule; }
  __device__ int tiles() const { return (granules + 1) / 2; }
};
__device__ __forceinline__ Span span_of(const Paged& c, int b, int window, int sinks) {
  Span s;
  const int len = length_of(c, b);
  s.n = min(len, paged_room(c));
  s.lo = window ? max(len - window, 0) : 0;
  s.sinks = sinks;
  const int end = (s.n + kGranule - 1) / kGranule;
  s.ga = (min(sinks, s.n) + kGranule - 1) / kGranule;
  s.gb = s.lo / kGranule;
  if (s.gb <= s.ga) s.ga = s.gb = end;
  s.granules = s.ga + max(end - s.gb, 0);
  return s;
}

// Pieces: `room` of them for all sequences together and one more for each sequence at most.
struct Piece {
  int b, index, count, slot, tiles;  // tiles of a piece
};
__device__ __forceinline__ Piece piece_of(const Paged& c, int window, int sinks, int room, int slot) {
  const int lane = threadIdx.x & 63;
  float total = 0.f;
  for (int b = 0; b < c.batch; b += 64) {
    float v = b + lane < c.batch ? (float)span_of(c, b + lane, window, sinks).tiles() : 0.f;
#pragma unroll
    for (int h = 1; h < 64; h <<= 1) v += __shfl_xor(v, h);
    total += v;
  }
  // at least total / room, whatever the float sum lost: so no more than room + batch pieces
  const int per = max(kMinTiles, (int)fminf(total / (float)room * 1.0001f + 1.f, 1e9f));
  Piece p{-1, 0, 0, 0, per};
  int base = 0;
  for (int b = 0; b < c.batch; b += 64) {
    const int mine = b + lane < c.batch ? max(1, (span_of(c, b + lane, window, sinks).tiles() + per - 1) / per) : 0;
    const int upto = wave_prefix(mine);
    const uint64_t after = __ballot(base + upto > slot);
    if (after) {
      const int at = __builtin_ctzll(after);
      p.b = b + at;
      p.count = __shfl(mine, at);
      p.slot = base + __shfl(upto, at) - p.count;
      p.index = slot - p.slot;
      break;
    }
    base += __shfl(upto, 63);
  }
  p.b = __builtin_amdgcn_readfirstlane(p.b);
  p.count = __builtin_amdgcn_readfirstlane(p.count);
  p.slot = __builtin_amdgcn_readfirstlane(p.slot);
  p.index = __builtin_amdgcn_readfirstlane(p.index);
  return p;
}

// A tile's raw bytes and its visible tokens.
template <int D, bool E4M3>
struct Raw {
  static constexpr int KL = E4M3 ? D / 64 : D / 32;  // 16-byte loads of a K row's lane
  static constexpr int VP = D == 256 ? 2 : 1;        // parts of V's dims, 16 rows of VDIM each
  static constexpr int VDIM = D / 16 / VP;
  static constexpr int VW = E4M3 ? VDIM / 4 : VDIM / 2;  // words of a token and part
  typedef unsigned VWord __attribute__((ext_vector_type(VW)));
  v4u k[2][KL];
  VWord v[8][VP];
  float scale;
  unsigned seen;  // bit i: token 8 (lane / 16) + i
};

struct Ids {
  int jk, jv, pk, pv;  // first tokens and pages of the lane's granules for K and for V
};

__device__ __forceinline__ Ids ids_of(const Paged& c, const int* row, const Span& s, int tile, int lane) {
  Ids r;
  const int gk = 2 * tile + ((lane >> 3) & 1), gv = 2 * tile + (lane >> 5);
  r.jk = gk < s.granules ? s.first_of(gk) : 0x7FFFFFFF - kTile;
  r.jv = gv < s.granules ? s.first_of(gv) : 0x7FFFFFFF - kTile;
  r.pk = r.jk < s.n ? row[r.jk >> c.shift] : -1;  // n is within the table's room
  r.pv = r.jv < s.n ? row[r.jv >> c.shift] : -1;
  return r;
}

template <int D, bool E4M3>
__device__ __forceinline__ void load(Raw<D, E4M3>& x, const Paged& c, int head, const Span& s, const Ids& id, int lane) {
  typedef Raw<D, E4M3> R;
  const int r = lane & 15, q = lane >> 4, mask = (1 << c.shift) - 1;
  const bool okk = (unsigned)id.pk < (unsigned)c.pages, okv = (unsigned)id.pv < (unsigned)c.pages;
  const int at = (okk ? id.jk & mask : 0) + 8 * ((r >> 2) & 1) + (r & 3);
  const uint8_t* k = c.k + (okk ? id.pk : 0) * c.page_stride + head * c.head_stride + at * c.token_stride + 16 * q;
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int i = 0; i < R::KL; ++i) x.k[a][i] = *reinterpret_cast<const v4u*>(k + 4 * a * c.token_stride + 64 * i);
  const int64_t pv = okv ? id.pv : 0;
  const int in = okv ? id.jv & mask : 0, tv = in + 8 * (q & 1);
  const uint8_t* v = c.v + pv * c.page_stride + head * c.head_stride + tv * c.token_stride + 4 * R::VW * r;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int p = 0; p < R::VP; ++p)
      x.v[i][p] = *reinterpret_cast<const typename R::VWord*>(v + i * c.token_stride + p * (64 * R::VW));
  if constexpr (E4M3) {
    const float* sc = (q & 1) ? c.v_scales : c.k_scales;
    x.scale = sc[pv * c.spage_stride + head * c.shead_stride + (in + r) * c.stoken_stride];
  }
  const int j = id.jv + 8 * (q & 1);
  unsigned seen = 0;
  if (okv) {
    if (j + 8 <= s.n && (j >= s.lo || j + 8 <= s.sinks)) seen = 0xFF;
    else
#pragma unroll
      for (int i = 0; i < 8; ++i) seen |= (j + i < s.n && (j + i >= s.lo || j + i < s.sinks)) ? 1u << i : 0u;
  }
  x.seen = seen;
}

template <int D, bool E4M3>
struct State {
  v8bf q[D / 32];
  v4f o[D / 16];
  float m, l;
};

template <int D, bool E4M3>
__device__ __forceinline__ void work(State<D, E4M3>& st, Raw<D, E4M3>& x, float factor, float* scales, int lane) {
  typedef Raw<D, E4M3> R;
  const int q = lane >> 4;
  const bool whole = __all(x.seen == 0xFF);
  v4f s[2];
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    s[a] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < R::KL; ++i) {
      if constexpr (E4M3) {
        const v2u w0 = bf16_of_codes(x.k[a][i][0]), w1 = bf16_of_codes(x.k[a][i][1]), w2 = bf16_of_codes(x.k[a][i][2]),
                  w3 = bf16_of_codes(x.k[a][i][3]);
        s[a] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, v4u{w0[0], w0[1], w1[0], w1[1]}), st.q[2 * i], s[a], 0, 0, 0);
        s[a] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, v4u{w2[0], w2[1], w3[0], w3[1]}), st.q[2 * i + 1], s[a], 0, 0, 0);
      } else {
        s[a] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, x.k[a][i]), st.q[i], s[a], 0, 0, 0);
      }
    }
  }
  float z[8], vs[8];
  if constexpr (E4M3) {
    // 16 scales of keys, 16 of values, then those of the second granule -> keys 0..31, values 0..31
    scales[(q & 1) * 32 + (q >> 1) * 16 + (lane & 15)] = x.scale;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const v4f k0 = *reinterpret_cast<const v4f*>(scales + 8 * q), k1 = *reinterpret_cast<const v4f*>(scales + 8 * q + 4);
    const v4f v0 = *reinterpret_cast<const v4f*>(scales + 32 + 8 * q), v1 = *reinterpret_cast<const v4f*>(scales + 36 + 8 * q);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      z[i] = s[0][i] * (k0[i] * factor);
      z[i + 4] = s[1][i] * (k1[i] * factor);
      vs[i] = v0[i];
      vs[i + 4] = v1[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      z[i] = s[0][i] * factor;
      z[i + 4] = s[1][i] * factor;
    }
  }
  if (!whole) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool on = (x.seen >> i) & 1;
      z[i] = on ? z[i] : kNever;
      if (E4M3) vs[i] = on ? vs[i] : 0.f;
#pragma unroll
      for (int p = 0; p < R::VP; ++p)
#pragma unroll
        for (int w = 0; w < R::VW; ++w) x.v[i][p][w] = on ? x.v[i][p][w] : 0u;  // whatever lies there, NaN too
    }
  }
  float top = fmaxf(fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3])), fmaxf(fmaxf(z[4], z[5]), fmaxf(z[6], z[7])));
  top = max_across<32>(max_across<16>(top));
  if (__any(top > st.m + kSlack)) {
    const float m = fmaxf(st.m, top), keep = m == st.m ? 1.f : exp2_hw(st.m - m);
    st.m = m;
    st.l *= keep;
#pragma unroll
    for (int n = 0; n < D / 16; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) st.o[n][i] *= keep;
  }
  const float m = st.m == kNever ? 0.f : st.m;
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = exp2_hw(z[i] - m);
  st.l += ((z[0] + z[1]) + (z[2] + z[3])) + ((z[4] + z[5]) + (z[6] + z[7]));
  if constexpr (E4M3) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] *= vs[i];
  }
  const v8bf p = __builtin_bit_cast(v8bf, v4u{bf16_pair(z[0], z[1]), bf16_pair(z[2], z[3]), bf16_pair(z[4], z[5]), bf16_pair(z[6], z[7])});
#pragma unroll
  for (int part = 0; part < R::VP; ++part) {
    unsigned w[8][R::VDIM / 2];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int c = 0; c < R::VW; ++c) {
        if constexpr (E4M3) {
          const v2u u = bf16_of_codes(x.v[i][part][c]);
          w[i][2 * c] = u[0];
          w[i][2 * c + 1] = u[1];
        } else {
          w[i][c] = x.v[i][part][c];
        }
      }
#pragma unroll
    for (int c = 0; c < R::VDIM / 2; ++c) {
      const v4u even{low_halves(w[0][c], w[1][c]), low_halves(w[2][c], w[3][c]), low_halves(w[4][c], w[5][c]), low_halves(w[6][c], w[7][c])};
      const v4u odd{high_halves(w[0][c], w[1][c]), high_halves(w[2][c], w[3][c]), high_halves(w[4][c], w[5][c]), high_halves(w[6][c], w[7][c])};
      const int n = part * R::VDIM + 2 * c;
      st.o[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, even), p, st.o[n], 0, 0, 0);
      st.o[n + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, odd), p, st.o[n + 1], 0, 0, 0);
    }
  }
}

template <int D, bool E4M3>
__global__ __launch_bounds__(64 * kWaves, D == 256 ? 1 : 2) void decode(Fp4AttentionArgs a, int group, int blocks, int room, int slots) {
  typedef Raw<D, E4M3> R;
  constexpr int PITCH = D + 1;
  __shared__ alignas(16) float outs[kWaves][16][PITCH];
  __shared__ float tops[kWaves][16], sums[kWaves][16];
  const Paged& c = a.cache;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int slot = blockIdx.x / (c.heads * blocks), rest = blockIdx.x - slot * (c.heads * blocks);
  const int head = rest / blocks, g0 = 16 * (rest - head * blocks), heads = min(16, group - g0);
  const Piece piece = piece_of(c, a.window, a.sinks, room, slot);
  if (piece.b < 0) return;
  const int b = piece.b;
  const Span span = span_of(c, b, a.window, a.sinks);
  const int* row = c.table + b * c.table_stride;
  const int end = min((piece.index + 1) * piece.tiles, span.tiles());
  int tile = piece.index * piece.tiles + wave;

  State<D, E4M3> st;
  const int r = lane & 15, q = lane >> 4;
  Raw<D, E4M3> x0, x1;
  Ids id = ids_of(c, row, span, tile, lane);
  {
    const uint16_t* qp = a.q + b * a.q_token + (head * group + g0 + min(r, heads - 1)) * a.q_head;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      // the dims of K's operand i: 32 i + 8 q, or of codes 64 (i / 2) + 16 q + 8 (i % 2)
      const int d = E4M3 ? 64 * (i / 2) + 16 * q + 8 * (i & 1) : 32 * i + 8 * q;
      st.q[i] = __builtin_bit_cast(v8bf, *reinterpret_cast<const v4u*>(qp + d));
    }
  }
#pragma unroll
  for (int n = 0; n < D / 16; ++n) st.o[n] = v4f{0.f, 0.f, 0.f, 0.f};
  st.m = kNever;
  st.l = 0.f;
  const float factor = a.scale * kLog2e;
  float* scales = &outs[wave][0][0];  // free until the waves meet
  if (tile < end) {
    load<D, E4M3>(x0, c, head, span, id, lane);
    id = ids_of(c, row, span, tile + kWaves, lane);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) arrived(st.q[i]);
    while (true) {
      if (tile + kWaves < end) load<D, E4M3>(x1, c, head, span, id, lane);
      id = ids_of(c, row, span, tile + 2 * kWaves, lane);
      work<D, E4M3>(st, x0, factor, scales, lane);
      tile += kWaves;
      if (tile >= end) break;
      if (tile + kWaves < end) load<D, E4M3>(x0, c, head, span, id, lane);
      id = ids_of(c, row, span, tile + 2 * kWaves, lane);
      work<D, E4M3>(st, x1, factor, scales, lane);
      tile += kWaves;
      if (tile >= end) break;
    }
  }
  st.l = sum_across<32>(sum_across<16>(st.l));
  if (q == 0) {
    tops[wave][r] = st.m;
    sums[wave][r] = st.l;
  }
  __syncthreads();
  const float top = fmaxf(fmaxf(tops[0][r], tops[1][r]), fmaxf(tops[2][r], tops[3][r]));
  const float keep = share_of(v2f{st.m, st.l}, top);
  if (r < heads) {
#pragma unroll
    for (int n = 0; n < D / 16; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) outs[wave][r][(n / R::VDIM) * (16 * R::VDIM) + (4 * q + i) * R::VDIM + n % R::VDIM] = st.o[n][i] * keep;
  }
  if (q == 0) sums[wave][r] = st.l * keep;
  __syncthreads();
  for (int e = threadIdx.x * 4; e < heads * D; e += 64 * kWaves * 4) {
    const int h = e / D, d = e % D;
    float l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      l += sums[w][h];
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] += outs[w][h][d + i];
    }
    const int hq = head * group + g0 + h;
    if (piece.count == 1) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      *reinterpret_cast<v2u*>(a.out + ((int64_t)b * a.q_heads + hq) * D + d) =
          v2u{bf16_pair(o[0] * inv, o[1] * inv), bf16_pair(o[2] * inv, o[3] * inv)};
    } else {
      const Parts parts = parts_of(a.workspace, (size_t)slots * a.q_heads, D);
      *reinterpret_cast<v4f*>(parts.o + ((size_t)slot * a.q_heads + hq) * D + d) = v4f{o[0], o[1], o[2], o[3]};
      if (d == 0) {
        float m = tops[0][h];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) m = fmaxf(m, tops[w][h]);
        parts.ml[(size_t)slot * a.q_heads + hq] = v2f{m, l};
      }
    }
  }
}

// o = sum_c 2^(m_c - m) o_c / sum_c 2^(m_c - m) l_c over the pieces of a sequence: a workgroup for a sequence and a query head.
template <int D>
__global__ __launch_bounds__(256) void join(Fp4AttentionArgs a, int room, int slots) {
  constexpr int LANES = D / 4, GROUPS = 256 / LANES;
  __shared__ v4f red[GROUPS][LANES];
  __shared__ float red_l[GROUPS];
  const int b = blockIdx.y, hq = blockIdx.x;
  // the first piece of sequence b: sum of the pieces of those before it
  const Paged& c = a.cache;
  const int lane = threadIdx.x & 63;
  float total = 0.f;
  for (int i = 0; i < c.batch; i += 64) {
    float v = i + lane < c.batch ? (float)span_of(c, i + lane, a.window, a.sinks).tiles() : 0.f;
#pragma unroll
    for (int h = 1; h < 64; h <<= 1) v += __shfl_xor(v, h);
    total += v;
  }
  const int per = max(kMinTiles, (int)fminf(total / (float)room * 1.0001f + 1.f, 1e9f));
  int before = 0;
  for (int i = 0; i < b; i += 64)
    before += wave_total(i + lane < b ? max(1, (span_of(c, i + lane, a.window, a.sinks).tiles() + per - 1) / per) : 0);
  const int count = max(1, (span_of(c, b, a.window, a.sinks).tiles() + per - 1) / per);
  if (count == 1) return;  // written by its only piece
  const Parts parts = parts_of(a.workspace, (size_t)slots * a.q_heads, D);
  const v2f* ml = parts.ml + (size_t)before * a.q_heads + hq;
  float m = kNever;
  for (int i = 0; i < count; i += 64)
    if (i + lane < count) m = fmaxf(m, ml[(size_t)(i + lane) * a.q_heads][0]);
#pragma unroll
  for (int h = 1; h < 64; h <<= 1) m = fmaxf(m, __shfl_xor(m, h));
  const float mm = m == kNever ? 0.f : m;
  const int g = threadIdx.x / LANES, e = threadIdx.x % LANES;
  v4f o{0.f, 0.f, 0.f, 0.f};
  float l = 0.f;
  for (int i = g; i < count; i += GROUPS) {
    const v2f x = ml[(size_t)i * a.q_heads];
    const float keep = share_of(x, mm);
    const v4f y = *reinterpret_cast<const v4f*>(parts.o + ((size_t)(before + i) * a.q_heads + hq) * D + 4 * e);
    l = __builtin_fmaf(x[1], keep, l);
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = __builtin_fmaf(y[k], keep, o[k]);
  }
  red[g][e] = o;
  if (e == 0) red_l[g] = l;
  __syncthreads();
  if (g == 0) {
#pragma unroll
    for (int i = 1; i < GROUPS; ++i) {
      l += red_l[i];
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] += red[i][e][k];
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    *reinterpret_cast<v2u*>(a.out + ((int64_t)b * a.q_heads + hq) * D + 4 * e) =
        v2u{bf16_pair(o[0] * inv, o[1] * inv), bf16_pair(o[2] * inv, o[3] * inv)};
  }
}

template <int D, bool E4M3>
hipError_t launch(const Fp4AttentionArgs& a, hipStream_t st) {
  const Paged& c = a.cache;
  const int group = a.q_heads / c.heads, blocks = (group + 15) / 16;
  const int room = FP4_ATTENTION_PIECES(a.q_heads, c.heads);
  // what the longest sequence that the table has room for can be cut into
  int64_t tokens = (int64_t)c.cols << c.shift;
  if (a.window && (int64_t)a.window + a.sinks + 2 * kTile < tokens) tokens = (int64_t)a.window + a.sinks + 2 * kTile;
  const int64_t most = ((tokens + kTile - 1) / kTile + 1 + kMinTiles - 1) / kMinTiles;
  const int slots = (int)(c.batch * most < room + c.batch ? c.batch * most : room + c.batch);
  hipLaunchKernelGGL((decode<D, E4M3>), dim3((unsigned)(slots * c.heads * blocks)), dim3(64 * kWaves), 0, st, a, group, blocks, room,
                     slots);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || most <= 1) return e;
  hipLaunchKernelGGL((join<D>), dim3((unsigned)a.q_heads, (unsigned)c.batch), dim3(256), 0, st, a, room, slots);
  return hipGetLastError();
}

}  // namespace
}  // namespace fp4

hipError_t fp4_launch_attention_decode(const Fp4AttentionArgs& a, int dim, bool e4m3, hipStream_t st) {
  using namespace fp4;
  if (dim == 64) return e4m3 ? launch<64, true>(a, st) : launch<64, false>(a, st);
  if (dim == 128) return e4m3 ? launch<128, true>(a, st) : launch<128, false>(a, st);
  return e4m3 ? launch<256, true>(a, st) : launch<256, false>(a, st);
}
