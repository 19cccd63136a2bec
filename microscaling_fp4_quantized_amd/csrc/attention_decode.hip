// Attention of one new token of each sequence over a paged key-value cache.
//
//   o_h = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q_h k_j - m),  over the visible tokens j
//
// Bound by reading keys and values once. A workgroup takes a piece of a sequence for one key-value head and up to 16 of the query
// heads that share it; its waves take tiles of 32 tokens in turn, each with a running maximum, sum and output of its own, and
// meet once at the end. Where a token's heads lie side by side in short rows, the waves take two or four heads instead: rows of 128
// bytes, read by workgroups that are not in step, cost memory a quarter of its rate (64 sequences, 8 bits: 64.6 -> 57 us). The tiles of
// all sequences, one after the other, are dealt out evenly: a workgroup has the same number of them whatever the lengths, and goes on
// with the next sequence where one ends. Pieces of a sequence meet in a second launch (join). Where the table or the window keep sequences
// short, a workgroup has one whole, and there is no second launch.
//
// Measured, with the join: 1000 tokens of 8 key-value heads 9.3 us, 5.6 of them here and 3.4 in the join, which together are near what two
// launches take; 131000 tokens 91 us (537 MB at 5.9 TB/s, as fast as memory is copied); 64 sequences in 8 bits 60 us (235 MB at 4.3 TB/s
// here).
//
// Both products run on the matrix cores with the tokens as rows and the heads as columns, so nothing has to change lanes:
//   S^T = K Q^T: a lane's K rows are 16-byte loads from the cache. Row r of half a of a tile is token 8 (r / 4) + 4 a + r % 4: the two
//   results then hold, in lane group q, the scores of tokens 8 q .. 8 q + 7 of one head.
//   O^T = V^T P^T: just those are the lane's part of P^T. Of V a lane loads the same dims of its 8 tokens, and a byte permute of each
//   pair of tokens turns them into rows of V^T, row r being dim 8 r + n of product n: no trip through LDS.
// The waves of a SIMD hide each other's loads; one tile ahead in registers was slower (one token 10.8 against 9.7 us, 131000 tokens 105
// against 102), as half the waves. Values stream past the caches (131000 tokens 101 -> 92 us); keys do not, because two loads
// share a line of theirs (8-bit codes 66 -> 70 us).
//
// 8-bit caches: codes are exact in bf16, so the matrix cores see codes and the scales are applied in float32, a key's to its score
// and a value's to its p. p is rounded to bf16 for the second product (at most 2^-8 of each p, and as often up as down); its sum is not.
#include "attention_device.hpp"

namespace fp4 {
namespace {

constexpr int kTile = kDecodeTile;
constexpr float kSlack = 8.f;  // the running maximum may lag behind by this many powers of two: p stays below 2^8

// The visible tokens of a sequence, as granules of 16: ga of them from token 0 on, then more from granule gb on.
struct Span {
  int n, lo, sinks, ga, gb, granules;
  __device__ int first_of(int g) const { return (g < ga ? g : g - ga + gb) * kGranule; }
  __device__ int tiles() const { return max(1, (granules + 1) / 2); }  // one of nothing for a sequence without tokens
};
__device__ __forceinline__ Span span_of(const Paged& c, int len, int window, int sinks) {
  Span s;
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
__device__ __forceinline__ int tiles_of(const Paged& c, int b, int window, int sinks) {
  return b < c.batch ? span_of(c, length_of(c, b), window, sinks).tiles() : 0;
}

// The tiles of all sequences dealt out to `count` of at most `most` workgroups, about `least` for each if there are few: the first
// `longer` have one more than `each`.
struct Deal {
  int total, count, each, longer;
  __device__ Deal(const Paged& c, int window, int sinks, int most, int least) {
    total = 0;
    for (int b = 0; b < c.batch; b += 64) total += wave_total(tiles_of(c, b + (threadIdx.x & 63), window, sinks));
    count = min(most, (total + least - 1) / least);
    each = total / count;
    longer = total - each * count;
  }
  __device__ int first_of(int w) const { return w * each + min(w, longer); }
  __device__ int who(int tile) const {
    const int with = longer * (each + 1);
    return tile < with ? tile / (each + 1) : longer + (tile - with) / each;
  }
};

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
      x.v[i][p] = __builtin_nontemporal_load(reinterpret_cast<const typename R::VWord*>(v + i * c.token_stride + p * (64 * R::VW)));
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

template <int D, bool E4M3, int BESIDE>
__global__ __launch_bounds__(64 * decode_waves(BESIDE), 2) void decode(Fp4AttentionArgs a, int group, int together, int most, int slots) {
  typedef Raw<D, E4M3> R;
  constexpr int PITCH = D + 1, WAVES = decode_waves(BESIDE);
  __shared__ alignas(16) float outs[WAVES][16][PITCH];
  __shared__ float tops[WAVES][16], sums[WAVES][16];
  const Paged& c = a.cache;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // workgroup i runs on XCD i % 8: the heads of the same tokens go to one XCD, where heads that share keys share its L2 (64 query
  // heads over one key-value head 31 -> 24 us)
  const int turn = blockIdx.x >> 3, w = turn / together * 8 + (blockIdx.x & 7), first = turn % together * BESIDE;
  constexpr int WAYS = WAVES / BESIDE;
  const int way = wave % WAYS, head = first + wave / WAYS, g0 = 16 * blockIdx.y, heads = min(16, group - g0);
  int at, stop;                              // the next tile, of all sequences', and where the workgroup's end
  int b = 0, begin = 0, tiles = 0, len = 0;  // its sequence, that one's first tile, number of tiles and tokens
  if (most == 0) {  // a sequence each
    if (w >= c.batch) return;
    b = w;
    len = length_of(c, b);
    tiles = span_of(c, len, a.window, a.sinks).tiles();
    at = 0;
    stop = tiles;
  } else {
    const Deal deal(c, a.window, a.sinks, most, WAYS);
    if (w >= deal.count) return;
    at = deal.first_of(w);
    stop = deal.first_of(w + 1);
    for (; b < c.batch; b += 64) {
      const int own = b + lane < c.batch ? length_of(c, b + lane) : 0;
      const int mine = b + lane < c.batch ? span_of(c, own, a.window, a.sinks).tiles() : 0, upto = wave_prefix(mine);
      const uint64_t after = __ballot(begin + upto > at);
      if (after) {
        const int i = __builtin_ctzll(after);
        b += i;
        tiles = __builtin_amdgcn_readlane(mine, i);
        len = __builtin_amdgcn_readlane(own, i);
        begin += __builtin_amdgcn_readlane(upto, i) - tiles;
        break;
      }
      begin += __builtin_amdgcn_readlane(upto, 63);
    }
  }
  const float factor = a.scale * kLog2e;
  float* scales = &outs[wave][0][0];  // free until the waves meet

  while (true) {
    const Span span = span_of(c, len, a.window, a.sinks);
    const int* row = c.table + b * c.table_stride;
    const int end = min(stop - begin, tiles);
    int tile = at - begin + way;
    State<D, E4M3> st;
    Raw<D, E4M3> x;
    Ids id = ids_of(c, row, span, tile, lane);
    {
      const int now = here(lane), r = now & 15, q = now >> 4;
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
    if (tile < end) {
      while (true) {
        load<D, E4M3>(x, c, head, span, id, lane);
        id = ids_of(c, row, span, tile + WAYS, lane);
        work<D, E4M3>(st, x, factor, scales, lane);
        tile += WAYS;
        if (tile >= end) break;
      }
    }
    const int now = here(lane), r = now & 15, q = now >> 4;
    st.l = sum_across<32>(sum_across<16>(st.l));
    if (q == 0) tops[wave][r] = st.m;
    __syncthreads();
    float top = st.m;
#pragma unroll
    for (int k = 1; k < WAYS; ++k) top = fmaxf(top, tops[wave ^ k][r]);
    const float keep = share_of(v2f{st.m, st.l}, top);
    if (r < heads) {
#pragma unroll
      for (int n = 0; n < D / 16; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) outs[wave][r][(n / R::VDIM) * (16 * R::VDIM) + (4 * q + i) * R::VDIM + n % R::VDIM] = st.o[n][i] * keep;
    }
    if (q == 0) sums[wave][r] = st.l * keep;
    __syncthreads();
    const bool whole = at == begin && end == tiles;
#pragma unroll
    for (int from = 0; from < WAVES; from += WAYS) {  // the first waves of the heads
      for (int e = threadIdx.x * 4; e < heads * D; e += 64 * WAVES * 4) {
        const int h = e / D, d = e % D;
        float l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = from; k < from + WAYS; ++k) {
          l += sums[k][h];
#pragma unroll
          for (int x = 0; x < 4; ++x) o[x] += outs[k][h][d + x];
        }
        const int hq = (first + from / WAYS) * group + g0 + h;
        if (whole) {
          const float inv = l == 0.f ? 0.f : 1.f / l;
          *reinterpret_cast<v2u*>(a.out + ((int64_t)b * a.q_heads + hq) * D + d) =
              v2u{bf16_pair(o[0] * inv, o[1] * inv), bf16_pair(o[2] * inv, o[3] * inv)};
        } else {
          // piece (w, b) has place w + b: along the tiles either w or b grows from one piece to the next, or both
          const Parts parts = parts_of(a.workspace, (size_t)slots * a.q_heads, D);
          *reinterpret_cast<v4f*>(parts.o + ((size_t)(w + b) * a.q_heads + hq) * D + d) = v4f{o[0], o[1], o[2], o[3]};
          if (d == 0) {
            float m = tops[from][h];
#pragma unroll
            for (int k = from + 1; k < from + WAYS; ++k) m = fmaxf(m, tops[k][h]);
            parts.ml[(size_t)(w + b) * a.q_heads + hq] = v2f{m, l};
          }
        }
      }
    }
    at = begin + end;
    if (at >= stop) return;
    begin = at;
    ++b;
    len = min(max(uniform_load(c.lengths + b), 0), 1 << 30);
    tiles = span_of(c, len, a.window, a.sinks).tiles();
    __syncthreads();  // outs and tops are read
  }
}

// o = sum_c 2^(m_c - m) o_c / sum_c 2^(m_c - m) l_c over the pieces of a sequence. D / 4 lanes hold an output; a workgroup has
// `wide` query heads of a sequence, its other lanes go over the pieces in turn with them.
template <int D>
__global__ __launch_bounds__(256) void join(Fp4AttentionArgs a, int wide, int most, int least, int slots) {
  constexpr int LANES = D / 4;
  const Paged& c = a.cache;
  const int lane = threadIdx.x & 63, b = blockIdx.y;
  const Deal deal(c, a.window, a.sinks, most, least);
  int begin = 0;
  for (int i = 0; i < b; i += 64) begin += wave_total(i + lane < b ? tiles_of(c, i + lane, a.window, a.sinks) : 0);
  const int first = deal.who(begin), last = deal.who(begin + tiles_of(c, b, a.window, a.sinks) - 1);
  if (first == last) return;  // written by its only workgroup
  const int hq = blockIdx.x * wide + threadIdx.x / LANES % wide, h = min(hq, a.q_heads - 1);
  const Parts parts = parts_of(a.workspace, (size_t)slots * a.q_heads, D);
  v2f ml;
  v4f o;
  if (join_all<D>(parts, wide, first, last, [&](int w) { return (size_t)(w + b) * a.q_heads + h; }, ml, o) && hq < a.q_heads) {
    const float inv = ml[1] == 0.f ? 0.f : 1.f / ml[1];
    *reinterpret_cast<v2u*>(a.out + ((int64_t)b * a.q_heads + hq) * D + 4 * (threadIdx.x % LANES)) =
        v2u{bf16_pair(o[0] * inv, o[1] * inv), bf16_pair(o[2] * inv, o[3] * inv)};
  }
}

template <int D, bool E4M3, int BESIDE>
hipError_t launch(const Fp4AttentionArgs& a, const DecodeWay& way, hipStream_t st) {
  const Paged& c = a.cache;
  const int group = a.q_heads / c.heads, blocks = (group + 15) / 16, together = c.heads / BESIDE;
  constexpr int WAVES = decode_waves(BESIDE), WAYS = WAVES / BESIDE;
  const int64_t count = way.whole ? c.batch : way.most;
  const int slots = (int)(way.most + c.batch);
  hipLaunchKernelGGL((decode<D, E4M3, BESIDE>), dim3((unsigned)((count + 7) / 8 * 8 * together), (unsigned)blocks), dim3(64 * WAVES), 0, st,
                     a, group, together, way.whole ? 0 : (int)way.most, slots);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || way.wide == 0) return e;
  hipLaunchKernelGGL((join<D>), dim3((unsigned)((a.q_heads + way.wide - 1) / way.wide), (unsigned)c.batch), dim3(256), 0, st, a, way.wide,
                     (int)way.most, WAYS, slots);
  return hipGetLastError();
}

template <int D, bool E4M3>
hipError_t launch(const Fp4AttentionArgs& a, hipStream_t st) {
  int dev = 0, cus = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e == hipSuccess) e = fp4_device_cus(dev, &cus);
  if (e != hipSuccess) return e;
  const DecodeWay way = decode_way(fp4_call_of(a, D, E4M3), cus);
  constexpr int bytes = D * (E4M3 ? 1 : 2);
  if constexpr (bytes <= 128)
    if (way.beside == 4) return launch<D, E4M3, 4>(a, way, st);
  if constexpr (bytes <= 256)
    if (way.beside == 2) return launch<D, E4M3, 2>(a, way, st);
  return launch<D, E4M3, 1>(a, way, st);
}

}  // namespace
}  // namespace fp4

hipError_t fp4_launch_attention_decode(const Fp4AttentionArgs& a, int dim, bool e4m3, hipStream_t st) {
  using namespace fp4;
  if (dim == 64) return e4m3 ? launch<64, true>(a, st) : launch<64, false>(a, st);
  if (dim == 128) return e4m3 ? launch<128, true>(a, st) : launch<128, false>(a, st);
  return e4m3 ? launch<256, true>(a, st) : launch<256, false>(a, st);
}
