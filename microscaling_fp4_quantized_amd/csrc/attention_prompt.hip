// Attention of many new tokens of each sequence over a paged key-value cache: causal, with or without a window and first tokens
// that stay visible.
//
// Bound by the matrix cores (4 D operations for a row, a head and a visible token); heads of 64 have more vector instructions than products.
// A workgroup takes 256 or 128 rows of a sequence and a key-value head: the query heads that share the head are rows side by side, so that
// few tokens still fill a tile and the keys are read once for all of them. Its eight or four waves have 32 rows each and go over tiles of 64
// tokens that all of them read from LDS. With 32 rows a wave the reads keep LDS busy for about half the time that the products take.
//
//   S^T = K Q^T (32 x 32 x 16 products): a lane has the scores of one row, half of the tile's tokens, so maxima and sums need one
//   step across the wave. K's row r is token r with bits 2 and 3 exchanged: the scores of a lane are then 8 consecutive tokens of
//   each 16, which is its part of P^T in
//   O^T = V^T P^T: P goes on in registers. V is turned on its way into LDS, by byte permutes of 4 tokens x 8 dims of a thread.
// Rows of 16 more bytes (K) and of 9 chunks of 16 bytes (V^T) keep the 16-byte reads of 32 rows free of bank conflicts.
// The next tile's loads are in flight during a tile's products, in registers, and go into the other half of LDS behind them.
//
// Measured: 8192 tokens of 32 heads of 128 517 to 555 us on different machines, 0.99 to 1.06 PFLOP/s, where torch's large bf16 product
// reaches 1.22; the matrix cores are busy 50% of the CUs' cycles, vector instructions 43%. Three sequences of up to 9000 tokens of 64
// heads of 64 with a window of 1024 395 to 421 us, 0.7 PFLOP/s: vector instructions take 72% of the cycles (exponentials, 8 cycles each, as many
// as half of the products'), the matrix cores 39%. Not faster: the scores a tile ahead of the sums (609 us against 545; heads of 256 207 and 200), two groups of waves half a tile apart (566 and 526),
// leaving out the tiles that a wave's rows do not see but another's do (552 and 540).
//
// The running maximum may lag behind by 2^8 before sums and outputs are scaled again. p is rounded to bf16 for the second product;
// its sum, in float32, is of the rounded ones, so what rounding does to both cancels in part. 8-bit caches: codes are exact in bf16, the scales
// are applied in float32 to scores and p, and the sum is of p before its scale.
#include <atomic>

#include "attention_device.hpp"

namespace fp4 {
namespace {

constexpr int kTokens = kPromptTokens;
constexpr float kSlack = 8.f;

typedef float v16f __attribute__((ext_vector_type(16)));

template <int D, bool E4M3>
struct Lds {
  static constexpr int KP = D + 8, VP = kTokens + 8;  // elements of a row
  uint16_t k[2][kTokens][KP];
  uint16_t v[2][D][VP];
  float scales[2][2][kTokens];
  unsigned long long odd[4];  // tokens of a tile whose V has an infinity or NaN, where not all rows see all tokens
};

// A wave's part of a tile on its way: a granule's keys as 16-byte loads, or its values as 4 tokens x VDIM dims of a thread.
template <int D, bool E4M3>
struct Part {
  static constexpr int LANES = D * (E4M3 ? 1 : 2) / 16, KL = LANES / 4;  // threads of a key, loads of a granule
  static constexpr int VDIM = D == 64 ? 4 : 8, VU = D == 256 ? 2 : 1;    // dims of a unit of V, units of a thread
  static constexpr int VW = E4M3 ? VDIM / 4 : VDIM / 2;                  // words of a token and unit
  typedef unsigned VWord __attribute__((ext_vector_type(VW)));
  unsigned w[4 * KL];
  float scale;
  static_assert(4 * KL == VU * 4 * VW, "as many bytes of keys as of values");
};

// What a workgroup looks at: tiles of 64 tokens, ta of them from token 0 on, then more from tile tb on.
struct Range {
  int n, ta, tb, tiles;
  __device__ int first_of(int t) const { return (t < ta ? t : t - ta + tb) * kTokens; }
};

// A tile's pages, -1 for those that are none and past the end: one for each of its granules, the same for the whole workgroup.
struct Ids {
  int page[4];
};
__device__ __forceinline__ Ids ids_of(const Paged& c, const int* row, const Range& r, int tile) {
  Ids x;
  const int j = tile < r.tiles ? r.first_of(tile) : r.n;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const int at = j + g * kGranule;
    const int page = at < r.n ? uniform_load(row + (at >> c.shift)) : -1;
    x.page[g] = (unsigned)page < (unsigned)c.pages ? page : -1;
  }
  return x;
}
__device__ __forceinline__ int pick(const Ids& x, int g) {
  const int a = (g & 1) ? x.page[1] : x.page[0], b = (g & 1) ? x.page[3] : x.page[2];
  return (g & 2) ? b : a;
}

// A granule's place is the same for a wave (scalar registers), the offset within it stays the thread's. Heads of 64, which are short of
// registers, make their addresses where they use them (seven sequences of 1 to 150 tokens and heads of 128: 10.5 us, 10.85 so).
template <int D, bool E4M3>
struct Fetch {
  typedef Part<D, E4M3> P;
  unsigned k, v, token;

  __device__ __forceinline__ Fetch(const Paged& c, int lane) {
    token = (unsigned)c.token_stride;  // at most 2^26 bytes
    k = (lane / P::LANES) * token + 16 * (lane % P::LANES);
    v = 4 * (lane >> 4) * token + 4 * P::VW * (lane & 15);
  }
  static __device__ __forceinline__ int64_t place(const Paged& c, int head, int page, int j) {
    return max(page, 0) * c.page_stride + head * c.head_stride + (j & ((1 << c.shift) - 1)) * c.token_stride;
  }
  static __device__ __forceinline__ float scale(const Paged& c, const float* scales, int head, const Ids& id, int j, int lane) {
    const int ps = max(pick(id, lane >> 4), 0);
    return scales[ps * c.spage_stride + head * c.shead_stride + ((j + lane) & ((1 << c.shift) - 1)) * c.stoken_stride];
  }
  __device__ __forceinline__ void keys(P& x, const Paged& c, int head, const Ids& id, int j, int g, int lane) const {
    const uint8_t* at = c.k + place(c, head, pick(id, g), j + g * kGranule);
    const unsigned k = D == 64 ? here(this->k) : this->k;
#pragma unroll
    for (int i = 0; i < P::KL; ++i) {
      const v4u y = *reinterpret_cast<const v4u*>(at + (k + i * (64 / P::LANES) * token));
#pragma unroll
      for (int n = 0; n < 4; ++n) x.w[4 * i + n] = y[n];
    }
    if (E4M3 && g == 0) x.scale = scale(c, c.k_scales, head, id, j, lane);
  }
  __device__ __forceinline__ void values(P& x, const Paged& c, int head, const Ids& id, int j, int g, int lane) const {
    const uint8_t* at = c.v + place(c, head, pick(id, g), j + g * kGranule);
    const unsigned v = D == 64 ? here(this->v) : this->v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int u = 0; u < P::VU; ++u) {
        const typename P::VWord y = *reinterpret_cast<const typename P::VWord*>(at + (v + i * token) + u * (64 * P::VW));
#pragma unroll
        for (int n = 0; n < P::VW; ++n) x.w[(u * 4 + i) * P::VW + n] = y[n];
      }
    if (E4M3 && g == 0) x.scale = scale(c, c.v_scales, head, id, j, lane);
  }
};

// bf16 pairs with an exponent of all ones, in either half.
__device__ __forceinline__ bool odd_pair(unsigned w) { return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u; }

// Fetched keys into LDS, as rows of bf16.
template <int D, bool E4M3>
__device__ __forceinline__ void store_keys(Lds<D, E4M3>& lds, const Part<D, E4M3>& x, int tile, float factor, int g, int lane) {
  typedef Part<D, E4M3> P;
#pragma unroll
  for (int i = 0; i < P::KL; ++i) {
    uint16_t* to = &lds.k[tile & 1][g * kGranule + lane / P::LANES + i * (64 / P::LANES)][(E4M3 ? 16 : 8) * (lane % P::LANES)];
    const unsigned* w = x.w + 4 * i;
    if constexpr (E4M3) {
      const v2u a = bf16_of_codes(w[0]), b = bf16_of_codes(w[1]), e = bf16_of_codes(w[2]), f = bf16_of_codes(w[3]);
      *reinterpret_cast<v4u*>(to) = v4u{a[0], a[1], b[0], b[1]};
      *reinterpret_cast<v4u*>(to + 8) = v4u{e[0], e[1], f[0], f[1]};
    } else {
      *reinterpret_cast<v4u*>(to) = v4u{w[0], w[1], w[2], w[3]};
    }
  }
  if (E4M3 && g == 0) lds.scales[tile & 1][0][lane] = x.scale * factor;
}

// Fetched values into LDS, turned. With `some` (not all rows see all of the tile's tokens) values and scales from token n on,
// of pages that are none and those that are no numbers are 0, and the tokens of the last are noted.
template <int D, bool E4M3>
__device__ __forceinline__ void store_values(Lds<D, E4M3>& lds, const Part<D, E4M3>& x, int tile, const Ids& id, int j, int n, bool some,
                                             int g, int lane) {
  typedef Part<D, E4M3> P;
  const int t = g * kGranule + 4 * (lane >> 4);
  const bool held = pick(id, g) >= 0;
#pragma unroll
  for (int u = 0; u < P::VU; ++u) {
    unsigned w[4][P::VDIM / 2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < P::VW; ++k) {
        const unsigned raw = x.w[(u * 4 + i) * P::VW + k];
        if constexpr (E4M3) {
          const v2u p = bf16_of_codes(raw);
          w[i][2 * k] = p[0];
          w[i][2 * k + 1] = p[1];
        } else {
          w[i][k] = raw;
        }
      }
    auto turn = [&] {
#pragma unroll
      for (int k = 0; k < P::VDIM / 2; ++k) {
        const int row = u * 128 + 32 * k + (lane & 15);  // dim 128 u + VDIM (row % 16) + row / 16
        *reinterpret_cast<v2u*>(&lds.v[tile & 1][row][t]) = v2u{low_halves(w[0][k], w[1][k]), low_halves(w[2][k], w[3][k])};
        *reinterpret_cast<v2u*>(&lds.v[tile & 1][row + 16][t]) = v2u{high_halves(w[0][k], w[1][k]), high_halves(w[2][k], w[3][k])};
      }
    };
    if (!some) {
      turn();
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool on = held && j + t + i < n;
        bool bad = false;
#pragma unroll
        for (int k = 0; k < P::VDIM / 2; ++k) bad |= odd_pair(w[i][k]);
        if (on && bad) atomicOr(&lds.odd[tile & 3], 1ull << (t + i));
#pragma unroll
        for (int k = 0; k < P::VDIM / 2; ++k) w[i][k] = on && !bad ? w[i][k] : 0u;
      }
      turn();
    }
  }
  if (E4M3 && g == 0) {
    float scale = x.scale;
    if (some) {
      const bool on = j + lane < n && pick(id, lane >> 4) >= 0;
      const bool bad = !(fabsf(scale) < __builtin_inff());
      if (on && bad) atomicOr(&lds.odd[tile & 3], 1ull << lane);
      scale = on && !bad ? scale : 0.f;
    }
    lds.scales[tile & 1][1][lane] = scale;
  }
}

// What rows at places i0 to i1 look at.
__device__ __forceinline__ Range range_of(const Paged& c, int len, int i0, int i1, int window, int sinks) {
  Range r;
  r.n = min(min(len, paged_room(c)), i1 + 1);
  const int end = max((r.n + kTokens - 1) / kTokens, 0);
  r.ta = max((min(sinks, r.n) + kTokens - 1) / kTokens, 0);
  r.tb = (window ? max(i0 - window + 1, 0) : 0) / kTokens;
  if (r.tb <= r.ta) r.ta = r.tb = end;
  r.tiles = r.ta + max(end - r.tb, 0);
  return r;
}
// Rows of a sequence: new tokens times the heads of a group.
struct Rows {
  int first, count;  // its first row of q, and its new tokens
};
__device__ __forceinline__ Rows rows_of(const int* starts, int b, int T) {
  const int t0 = min(max(starts[b], 0), T), t1 = min(max(starts[b + 1], t0), T);
  return {t0, t1 - t0};
}

// SPLIT: blockIdx.y takes one of `splits` parts of its rows' tokens, at most. A kernel of its own, because what it adds to the registers
// costs heads of 64 4% (455 -> 468 us with a window).
template <int D, bool E4M3, int WAVES, bool SPLIT>
__global__ __launch_bounds__(64 * WAVES, D == 256 ? 1 : D == 128 ? 2 : WAVES == 8 ? 4 : 3) void prompt(Fp4AttentionArgs a, int group, int tiles, int splits) {
  extern __shared__ __align__(16) uint8_t memory[];
  typedef Lds<D, E4M3> L;
  constexpr int kRows = 32 * WAVES;
  // Left to itself the compiler reads an operand of the scores, waits for it and multiplies. Us so and with reads ahead: 8192 tokens 570 / 555,
  // over 8 bits 637 / 621, heads of 256 201 / 192 and 215 / 204; heads of 64 the same or worse.
  constexpr int kReads = D == 64 ? 0 : E4M3 ? 6 : 4;
  // Where the pages of the tile after next are looked up: ahead of the scores, whose first read then waits for them too, or behind. Us: heads
  // of 64 with a window 428 / 421, pieces over 8 bits 328 / 314; the others lose 1%.
  constexpr bool kLate = E4M3 ? SPLIT && D == 128 : D == 64;
  static_assert(sizeof(L) >= (size_t)kRows * (D + 8) * 2, "the rows of out pass through the same memory");
  L& lds = *reinterpret_cast<L*>(memory);
  const Paged& c = a.cache;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int slot = blockIdx.x / c.heads, head = blockIdx.x - slot * c.heads;
  // which rows: the last tiles first, they see the most
  int b = -1, tile = tiles - 1 - slot, len = 0;
  Rows rows{0, 0};
  for (int b0 = 0; b0 < c.batch; b0 += 64) {
    const bool is = b0 + lane < c.batch;
    const Rows own = is ? rows_of(a.starts, b0 + lane, a.T) : Rows{0, 0};
    const int tokens = is ? length_of(c, b0 + lane) : 0;
    const int mine = (own.count * group + kRows - 1) / kRows, upto = wave_prefix(mine);
    const uint64_t after = __ballot(upto > tile);
    if (after) {
      const int at = __builtin_ctzll(after);
      b = b0 + at;
      tile -= __builtin_amdgcn_readlane(upto, at) - __builtin_amdgcn_readlane(mine, at);
      rows = Rows{__builtin_amdgcn_readlane(own.first, at), __builtin_amdgcn_readlane(own.count, at)};
      len = __builtin_amdgcn_readlane(tokens, at);
      break;
    }
    tile -= __builtin_amdgcn_readlane(upto, 63);
  }
  if (b < 0) return;
  const int base = len - rows.count;                              // place of the first new token
  const int last = rows.count * group - 1;                        // its last row
  const int row = tile * kRows + wave * 32 + (lane & 31);
  const int mine = min(row, last), token = mine / group, place = base + token;
  const int* pages = c.table + b * c.table_stride;

  const Range range = range_of(c, len, base + tile * kRows / group, base + min(tile * kRows + kRows - 1, last) / group, a.window, a.sinks);
  const int parts = SPLIT ? max((int)min((int64_t)splits, worth(range.tiles, a.T, a.q_heads, D)), 1) : 1, part = SPLIT ? blockIdx.y : 0;
  if (part >= parts) return;
  const int from = SPLIT ? (int)((int64_t)range.tiles * part / parts) : 0;
  const int end = SPLIT ? (int)((int64_t)range.tiles * (part + 1) / parts) : range.tiles;
  const int half = lane >> 5;
  v8bf q[D / 16];
  {
    const uint16_t* qp = a.q + (int64_t)(rows.first + token) * a.q_token + (int64_t)(head * group + mine - token * group) * a.q_head;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) q[i] = __builtin_bit_cast(v8bf, *reinterpret_cast<const v4u*>(qp + 16 * i + 8 * half));
  }
  v16f o[D / 32];
#pragma unroll
  for (int m = 0; m < D / 32; ++m)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[m][i] = 0.f;
  float top = kNever, sum = 0.f;
  const float factor = a.scale * kLog2e, unit = E4M3 ? 1.f : factor;  // 8 bits: the factor is in the keys' scales
  // A tile of pages that are all there counts whole, for every row from `low` to `high`, if its first token is at most `upto` and, with a
  // window, at least `from` or one of so few that it ends with the first tokens.
  struct Whole {
    int upto, from, ends;
    __device__ Whole(const Range& r, int low, int high, int window, int sinks) {
      upto = min(r.n, low + 1) - kTokens;
      from = window ? high - window + 1 : 0;
      ends = sinks - kTokens;
    }
    __device__ bool operator()(bool held, int j) const { return held & (j <= upto) & ((j >= from) | (j <= ends)); }
  };
  const int r0 = tile * kRows, rw = r0 + wave * 32;
  const Whole for_all(range, base + r0 / group, base + min(r0 + kRows - 1, last) / group, a.window, a.sinks);
  const Whole for_wave(range, base + min(rw, last) / group, base + min(rw + 31, last) / group, a.window, a.sinks);
  auto held = [](const Ids& id) { return (id.page[0] | id.page[1] | id.page[2] | id.page[3]) >= 0; };

  // Of eight waves four bring the values and four the keys; four waves bring both.
  Part<D, E4M3> bring[WAVES == 8 ? 1 : 2];
  Part<D, E4M3>&vpart = bring[0], &kpart = bring[WAVES == 8 ? 0 : 1];
  const bool brings_v = WAVES == 4 || wave < 4, brings_k = WAVES == 4 || wave >= 4;
  const int g = wave & 3;
  const Fetch<D, E4M3> fetch(c, lane);
  Ids id = ids_of(c, pages, range, from), id1 = ids_of(c, pages, range, from + 1);
  if (tid < 4) lds.odd[tid] = 0;
  __syncthreads();
  if (from < end) {
    const int j = range.first_of(from);
    if (brings_v) {
      fetch.values(vpart, c, head, id, j, g, lane);
      store_values<D, E4M3>(lds, vpart, from, id, j, range.n, !for_all(held(id), j), g, lane);
    }
    if (brings_k) {
      fetch.keys(kpart, c, head, id, j, g, lane);
      store_keys<D, E4M3>(lds, kpart, from, factor, g, lane);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < D / 16; ++i) arrived(q[i]);
  for (int it = from; it < end; ++it) {
    const int j = range.first_of(it), j1 = range.first_of(it + 1);
    // past the last tile too, from page 0 then: a branch around loads makes every later use of their registers wait for them
    if (brings_v) fetch.values(vpart, c, head, id1, j1, g, lane);
    if (brings_k) fetch.keys(kpart, c, head, id1, j1, g, lane);
    Ids id2;
    if constexpr (!kLate) id2 = ids_of(c, pages, range, it + 2);
    if (tid == 0) lds.odd[(it + 2) & 3] = 0;  // read two tiles ago, next written behind the next barrier
    // scores as plain floats: changing elements of a matrix register under a branch was compiled wrongly (D = 256, one
    // element copied over all others, by the clang of ROCm 7.2)
    float s[2][16];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      v16f acc;
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[i] = 0.f;
      const int r = lane & 31, key = 32 * u + ((r & 0x13) | ((r & 4) << 1) | ((r & 8) >> 1));
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const v8bf k = __builtin_bit_cast(v8bf, *reinterpret_cast<const v4u*>(&lds.k[it & 1][key][16 * i + 8 * half]));
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k, q[i], acc, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[u][i] = acc[i];
        if (E4M3) s[u][i] *= lds.scales[it & 1][0][32 * u + 16 * (i / 8) + 8 * half + i % 8];
      }
    }
    if constexpr (kReads > 0) {  // that many of the keys' reads ahead of the products
      __builtin_amdgcn_sched_group_barrier(0x100, kReads, 0);
#pragma unroll
      for (int i = 0; i < D / 8 - kReads; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      }
      __builtin_amdgcn_sched_group_barrier(0x8, kReads, 0);
    }
    if constexpr (kLate) id2 = ids_of(c, pages, range, it + 2);
    unsigned hidden = 0;  // bit 8 n + k: the lane's token j + 8 half + 16 n + k, which its row does not see
    if (!for_wave(held(id), j)) {
      const int at = j + 8 * half, to = min(place, range.n - 1) - at;
      const int from = (a.window ? place - a.window : -1) - at, first = a.sinks - at;
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        auto below = [&](int t) { return (1u << min(max(t - 16 * n, 0), 8)) - 1; };  // of the 8, those before token t
        unsigned seen = below(to + 1) & (~below(from + 1) | below(first));
        if (id.page[n] < 0) seen = 0;
        hidden |= (~seen & 0xFFu) << (8 * n);
      }
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        unsigned off[4];  // all ones if hidden; as asm, because the compiler makes a compare and a select of each
        asm("v_bfe_i32 %0, %4, %5, 1\n\tv_bfe_i32 %1, %4, %6, 1\n\tv_bfe_i32 %2, %4, %7, 1\n\tv_bfe_i32 %3, %4, %8, 1"
            : "=&v"(off[0]), "=&v"(off[1]), "=&v"(off[2]), "=&v"(off[3])
            : "v"(hidden), "n"(i), "n"(i + 1), "n"(i + 2), "n"(i + 3));
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // off ? kNever : s
          float& x = s[i / 16][i % 16 + k];
          x = __uint_as_float(__builtin_amdgcn_bitop3_b32(off[k], __float_as_uint(kNever), __float_as_uint(x), 0xCA));
        }
      }
    }
    if (!for_all(held(id), j)) {
      if (const unsigned long long odd = lds.odd[it & 3]) {  // a row that sees such a token is none of numbers
        unsigned bits = 0;
#pragma unroll
        for (int n = 0; n < 4; ++n) bits |= ((unsigned)(odd >> (16 * n + 8 * half)) & 0xFFu) << (8 * n);
        if (bits & ~hidden) sum = __builtin_nanf("");
      }
    }
    float z = fmaxf(s[0][0], s[1][0]);
#pragma unroll
    for (int i = 1; i < 16; ++i) z = fmaxf(fmaxf(z, s[0][i]), s[1][i]);
    z = max_across<32>(z) * unit;
    if (__any(z > top + kSlack)) {
      const float m = fmaxf(top, z), keep = m == top ? 1.f : exp2_hw(top - m);
      top = m;
      sum *= keep;
#pragma unroll
      for (int m2 = 0; m2 < D / 32; ++m2) {
        // heads of 256 have their outputs in accumulation registers: held there up to here, or the compiler moves all of them to
        // others and back for every tile (230 -> 200 us at 4096 tokens)
        if constexpr (D == 256) asm volatile("" : "+a"(o[m2]));
        o[m2] *= keep;
        if constexpr (D == 256) asm volatile("" : "+a"(o[m2]));
      }
    }
    const float m = top == kNever ? 0.f : top;
    unsigned w[16];
    auto weigh = [&](int n) {  // p of scores 2 n and 2 n + 1
      float x[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int u = n / 8, i = 2 * (n % 8) + k;
        x[k] = exp2_hw(__builtin_fmaf(s[u][i], unit, -m));
        if constexpr (E4M3) {
          sum += x[k];
          x[k] *= lds.scales[it & 1][1][32 * u + 16 * (i / 8) + 8 * half + i % 8];
        }
      }
      w[n] = bf16_pair(x[0], x[1]);
      if (!E4M3) sum = add_pair(w[n], sum);
    };
    auto add = [&](int n, int m2) {  // 16 tokens' part of 32 dims
      const v8bf p = __builtin_bit_cast(v8bf, v4u{w[4 * n], w[4 * n + 1], w[4 * n + 2], w[4 * n + 3]});
      const v8bf v = __builtin_bit_cast(v8bf, *reinterpret_cast<const v4u*>(&lds.v[it & 1][32 * m2 + (lane & 31)][16 * n + 8 * half]));
      o[m2] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, p, o[m2], 0, 0, 0);
    };
    // ahead of the SIMD's other waves from here on: their loads and products fill in behind (547 -> 538 us at 8192 tokens)
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int k = 0; k < 16; ++k) weigh(k);
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int m2 = 0; m2 < D / 32; ++m2) add(n, m2);
    __builtin_amdgcn_s_setprio(0);
    if (brings_v) store_values<D, E4M3>(lds, vpart, it + 1, id1, j1, range.n, !for_all(held(id1), j1), g, lane);
    if (brings_k) store_keys<D, E4M3>(lds, kpart, it + 1, factor, g, lane);
    id = id1;
    id1 = id2;
    __syncthreads();
  }
  sum = sum_across<32>(sum);
  constexpr int VDIM = Part<D, E4M3>::VDIM;
  if (SPLIT && parts > 1) {
    // a lane has VDIM dims in a row of every eighth: (m2 / 4) 128 + VDIM r + {0 .. VDIM - 1}
    const int token = (D == 64 ? here(place) : place) - base, row = r0 + wave * 32 + ((D == 64 && E4M3 ? here(lane) : lane) & 31);
    if (row <= last) {
      const size_t n = (size_t)a.T * a.q_heads, at = part * n + (size_t)(rows.first + token) * a.q_heads + head * group + (row - token * group);
      const Parts to = parts_of(a.workspace, splits * n, D);
#pragma unroll
      for (int p = 0; p < D / 32; p += VDIM / 2)
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int k = 0; k < VDIM / 2; k += 2) {
            float* y = to.o + at * D + (p / 4) * 128 + VDIM * (8 * (i / 4) + 4 * half + i % 4) + 2 * k;
            *reinterpret_cast<v4f*>(y) = v4f{o[p + k][i], o[p + k][i + 8], o[p + k + 1][i], o[p + k + 1][i + 8]};
          }
      if (half == 0) to.ml[at] = v2f{top, sum};
    }
    return;
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  // rows of out through LDS: a wave's 32 rows, D + 8 elements apart
  uint16_t* mem = reinterpret_cast<uint16_t*>(memory) + wave * 32 * (D + 8);
#pragma unroll
  for (int m2 = 0; m2 < D / 32; ++m2)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 8 * (i / 4) + 4 * half + i % 4;
      const int dim = (m2 / 4) * 128 + VDIM * r + 2 * (m2 % 4);
      *reinterpret_cast<unsigned*>(mem + (lane & 31) * (D + 8) + dim) = bf16_pair(o[m2][i] * inv, o[m2][i + 8] * inv);
    }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    const int e = i * 64 + lane, r = e / (D / 8), d = e % (D / 8) * 8, at = tile * kRows + wave * 32 + r;
    if (at > last) break;
    const int t = at / group;
    *reinterpret_cast<v4u*>(a.out + ((int64_t)(rows.first + t) * a.q_heads + head * group + at - t * group) * D + d) =
        *reinterpret_cast<const v4u*>(mem + r * (D + 8) + d);
  }
}

// out = sum_p 2^(m_p - m) o_p / sum_p 2^(m_p - m) l_p over the parts of a row and head, where there is more than one. A workgroup has
// `wide` heads of a token.
template <int D>
__global__ __launch_bounds__(256) void join(Fp4AttentionArgs a, int group, int tile_rows, int splits, int wide) {
  constexpr int LANES = D / 4;
  const Paged& c = a.cache;
  const int t = blockIdx.x, hq = blockIdx.y * wide + threadIdx.x / LANES % wide, h = min(hq, a.q_heads - 1);
  const int b = __builtin_amdgcn_readfirstlane(sequence_of(a.starts, c.batch, t));
  if (b < 0) return;
  const Rows rows = rows_of(a.starts, b, a.T);
  const int len = length_of(c, b), base = len - rows.count, last = rows.count * group - 1;
  const int first = ((t - rows.first) * group + h % group) / tile_rows * tile_rows;
  const Range range = range_of(c, len, base + first / group, base + min(first + tile_rows - 1, last) / group, a.window, a.sinks);
  const int parts = max((int)min((int64_t)splits, worth(range.tiles, a.T, a.q_heads, D)), 1);
  const size_t n = (size_t)a.T * a.q_heads, at = (size_t)t * a.q_heads + h;
  v2f ml;
  v4f o;
  const bool has = join_all<D>(parts_of(a.workspace, splits * n, D), wide, 0, parts > 1 ? parts - 1 : -1, [&](int p) { return p * n + at; }, ml, o);
  if (!has || parts == 1 || hq >= a.q_heads) return;  // one part: written by it
  const float inv = ml[1] == 0.f ? 0.f : 1.f / ml[1];
  *reinterpret_cast<v2u*>(a.out + at * D + 4 * (threadIdx.x % LANES)) = v2u{bf16_pair(o[0] * inv, o[1] * inv), bf16_pair(o[2] * inv, o[3] * inv)};
}

template <int D, bool E4M3, int WAVES, bool SPLIT>
hipError_t launch(const Fp4AttentionArgs& a, const PromptWay& way, int dev, hipStream_t st) {
  const int group = a.q_heads / a.cache.heads, rows = 32 * WAVES, splits = SPLIT ? way.splits : 1;
  const int64_t tiles = ((int64_t)a.T * group + rows - 1) / rows + a.cache.batch;
  constexpr int bytes = sizeof(Lds<D, E4M3>);
  static std::atomic<int> ready[64];  // by device
  auto kern = prompt<D, E4M3, WAVES, SPLIT>;
  const bool cached = dev >= 0 && dev < 64;
  hipError_t e = hipSuccess;
  if (!cached || !ready[dev].load(std::memory_order_acquire)) {
    e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    if (cached) ready[dev].store(1, std::memory_order_release);
  }
  hipLaunchKernelGGL(kern, dim3((unsigned)(tiles * a.cache.heads), splits), dim3(64 * WAVES), bytes, st, a, group, (int)tiles, splits);
  e = hipGetLastError();
  if (e != hipSuccess || !SPLIT) return e;
  hipLaunchKernelGGL((join<D>), dim3((unsigned)a.T, (unsigned)((a.q_heads + way.wide - 1) / way.wide)), dim3(256), 0, st, a, group, rows, splits,
                     way.wide);
  return hipGetLastError();
}

template <int D, bool E4M3>
hipError_t launch(const Fp4AttentionArgs& a, hipStream_t st) {
  int dev = 0, cus = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e == hipSuccess) e = fp4_device_cus(dev, &cus);
  if (e != hipSuccess) return e;
  const PromptWay way = prompt_way(fp4_call_of(a, D, E4M3), cus);
  if constexpr (prompt_eight(D, E4M3, true))
    if (way.waves == 8 && way.splits > 1) return launch<D, E4M3, 8, true>(a, way, dev, st);
  if constexpr (prompt_eight(D, E4M3, false))
    if (way.waves == 8) return launch<D, E4M3, 8, false>(a, way, dev, st);
  return way.splits > 1 ? launch<D, E4M3, 4, true>(a, way, dev, st) : launch<D, E4M3, 4, false>(a, way, dev, st);
}

}  // namespace
}  // namespace fp4

hipError_t fp4_launch_attention_prompt(const Fp4AttentionArgs& a, int dim, bool e4m3, hipStream_t st) {
  using namespace fp4;
  if (dim == 64) return e4m3 ? launch<64, true>(a, st) : launch<64, false>(a, st);
  if (dim == 128) return e4m3 ? launch<128, true>(a, st) : launch<128, false>(a, st);
  return e4m3 ? launch<256, true>(a, st) : launch<256, false>(a, st);
}
