// Attention of many new tokens of each sequence over a paged key-value cache: causal, with or without a window and first tokens
// that stay visible.
//
// Bound by the matrix cores (4 D operations for a row, a head and a visible token). A workgroup takes 128 rows of a sequence and a
// key-value head: the query heads that share the head are rows side by side, so that few tokens still fill a tile and the keys
// are read once for all of them. Its four waves have 32 rows each and go over tiles of 64 tokens that all of them read from LDS.
//
//   S^T = K Q^T (32 x 32 x 16 products): a lane has the scores of one row, half of the tile's tokens, so maxima and sums need one
//   step across the wave. K's row r is token r with bits 2 and 3 exchanged: the scores of a lane are then 8 consecutive tokens of
//   each 16, which is its part of P^T in
//   O^T = V^T P^T: P goes on in registers. V is turned on its way into LDS, by byte permutes of 4 tokens x 8 dims of a thread.
// Rows of 16 more bytes (K) and of 9 chunks of 16 bytes (V^T) keep the 16-byte reads of 32 rows free of bank conflicts.
// The next tile's loads are in flight during a tile's products, in registers, and go into the other half of LDS behind them.
//
// The running maximum may lag behind by 2^8 before sums and outputs are scaled again. p is rounded to bf16 for the second product;
// its sum is not. 8-bit caches: codes are exact in bf16, the scales are applied in float32 to scores and p.
#include <atomic>

#include "attention_device.hpp"

namespace fp4 {
namespace {

constexpr int kWaves = 4;
constexpr int kRows = 128;   // of a workgroup
constexpr int kTokens = 64;  // of a tile
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

template <int D, bool E4M3>
struct Staged {
  static constexpr int KL = kTokens * D * (E4M3 ? 1 : 2) / (64 * kWaves * 16);  // 16-byte loads of K of a thread
  static constexpr int VDIM = D == 64 ? 4 : 8, VU = D == 256 ? 2 : 1;           // dims of a unit of V, units of a thread
  static constexpr int VW = E4M3 ? VDIM / 4 : VDIM / 2;
  typedef unsigned VWord __attribute__((ext_vector_type(VW)));
  v4u k[KL];
  VWord v[VU][4];
  float scale;
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

// A thread's loads of a tile: a granule's place is the same for a wave (scalar registers), the offset within it stays the thread's.
template <int D, bool E4M3>
struct Fetch {
  typedef Staged<D, E4M3> S;
  static constexpr int LANES = D * (E4M3 ? 1 : 2) / 16, STEP = 64 * kWaves / LANES;  // threads of a K row, rows of a pass
  unsigned k, v, token;

  __device__ __forceinline__ Fetch(const Paged& c, int tid) {
    token = (unsigned)c.token_stride;  // at most 2^26 bytes
    k = (tid / LANES % kGranule) * token + 16 * (tid % LANES);
    v = (4 * (tid >> 4) % kGranule) * token + 4 * S::VW * (tid & 15);
  }
  static __device__ __forceinline__ int64_t place(const Paged& c, int head, int page, int j) {
    return max(page, 0) * c.page_stride + head * c.head_stride + (j & ((1 << c.shift) - 1)) * c.token_stride;
  }
  __device__ __forceinline__ void operator()(S& x, const Paged& c, int head, const Ids& id, int j, int wave, int tid) const {
#pragma unroll
    for (int i = 0; i < S::KL; ++i) {
      const int t = wave * (64 / LANES) / kGranule * kGranule + i * STEP;  // the wave's rows are in this one's granule
      const int g = t / kGranule, more = STEP < kGranule ? i * STEP % kGranule : 0;
      const uint8_t* at = c.k + place(c, head, pick(id, g), j + g * kGranule);
      x.k[i] = *reinterpret_cast<const v4u*>(at + (k + more * token));
    }
    const uint8_t* at = c.v + place(c, head, pick(id, wave), j + wave * kGranule);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int u = 0; u < S::VU; ++u)
        x.v[u][i] = *reinterpret_cast<const typename S::VWord*>(at + (v + i * token) + u * (64 * S::VW));
    if constexpr (E4M3) {
      const int ts = tid & 63, ps = max(pick(id, ts >> 4), 0);
      if (tid < 128)
        x.scale = (tid < 64 ? c.k_scales : c.v_scales)[ps * c.spage_stride + head * c.shead_stride +
                                                       ((j + ts) & ((1 << c.shift) - 1)) * c.stoken_stride];
    }
  }
};

// bf16 pairs with an exponent of all ones, in either half.
__device__ __forceinline__ bool odd_pair(unsigned w) { return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u; }

// The fetched tile into LDS: K as rows of bf16, V turned. Tokens from `n` on and of pages that are none have values of 0. With
// `some` (not all rows see all tokens) values that are no numbers are 0 and their tokens noted.
template <int D, bool E4M3>
__device__ __forceinline__ void store(Lds<D, E4M3>& lds, const Staged<D, E4M3>& x, int buf, const Ids& id, int j, int n, float factor,
                                      bool some, unsigned long long* odd, int wave, int tid) {
  typedef Staged<D, E4M3> S;
  constexpr int LANES = D * (E4M3 ? 1 : 2) / 16, STEP = 64 * kWaves / LANES;
#pragma unroll
  for (int i = 0; i < S::KL; ++i) {
    const int t = tid / LANES + i * STEP;
    uint16_t* to = &lds.k[buf][t][(E4M3 ? 16 : 8) * (tid % LANES)];
    if constexpr (E4M3) {
      const v2u a = bf16_of_codes(x.k[i][0]), b = bf16_of_codes(x.k[i][1]), e = bf16_of_codes(x.k[i][2]), f = bf16_of_codes(x.k[i][3]);
      *reinterpret_cast<v4u*>(to) = v4u{a[0], a[1], b[0], b[1]};
      *reinterpret_cast<v4u*>(to + 8) = v4u{e[0], e[1], f[0], f[1]};
    } else {
      *reinterpret_cast<v4u*>(to) = x.k[i];
    }
  }
  const int t = 4 * (tid >> 4);
  const bool held = pick(id, wave) >= 0;
#pragma unroll
  for (int u = 0; u < S::VU; ++u) {
    unsigned w[4][S::VDIM / 2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < S::VW; ++k) {
        if constexpr (E4M3) {
          const v2u p = bf16_of_codes(x.v[u][i][k]);
          w[i][2 * k] = p[0];
          w[i][2 * k + 1] = p[1];
        } else {
          w[i][k] = x.v[u][i][k];
        }
      }
    if (some) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool on = held && j + t + i < n;
        bool bad = false;
#pragma unroll
        for (int k = 0; k < S::VDIM / 2; ++k) bad |= odd_pair(w[i][k]);
        if (on && bad) atomicOr(odd, 1ull << (t + i));
#pragma unroll
        for (int k = 0; k < S::VDIM / 2; ++k) w[i][k] = on && !bad ? w[i][k] : 0u;
      }
    }
#pragma unroll
    for (int k = 0; k < S::VDIM / 2; ++k) {
      const int row = u * 128 + 32 * k + (tid & 15);  // dim 128 u + VDIM (row % 16) + row / 16
      *reinterpret_cast<v2u*>(&lds.v[buf][row][t]) = v2u{low_halves(w[0][k], w[1][k]), low_halves(w[2][k], w[3][k])};
      *reinterpret_cast<v2u*>(&lds.v[buf][row + 16][t]) = v2u{high_halves(w[0][k], w[1][k]), high_halves(w[2][k], w[3][k])};
    }
  }
  if constexpr (E4M3) {
    if (tid < 128) lds.scales[buf][tid >> 6][tid & 63] = tid < 64 ? x.scale * factor : x.scale;
  }
}

// Rows of a sequence: new tokens times the heads of a group.
struct Rows {
  int first, count;  // its first row of q, and its new tokens
};
__device__ __forceinline__ Rows rows_of(const int* starts, int b, int T) {
  const int t0 = min(max(starts[b], 0), T), t1 = min(max(starts[b + 1], t0), T);
  return {t0, t1 - t0};
}

template <int D, bool E4M3>
__global__ __launch_bounds__(64 * kWaves, D == 256 ? 1 : 2) void prompt(Fp4AttentionArgs a, int group, int tiles) {
  extern __shared__ __align__(16) uint8_t memory[];
  typedef Lds<D, E4M3> L;
  L& lds = *reinterpret_cast<L*>(memory);
  const Paged& c = a.cache;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int slot = blockIdx.x / c.heads, head = blockIdx.x - slot * c.heads;
  // which rows: the last tiles first, they see the most
  int b = -1, tile = tiles - 1 - slot;
  for (int b0 = 0; b0 < c.batch; b0 += 64) {
    const int mine = b0 + lane < c.batch ? (rows_of(a.starts, b0 + lane, a.T).count * group + kRows - 1) / kRows : 0;
    const int upto = wave_prefix(mine);
    const uint64_t after = __ballot(upto > tile);
    if (after) {
      const int at = __builtin_ctzll(after);
      b = b0 + at;
      tile -= __shfl(upto, at) - __shfl(mine, at);
      break;
    }
    tile -= __shfl(upto, 63);
  }
  b = __builtin_amdgcn_readfirstlane(b);
  tile = __builtin_amdgcn_readfirstlane(tile);
  if (b < 0) return;
  const Rows rows = rows_of(a.starts, b, a.T);
  const int len = length_of(c, b), base = len - rows.count;  // place of the first new token
  const int last = rows.count * group - 1;                        // its last row
  const int row = tile * kRows + wave * 32 + (lane & 31);
  const int mine = min(row, last), token = mine / group, place = base + token;
  const int* pages = c.table + b * c.table_stride;

  Range range;
  {
    const int i0 = base + tile * kRows / group, i1 = base + min(tile * kRows + kRows - 1, last) / group;
    range.n = min(min(len, paged_room(c)), i1 + 1);
    const int lo = a.window ? max(i0 - a.window + 1, 0) : 0;
    const int end = max((range.n + kTokens - 1) / kTokens, 0);
    range.ta = max((min(a.sinks, range.n) + kTokens - 1) / kTokens, 0);
    range.tb = lo / kTokens;
    if (range.tb <= range.ta) range.ta = range.tb = end;
    range.tiles = range.ta + max(end - range.tb, 0);
  }
  // the wave's first and last places
  const int w0 = base + min(tile * kRows + wave * 32, last) / group, w1 = base + min(tile * kRows + wave * 32 + 31, last) / group;
  const int g0 = base + tile * kRows / group, g1 = base + min(tile * kRows + kRows - 1, last) / group;

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
  // does everything in the tile from j on count for all rows of places from i0 to i1?
  auto whole = [&](const Ids& id, int j, int i0, int i1) {
    return j + kTokens <= range.n && j + kTokens - 1 <= i0 && (a.window == 0 || j > i1 - a.window || j + kTokens <= a.sinks) &&
           (id.page[0] | id.page[1] | id.page[2] | id.page[3]) >= 0;
  };

  Staged<D, E4M3> next;
  const Fetch<D, E4M3> fetch(c, tid);
  Ids id = ids_of(c, pages, range, 0), ahead = ids_of(c, pages, range, 1);
  bool some = false;  // not all rows see all of the tile that lies in LDS
  if (tid < 4) lds.odd[tid] = 0;
  __syncthreads();
  if (range.tiles > 0) {
    const int j = range.first_of(0);
    fetch(next, c, head, id, j, wave, tid);
    some = !whole(id, j, g0, g1);
    store<D, E4M3>(lds, next, 0, id, j, range.n, factor, some, &lds.odd[0], wave, tid);
  }
  __syncthreads();
  for (int it = 0; it < range.tiles; ++it) {
    const int buf = it & 1, j = range.first_of(it), jn = range.first_of(it + 1);
    const bool more = it + 1 < range.tiles;
    if (more) fetch(next, c, head, ahead, jn, wave, tid);
    const Ids after = ids_of(c, pages, range, it + 2);
    if (tid == 0) lds.odd[(it + 2) & 3] = 0;  // read two tiles ago, next written behind the next barrier
    const bool hidden = j > w1 || (a.window && j + kTokens - 1 <= w0 - a.window && j >= a.sinks);
    if (!hidden) {
      // scores as plain floats: changing elements of a matrix register under a branch was compiled wrongly (D = 256, one
      // element copied over all others, by the clang of ROCm 7.2)
      float s[2][16];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        v16f acc;
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = 0.f;
        const int r = lane & 31, t = 32 * u + ((r & 0x13) | ((r & 4) << 1) | ((r & 8) >> 1));
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const v8bf k = __builtin_bit_cast(v8bf, *reinterpret_cast<const v4u*>(&lds.k[buf][t][16 * i + 8 * half]));
          acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k, q[i], acc, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[u][i] = acc[i];
          if (E4M3) s[u][i] *= lds.scales[buf][0][32 * u + 16 * (i / 8) + 8 * half + i % 8];
        }
      }
      const bool all = whole(id, j, w0, w1);
      if (!all) {
        const int from = a.window ? place - a.window : -1, to = min(place, range.n - 1);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int at = j + 32 * u + 16 * (i / 8) + 8 * half + i % 8;
            const bool on = (at <= to) & ((at > from) | (at < a.sinks)) & (id.page[2 * u + i / 8] >= 0);
            s[u][i] = on ? s[u][i] : kNever;
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
        for (int m2 = 0; m2 < D / 32; ++m2)
#pragma unroll
          for (int i = 0; i < 16; ++i) o[m2][i] *= keep;
      }
      const float m = top == kNever ? 0.f : top;
      if (some) {
        if (const unsigned long long odd = lds.odd[it & 3]) {  // a row that sees such a token is none of numbers
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (((odd >> (32 * u + 16 * (i / 8) + 8 * half + i % 8)) & 1) && s[u][i] != kNever) sum = __builtin_nanf("");
        }
      }
      v8bf p[2][2];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          v4u w;
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            float x[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) x[k] = exp2_hw(__builtin_fmaf(s[u][8 * e + i + k], unit, -m));
            if constexpr (E4M3) {
              sum += x[0] + x[1];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const float y = x[k] * lds.scales[buf][1][32 * u + 16 * e + 8 * half + i + k];
                x[k] = s[u][8 * e + i + k] == kNever ? 0.f : y;  // a hidden token's scale may be anything
              }
            }
            w[i / 2] = bf16_pair(x[0], x[1]);
            if (!E4M3) sum = add_pair(w[i / 2], sum);
          }
          p[u][e] = __builtin_bit_cast(v8bf, w);
        }
#pragma unroll
      for (int m2 = 0; m2 < D / 32; ++m2)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const v8bf v = __builtin_bit_cast(
                v8bf, *reinterpret_cast<const v4u*>(&lds.v[buf][32 * m2 + (lane & 31)][32 * u + 16 * e + 8 * half]));
            o[m2] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, p[u][e], o[m2], 0, 0, 0);
          }
    }
    if (more) {
      some = !whole(ahead, jn, g0, g1);
      store<D, E4M3>(lds, next, buf ^ 1, ahead, jn, range.n, factor, some, &lds.odd[(it + 1) & 3], wave, tid);
    }
    id = ahead;
    ahead = after;
    __syncthreads();
  }
  sum = sum_across<32>(sum);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  // rows of out through LDS: a wave's 32 rows, D + 8 elements apart
  uint16_t* mem = reinterpret_cast<uint16_t*>(memory) + wave * 32 * (D + 8);
  constexpr int VDIM = Staged<D, E4M3>::VDIM;
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

template <int D, bool E4M3>
hipError_t launch(const Fp4AttentionArgs& a, hipStream_t st) {
  const int group = a.q_heads / a.cache.heads;
  const int64_t tiles = ((int64_t)a.T * group + kRows - 1) / kRows + a.cache.batch;
  constexpr int bytes = sizeof(Lds<D, E4M3>);
  static std::atomic<int> ready[64];  // by device
  auto kern = prompt<D, E4M3>;
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const bool cached = dev >= 0 && dev < 64;
  if (!cached || !ready[dev].load(std::memory_order_acquire)) {
    e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    if (cached) ready[dev].store(1, std::memory_order_release);
  }
  hipLaunchKernelGGL(kern, dim3((unsigned)(tiles * a.cache.heads)), dim3(64 * kWaves), bytes, st, a, group, (int)tiles);
  return hipGetLastError();
}

}  // namespace
}  // namespace fp4

hipError_t fp4_launch_attention_prompt(const Fp4AttentionArgs& a, int dim, bool e4m3, hipStream_t st) {
  using namespace fp4;
  if (dim == 64) return e4m3 ? launch<64, true>(a, st) : launch<64, false>(a, st);
  if (dim == 128) return e4m3 ? launch<128, true>(a, st) : launch<128, false>(a, st);
  return e4m3 ? launch<256, true>(a, st) : launch<256, false>(a, st);
}
