// Keys and values of new tokens into a paged cache, with the position rotation of keys and queries on the way.
//
//   pair (a, b) -> (a cos w - b sin w, a sin w + b cos w),  w = position * freqs[f]
//   E4M3 cache: scale = max(|x|, 2^-100) / 448 over a token's values of a head, codes of x / scale
//
// Bound by memory: 2 bytes read for an element, 2 written (1 for a code). A wave takes a token, or a part of one where there are few
// tokens; a lane holds 16 elements, 8 pairs, so that both numbers of a pair are at hand in either order and a head of 64, 128 or
// 256 is 4, 8 or 16 lanes of one DPP row: its largest magnitude needs no LDS. Waves share nothing and never wait for each other.
//
// Angles: a position of 10^6 times a frequency of 1 has a float32 error of 0.03, so the product and its remainder of whole turns are
// taken in float64 (once for a token's heads) and only the remainder's sine and cosine in float32.
#include "paged.hpp"

namespace fp4 {
namespace {

constexpr int kWaves = 4;

// Largest magnitude over the 4, 8 or 16 lanes that hold a head.
template <int LANES>
__device__ __forceinline__ unsigned head_max(unsigned m) {
  m = max(m, (unsigned)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, false));                   // lane ^ 1
  m = max(m, (unsigned)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, false));                   // lane ^ 2
  if (LANES > 4) m = max(m, (unsigned)__builtin_amdgcn_update_dpp(0, (int)m, 0x141, 0xF, 0xF, false));   // 7 - lane of 8
  if (LANES > 8) m = max(m, (unsigned)__builtin_amdgcn_update_dpp(0, (int)m, 0x140, 0xF, 0xF, false));   // 15 - lane of 16
  return m;
}

// Calls that read more than this stream rows and rotated queries past the caches; of smaller ones the next kernel finds them there.
// Both ways, us: 26601 tokens of 48 heads of 128 (327 MB) 119.5 / 103.4, 3216 of 20 heads (16 MB) 9.3 / 9.7. The cache's entries are
// stored the usual way: a token's 8 or 16 bytes of a lane do not fill a line (streamed: 111.7).
constexpr int64_t kStreamBytes = (int64_t)96 << 20;

template <bool STREAM>
__device__ __forceinline__ void put(void* to, v4u v) {
  if constexpr (STREAM) __builtin_nontemporal_store(v, reinterpret_cast<v4u*>(to));
  else *reinterpret_cast<v4u*>(to) = v;
}
template <bool STREAM>
__device__ __forceinline__ v4u take(const void* from) {
  return STREAM ? __builtin_nontemporal_load(reinterpret_cast<const v4u*>(from)) : *reinterpret_cast<const v4u*>(from);
}

// 16 elements of a token's head, as two halves of 8: those of a rotated piece that are not interleaved lie half a rotation apart.
struct Piece {
  int head, piece, e0, e1;  // the halves' first elements
  bool query, key, turn;
  v4u w0, w1;
};
template <int D, bool STREAM>
__device__ __forceinline__ Piece piece_of(const Fp4AppendArgs& a, int t, int u) {
  constexpr int PIECES = D / 16;
  Piece p;
  const int h = u / PIECES;
  p.piece = u % PIECES;
  p.query = h < a.q_heads;
  p.key = !p.query && h < a.q_heads + a.cache.heads;
  p.head = p.query ? h : p.key ? h - a.q_heads : h - a.q_heads - a.cache.heads;
  p.turn = (p.query || p.key) && p.piece < a.half / 8;
  const bool apart = p.turn && !a.interleaved;
  p.e0 = apart ? 8 * p.piece : 16 * p.piece;
  p.e1 = apart ? a.half + 8 * p.piece : 16 * p.piece + 8;
  const uint16_t* x = p.query ? a.q + t * a.q_token + p.head * a.q_head
                      : p.key ? a.k + t * a.k_token + p.head * a.k_head
                              : a.v + t * a.v_token + p.head * a.v_head;
  p.w0 = take<STREAM>(x + p.e0);
  p.w1 = take<STREAM>(x + p.e1);
  return p;
}

template <int D, bool E4M3, bool STREAM>
__global__ __launch_bounds__(64 * kWaves) void kv_append(Fp4AppendArgs a, int parts) {
  constexpr int PIECES = D / 16;  // lanes of a head
  __shared__ float trig[kWaves][2][D / 2];
  const Paged& c = a.cache;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t id = (int64_t)blockIdx.x * kWaves + wave;
  const int t = (int)(id / parts), part = (int)(id - (int64_t)t * parts);
  if (t >= a.T) return;
  const int units = (a.q_heads + 2 * c.heads) * PIECES;
  const int b = __builtin_amdgcn_readfirstlane(sequence_of(a.starts, c.batch, t));
  if (b < 0) return;
  const int i = (int)((unsigned)c.lengths[b] - (unsigned)(a.starts ? a.starts[b + 1] - t : 1));
  int page = -1;
  if (i >= 0 && (i >> c.shift) < c.cols) page = c.table[b * c.table_stride + (i >> c.shift)];
  const bool held = (unsigned)page < (unsigned)c.pages;
  float* cosines = trig[wave][0];
  float* sines = trig[wave][1];
  for (int f = lane; f < a.half; f += 64) {
    int pos = i;
    if (a.positions) {
      const int axis = a.axes ? a.axes[f] : 0;
      pos = (unsigned)axis < (unsigned)a.naxes ? a.positions[(int64_t)axis * a.T + t] : 0;
    }
    const double turns = (double)pos * (double)a.freqs[f] * 0.15915494309189533577;  // 1 / (2 pi)
    const float r = (float)(turns - __builtin_rint(turns));
    float sn, cs;
    sincospif(2.0f * r, &sn, &cs);
    cosines[f] = cs;
    sines[f] = sn;
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();

  const int64_t in = i & ((1 << c.shift) - 1);
  const int64_t place = held ? page * c.page_stride + in * c.token_stride : 0;
  const int64_t splace = held && E4M3 ? page * c.spage_stride + in * c.stoken_stride : 0;
  for (int u = part * 64 + lane; u < units; u += parts * 64) {
    const Piece p = piece_of<D, STREAM>(a, t, u);
    if (!p.query && !held) continue;  // for all lanes of a head
    float f[16];
    widen8(p.w0, f);
    widen8(p.w1, f + 8);
    if (p.turn) {
      const float *cs = cosines + 8 * p.piece, *sn = sines + 8 * p.piece;
      if (a.interleaved) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float x0 = f[2 * j], x1 = f[2 * j + 1];
          f[2 * j] = x0 * cs[j] - x1 * sn[j];
          f[2 * j + 1] = x0 * sn[j] + x1 * cs[j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float x0 = f[j], x1 = f[j + 8];
          f[j] = x0 * cs[j] - x1 * sn[j];
          f[j + 8] = x0 * sn[j] + x1 * cs[j];
        }
      }
    }
    if (p.query) {
      uint16_t* y = a.q_out + t * a.out_token + p.head * a.out_head;
      put<STREAM>(y + p.e0, narrow8(f));
      put<STREAM>(y + p.e1, narrow8(f + 8));
      continue;
    }
    uint8_t* y = const_cast<uint8_t*>(p.key ? c.k : c.v) + place + p.head * c.head_stride;
    if (E4M3) {
      unsigned m = 0;
#pragma unroll
      for (int j = 0; j < 16; ++j) m = max(m, abs_bits(f[j]));
      m = head_max<PIECES>(m);
      const float inv = f8_inverse(m);
      *reinterpret_cast<v2u*>(y + p.e0) = f8_codes8(f, inv);
      *reinterpret_cast<v2u*>(y + p.e1) = f8_codes8(f + 8, inv);
      if (p.piece == 0) const_cast<float*>(p.key ? c.k_scales : c.v_scales)[splace + p.head * c.shead_stride] = f8_scale(m);
    } else {
      *reinterpret_cast<v4u*>(y + 2 * p.e0) = p.turn ? narrow8(f) : p.w0;
      *reinterpret_cast<v4u*>(y + 2 * p.e1) = p.turn ? narrow8(f + 8) : p.w1;
    }
  }
}

template <int D, bool E4M3>
hipError_t launch(const Fp4AppendArgs& a, hipStream_t st) {
  const int64_t per = ((int64_t)(a.q_heads + 2 * a.cache.heads) * (D / 16) + 63) / 64;  // waves that a token can use
  int64_t parts = (2048 + a.T - 1) / a.T;  // few tokens are spread over 8 waves of each CU
  if (parts > per) parts = per;
  const int64_t waves = a.T * parts;
  auto kern = (int64_t)a.T * (a.q_heads + 2 * a.cache.heads) * D * 2 > kStreamBytes ? kv_append<D, E4M3, true> : kv_append<D, E4M3, false>;
  hipLaunchKernelGGL(kern, dim3((unsigned)((waves + kWaves - 1) / kWaves)), dim3(64 * kWaves), 0, st, a, (int)parts);
  return hipGetLastError();
}

}  // namespace
}  // namespace fp4

hipError_t fp4_launch_kv_append(const Fp4AppendArgs& a, int dim, bool e4m3, hipStream_t st) {
  using namespace fp4;
  if (dim == 64) return e4m3 ? launch<64, true>(a, st) : launch<64, false>(a, st);
  if (dim == 128) return e4m3 ? launch<128, true>(a, st) : launch<128, false>(a, st);
  return e4m3 ? launch<256, true>(a, st) : launch<256, false>(a, st);
}
