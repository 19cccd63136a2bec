// The paged key-value cache as the kernels see it, and its launchers. A page holds page_size = 1 << shift tokens of every head;
// table[b, i >> shift] names the page of token i of sequence b. Page sizes are powers of two from 16 on, so 16 consecutive tokens
// from a multiple of 16 lie in one page: a "granule", for which one look into the table is enough.
#pragma once

#include "fp8_device.hpp"

namespace fp4 {

struct Paged {
  const uint8_t *k, *v;               // bf16, or E4M3 codes
  const float *k_scales, *v_scales;   // E4M3: one for a token's values of a head
  int64_t page_stride, head_stride, token_stride;     // bytes
  int64_t spage_stride, shead_stride, stoken_stride;  // scales, elements
  const int* table;
  int64_t table_stride;
  const int* lengths;
  int pages, shift, cols, batch, heads;
};

constexpr int kGranule = 16;

// Tokens that the table has room for.
__device__ __forceinline__ int paged_room(const Paged& p) { return p.cols << p.shift; }

// Tokens of sequence b, those that the table has no room for included; no more than 2^30 count, so that places and their
// differences from a window (at most 2^30 too) stay within 32 bits.
__device__ __forceinline__ int length_of(const Paged& p, int b) { return min(max(p.lengths[b], 0), 1 << 30); }

// Sum over the lanes up to this one, and over all 64: additions with DPP, in rows of 16 and then across them (through LDS, as shuffles
// go, these sums were a microsecond of a call).
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_part(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ int wave_prefix(int v) {
  v += dpp_part<0x111, 0xF>(v);  // row_shr:1, 2, 4, 8
  v += dpp_part<0x112, 0xF>(v);
  v += dpp_part<0x114, 0xF>(v);
  v += dpp_part<0x118, 0xF>(v);
  v += dpp_part<0x142, 0xA>(v);  // row_bcast:15 into rows 1 and 3
  v += dpp_part<0x143, 0xC>(v);  // row_bcast:31 into rows 2 and 3
  return v;
}
__device__ __forceinline__ int wave_total(int v) { return __builtin_amdgcn_readlane(wave_prefix(v), 63); }

// The sequence of row t of a batch of rows, or -1 where it belongs to none. starts is NULL for one row each.
__device__ __forceinline__ int sequence_of(const int* starts, int batch, int t) {
  if (starts == nullptr) return t < batch ? t : -1;
  int n = 0;
  for (int b = 0; b < batch; b += 64) {
    const int at = b + (threadIdx.x & 63);
    n += __popcll(__ballot(at < batch && starts[at + 1] <= t));
  }
  return n < batch && starts[n] <= t ? n : -1;
}

}  // namespace fp4

struct Fp4AppendArgs {
  fp4::Paged cache;
  const int* starts;
  const uint16_t *q, *k, *v;
  uint16_t* q_out;
  int64_t q_token, q_head, k_token, k_head, v_token, v_head, out_token, out_head;  // strides, elements
  const float* freqs;
  const int *positions, *axes;  // positions [naxes, T]
  int T, q_heads, half, naxes;
  bool interleaved;
};
hipError_t fp4_launch_kv_append(const Fp4AppendArgs& a, int dim, bool e4m3, hipStream_t stream);

struct Fp4AttentionArgs {
  fp4::Paged cache;
  const int* starts;  // prompt only
  const uint16_t* q;
  uint16_t* out;  // contiguous [T, q_heads, dim]
  int64_t q_token, q_head;
  float scale;
  int T, q_heads, window, sinks;
  void* workspace;
};
inline fp4::AttentionCall fp4_call_of(const Fp4AttentionArgs& a, int dim, bool e4m3) {
  const fp4::Paged& c = a.cache;
  return {dim, e4m3, a.T, c.batch, a.q_heads, c.heads, (int64_t)c.cols << c.shift, a.window, a.sinks, c.head_stride == (int64_t)dim * (e4m3 ? 1 : 2)};
}
hipError_t fp4_launch_attention_decode(const Fp4AttentionArgs& a, int dim, bool e4m3, hipStream_t stream);
hipError_t fp4_launch_attention_prompt(const Fp4AttentionArgs& a, int dim, bool e4m3, hipStream_t stream);
