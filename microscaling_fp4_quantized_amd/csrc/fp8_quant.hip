// 8-bit quantizers of the blockwise-scaled E4M3 layers, and the RMS norm that feeds them (gfx950).
//
//   fp8_quantize              codes and one scale for 1 x 128 values of bf16 activations
//   fp8_quantize_weights      codes and one scale for 128 x 128 values of bf16 weights
//   fp8_add_rmsnorm_quantize  h = x + r, n = h / sqrt(mean(h^2) + eps) * w, n as fp8_quantize stores it
//
// All three are bound by memory: 2 bytes read and 1 + 4/128 written for an element (the norm also
// reads r and writes h and n where asked). Every element is read once: a lane holds 8 consecutive
// ones (16 bytes), so the 16 lanes of a DPP row hold the 128 of a scale and the maximum is four
// cross-lane steps without LDS. The norm keeps its row in registers between the sum of squares and
// the scaling. The sum of squares, the mean and the normalised row are float32.
//
// Measured, us of a call among others: norm with residual 16384 x 8192 155 (944 MB, 6.1 TB/s: a copy's rate), 1 x 4096 3.9-4.7
// (launch and host; 2.4 on the GPU); activations 2047 x 4096 6.0, weights 14336 x 4096 30.3 (176 MB, 5.8 TB/s).
#include <type_traits>

#include "fp8_device.hpp"

namespace fp4 {
namespace {

// Inputs of more than this are read and their outputs written past the caches (nontemporal): nothing of them would
// stay there for the next kernel, while smaller ones are mostly where the kernel before left them. Cached against
// nontemporal, us: norm with a residual 2048 x 4096 (34 MB read) 12.1 / 15.4, 8192 x 4096 (134 MB) 42.7 / 39.4,
// 16384 x 8192 (537 MB) 164.6 / 157.2; activations 14000 x 4096 (115 MB) 31.9 / 28.2; weights 14336 x 4096 (117 MB)
// 34.0 / 30.5, 28672 x 8192 130 / 118.
constexpr int64_t kStreamBytes = (int64_t)96 << 20;

template <bool NT, class T>
__device__ __forceinline__ T load_as(const void* p) {
  return NT ? __builtin_nontemporal_load(reinterpret_cast<const T*>(p)) : *reinterpret_cast<const T*>(p);
}
template <bool NT, class T>
__device__ __forceinline__ void store_as(void* p, T v) {
  if constexpr (NT) __builtin_nontemporal_store(v, reinterpret_cast<T*>(p));
  else *reinterpret_cast<T*>(p) = v;
}

constexpr int kQThreads = 256;
constexpr int kQUnroll = 4;  // chunks of 8 values in flight per lane

// Chunk c (8 values) of row c / cpr. Consecutive lanes take consecutive chunks; K % 128 == 0 makes
// every DPP row of lanes hold one whole group, and its lanes are past the end together.
template <bool CONTIG, bool STREAM>
__global__ __launch_bounds__(kQThreads) void quantize_rows(const uint16_t* __restrict__ X, int64_t ldx, uint32_t cpr,
                                                           uint32_t chunks, uint8_t* __restrict__ codes,
                                                           float* __restrict__ scales) {
  const uint32_t c0 = blockIdx.x * (uint32_t)(kQThreads * kQUnroll) + threadIdx.x;
  v4u w[kQUnroll];
#pragma unroll
  for (int u = 0; u < kQUnroll; ++u) {
    const uint32_t c = min(c0 + u * kQThreads, chunks - 1);
    const uint32_t row = CONTIG ? 0 : c / cpr;
    w[u] = load_as<STREAM, v4u>(X + (size_t)row * (size_t)ldx + (size_t)(c - row * cpr) * 8);
  }
#pragma unroll
  for (int u = 0; u < kQUnroll; ++u) {
    const uint32_t c = c0 + u * kQThreads;
    if (c >= chunks) break;
    float v[8];
    widen8(w[u], v);
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
    m = row16_max(m);
    store_as<STREAM>(codes + (size_t)c * 8, f8_codes8(v, f8_inverse(m)));
    if ((threadIdx.x & 15) == 0) scales[c >> 4] = f8_scale(m);
  }
}

// One 128 x 128 block of W per workgroup: lane l of load i takes 8 columns of row 16 i + l / 16.
template <bool STREAM>
__global__ __launch_bounds__(kQThreads) void quantize_blocks(const uint16_t* __restrict__ W, int64_t ldw, int64_t N,
                                                             int64_t K, uint8_t* __restrict__ codes,
                                                             float* __restrict__ scales) {
  __shared__ unsigned red[kQThreads / 64];
  const int64_t kb = K / kF8Group;
  const int64_t bn = (int64_t)blockIdx.x / kb, bk = (int64_t)blockIdx.x % kb;
  const int64_t r0 = bn * kF8Group + (threadIdx.x >> 4), col = bk * kF8Group + (threadIdx.x & 15) * 8;
  v4u w[8];
  unsigned m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = min(r0 + 16 * i, N - 1);  // rows past N repeat the last one: no new maximum
    w[i] = load_as<STREAM, v4u>(W + r * ldw + col);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v[8];
    widen8(w[i], v);
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[j]));
  }
#pragma unroll
  for (int h = 32; h > 0; h >>= 1) m = max(m, (unsigned)__shfl_xor((int)m, h));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  m = max(max(red[0], red[1]), max(red[2], red[3]));
  const float inv = f8_inverse(m);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + 16 * i;
    if (r >= N) break;
    float v[8];
    widen8(w[i], v);
    store_as<STREAM>(codes + r * K + col, f8_codes8(v, inv));
  }
  if (threadIdx.x == 0) scales[blockIdx.x] = f8_scale(m);
}

// NT threads per row, V chunks of 8 values per thread, ROWS rows per workgroup (ROWS > 1: one wave
// per row, no LDS).
template <int NT, int V, int ROWS, bool RES, bool STREAM>
__global__ __launch_bounds__(NT* ROWS) void add_rmsnorm_quantize(const uint16_t* __restrict__ X, int64_t ldx,
                                                                 const uint16_t* R, int64_t ldr,
                                                                 const uint16_t* __restrict__ G, float eps, int64_t M,
                                                                 uint32_t K, uint8_t* __restrict__ codes,
                                                                 float* __restrict__ scales, uint16_t* H,
                                                                 uint16_t* __restrict__ Y) {
  static_assert(ROWS == 1 || NT == 64, "one row per workgroup, or one per wave");
  __shared__ float red[NT / 64];
  const int tid = ROWS > 1 ? threadIdx.x & 63 : threadIdx.x;
  // rows of one workgroup each are long, so their number fits the grid's x (fp8_launch_add_rmsnorm_quantize)
  const int64_t row =
      ROWS > 1 ? ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * ROWS + (threadIdx.x >> 6) : (int64_t)blockIdx.x;
  if (ROWS > 1 && row >= M) return;
  const uint32_t chunks = K / 8;
  const uint16_t* x = X + row * ldx;
  v4u xw[V], rw[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const uint32_t c = min((uint32_t)(i * NT + tid), chunks - 1);
    xw[i] = load_as<STREAM, v4u>(x + (size_t)c * 8);
    if constexpr (RES) rw[i] = load_as<STREAM, v4u>(R + row * ldr + (size_t)c * 8);
  }
  float h[V][8], sum = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    widen8(xw[i], h[i]);
    if constexpr (RES) {
      float r[8];
      widen8(rw[i], r);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] += r[j];
    }
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) s = __builtin_fmaf(h[i][j], h[i][j], s);
    if ((uint32_t)(i * NT + tid) < chunks) sum += s;
  }
  sum = wave_sum(sum);
  if constexpr (ROWS == 1 && NT > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = sum;
    __syncthreads();
    sum = red[0];
#pragma unroll
    for (int w = 1; w < NT / 64; ++w) sum += red[w];
  }
  const float rs = 1.0f / __builtin_sqrtf(sum / (float)K + eps);
  const size_t base = (size_t)row * K;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const uint32_t c = i * NT + tid;
    if (c >= chunks) break;  // whole DPP rows of lanes: K % 128 == 0
    if constexpr (RES) store_as<STREAM>(H + base + (size_t)c * 8, narrow8(h[i]));
    float g[8];
    widen8(*reinterpret_cast<const v4u*>(G + (size_t)c * 8), g);
    unsigned m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      h[i][j] = h[i][j] * rs * g[j];
      m = max(m, abs_bits(h[i][j]));
    }
    if (Y) store_as<STREAM>(Y + base + (size_t)c * 8, narrow8(h[i]));
    m = row16_max(m);
    store_as<STREAM>(codes + base + (size_t)c * 8, f8_codes8(h[i], f8_inverse(m)));
    if ((tid & 15) == 0) scales[(base >> 7) + (c >> 4)] = f8_scale(m);
  }
}

template <int NT, int V, int ROWS>
hipError_t launch_norm(const uint16_t* X, int64_t M, int64_t K, int64_t ldx, const uint16_t* R, int64_t ldr,
                       const uint16_t* G, float eps, uint8_t* codes, float* scales, uint16_t* H, uint16_t* Y,
                       hipStream_t st) {
  const bool stream = M * K * (R ? 4 : 2) > kStreamBytes;
  auto kern = R ? (stream ? add_rmsnorm_quantize<NT, V, ROWS, true, true> : add_rmsnorm_quantize<NT, V, ROWS, true, false>)
                : (stream ? add_rmsnorm_quantize<NT, V, ROWS, false, true> : add_rmsnorm_quantize<NT, V, ROWS, false, false>);
  const Grid grid = grid_of((M + ROWS - 1) / ROWS, NT * ROWS);
  hipLaunchKernelGGL(kern, dim3(grid.x, grid.y), dim3(NT * ROWS), 0, st, X, ldx, R, ldr, G, eps, M, (uint32_t)K, codes,
                     scales, H, Y);
  return hipGetLastError();
}

}  // namespace
}  // namespace fp4

hipError_t fp8_launch_quantize(const uint16_t* X, int64_t M, int64_t K, int64_t ldx, uint8_t* codes, float* scales,
                               hipStream_t st) {
  using namespace fp4;
  const uint32_t chunks = (uint32_t)(M * (K / 8)), per = kQThreads * kQUnroll;
  const bool stream = M * K * 2 > kStreamBytes;
  auto kern = ldx == K ? (stream ? quantize_rows<true, true> : quantize_rows<true, false>)
                       : (stream ? quantize_rows<false, true> : quantize_rows<false, false>);
  hipLaunchKernelGGL(kern, dim3((chunks + per - 1) / per), dim3(kQThreads), 0, st, X, ldx, (uint32_t)(K / 8), chunks,
                     codes, scales);
  return hipGetLastError();
}

hipError_t fp8_launch_quantize_weights(const uint16_t* W, int64_t N, int64_t K, int64_t ldw, uint8_t* codes,
                                       float* scales, hipStream_t st) {
  using namespace fp4;
  const int64_t blocks = (N + kF8Group - 1) / kF8Group * (K / kF8Group);
  auto kern = N * K * 2 > kStreamBytes ? quantize_blocks<true> : quantize_blocks<false>;
  hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(kQThreads), 0, st, W, ldw, N, K, codes, scales);
  return hipGetLastError();
}

hipError_t fp8_launch_add_rmsnorm_quantize(const uint16_t* X, int64_t M, int64_t K, int64_t ldx, const uint16_t* R,
                                           int64_t ldr, const uint16_t* G, float eps, uint8_t* codes, float* scales,
                                           uint16_t* H, uint16_t* Y, hipStream_t st) {
  using namespace fp4;
  auto go = [&](auto nt, auto v, auto rows) {
    return launch_norm<decltype(nt)::value, decltype(v)::value, decltype(rows)::value>(X, M, K, ldx, R, ldr, G, eps,
                                                                                       codes, scales, H, Y, st);
  };
  using std::integral_constant;
  typedef integral_constant<int, 1> i1;
  typedef integral_constant<int, 2> i2;
  typedef integral_constant<int, 4> i4;
  typedef integral_constant<int, 8> i8;
  typedef integral_constant<int, 64> t64;
  typedef integral_constant<int, 256> t256;
  typedef integral_constant<int, 1024> t1024;
  // M * K / 8 < 2^31: rows of more than 1024 are so few that 256 or 1024 threads each make less than 2^32
  if (K <= 512) return go(t64{}, i1{}, i4{});
  if (K <= 1024) return go(t64{}, i2{}, i4{});
  if (K <= 2048) return go(t256{}, i1{}, i1{});
  if (K <= 4096) return go(t256{}, i2{}, i1{});
  if (K <= 8192) return go(t256{}, i4{}, i1{});
  if (K <= 16384) return go(t256{}, i8{}, i1{});
  if (K <= 32768) return go(t1024{}, i4{}, i1{});
  return go(t1024{}, i8{}, i1{});  // K <= 65536
}
