// Blockwise-scaled E4M3 GEMM for few rows of X (gfx950): Y[m, n] = sum over blocks b of 128 along K of
// xs[m, b] * ws[n / 128, b] * sum over k in b of xq[m, k] * wq[n, k].
//
// W (N x K bytes) is the only large operand, so the product is bound by streaming it from HBM:
//  * One workgroup owns T tiles of 16 output features and all of K; its 8 waves split K into slices
//    of 256 bytes (two scale blocks), slice s going to wave s % 8. Each wave fetches its slices into its
//    own LDS ring of kRing slices with the LDS DMA (one instruction: 4 rows x 256 contiguous bytes), 16-byte
//    chunks XOR-swizzled by the row so that the fragment reads hit distinct banks, and multiplies a
//    slice when its own loads have landed: no barrier stands between a wave's data and its products.
//  * v_mfma_f32_16x16x128_f8f6f4 with W as the row operand and X as the column operand: one
//    instruction is one scale block, and its 16x16 result gives each lane 4 features of ONE token, so
//    the block's scale xs * ws is one value per lane and acc += p * s is four float32 FMAs.
//  * X (a few rows) is read per lane from L2. MF = ceil(M / 16) column fragments share every W
//    fragment, so W is read once for up to 64 rows; more rows take further workgroups (grid y).
//  * The waves' float32 sums meet through LDS in a fixed order: the result does not depend on timing.
#include <atomic>
#include <type_traits>

#include "fp8_device.hpp"

namespace fp4 {
namespace {

typedef __attribute__((address_space(3))) void lds_void;

constexpr int kWaves = 8;
constexpr int kThreads = kWaves * 64;
constexpr int kSlice = 256;            // bytes of K of a slice: two scale blocks
constexpr int kSliceBytes = 16 * kSlice;  // of 16 rows
constexpr int kRing = 2;               // slices a wave holds or has in flight

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_rsrc(const void* base, unsigned bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00020000);
}

// Y[m][n .. n+3] = a rounded to bf16, bounds-checked.
__device__ __forceinline__ void store4(uint16_t* __restrict__ Y, int64_t M, int N, int64_t m, int n, v4f a) {
  if (m >= M) return;
  uint16_t* dst = Y + (size_t)m * N + n;
  uint16_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = __builtin_bit_cast(uint16_t, (__bf16)a[i]);
  if ((N & 3) == 0 && n + 3 < N) {
    *reinterpret_cast<v2u*>(dst) = v2u{b[0] | ((unsigned)b[1] << 16), b[2] | ((unsigned)b[3] << 16)};
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < N) dst[i] = b[i];
  }
}

__device__ __forceinline__ v4f mfma_f8(v4u a0, v4u a1, v4u b0, v4u b1) {
  const v8i a = {(int)a0[0], (int)a0[1], (int)a0[2], (int)a0[3], (int)a1[0], (int)a1[1], (int)a1[2], (int)a1[3]};
  const v8i b = {(int)b0[0], (int)b0[1], (int)b0[2], (int)b0[3], (int)b1[0], (int)b1[1], (int)b1[2], (int)b1[3]};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

template <int T, int MF>
__global__ __launch_bounds__(kThreads) void gemm_fp8_decode(const uint8_t* __restrict__ Xq,
                                                            const float* __restrict__ Xs,
                                                            const uint8_t* __restrict__ Wq,
                                                            const float* __restrict__ Ws, uint16_t* __restrict__ Y,
                                                            int64_t M, int N, int K) {
  static_assert(MF * T <= kWaves && MF <= 4, "one output fragment per wave in the reduction");
  static_assert(MF <= 4 * kRing, "the partial sums fit a wave's ring");
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  constexpr int area_bytes = kRing * T * kSliceBytes;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int nb = blockIdx.x * 16 * T;
  const int64_t m0 = (int64_t)blockIdx.y * (16 * MF);
  const int kb = K / kF8Group, nsl = (kb + 1) / 2;
  const int mine = nsl > wave ? (nsl - wave + kWaves - 1) / kWaves : 0;  // this wave's slices
  uint8_t* area = lds + wave * area_bytes;
  const float* ws = Ws + (size_t)(nb / kF8Group) * kb;  // 16 T divides 128: one row of scales

  // W slice j of this wave into ring slot j % kRing. Chunk q of row i sits at slot q ^ i of the row;
  // rows past N and bytes past the operand read as zero. The second half of the last slice of an odd
  // number of blocks holds other data, which no product reads.
  auto fetch = [&](int j) {
    const unsigned at = (unsigned)(wave + kWaves * j) * kSlice;
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const int n0 = min(nb + 16 * t, N - 1);
      const __amdgpu_buffer_rsrc_t rw = buffer_rsrc(Wq + (size_t)n0 * K, (unsigned)min(16, N - n0) * (unsigned)K);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 4 * i + g;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)(area + ((j % kRing) * T + t) * kSliceBytes + i * 1024),
                                                 16, (unsigned)row * (unsigned)K + at + 16u * (unsigned)(r ^ row), 0, 0, 0);
      }
    }
  };
  const uint8_t* xp[MF];
  const float* xsp[MF];
#pragma unroll
  for (int f = 0; f < MF; ++f) {
    const int64_t m = min(m0 + 16 * f + r, M - 1);  // rows past M repeat the last one and are not stored
    xp[f] = Xq + (size_t)m * K + 32 * g;
    xsp[f] = Xs + (size_t)m * kb;
  }

  v4f acc[MF][T];
#pragma unroll
  for (int f = 0; f < MF; ++f)
#pragma unroll
    for (int t = 0; t < T; ++t) acc[f][t] = v4f{0.f, 0.f, 0.f, 0.f};

  for (int j = 0; j < kRing && j < mine; ++j) fetch(j);
  for (int j = 0; j < mine; ++j) {
    const int s = wave + kWaves * j;
    const int blocks = min(2, kb - 2 * s);
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): the slice has landed
    asm volatile("" ::: "memory");
    v4u wf[T][2][2];
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          wf[t][u][h] = *reinterpret_cast<const v4u*>(area + ((j % kRing) * T + t) * kSliceBytes + r * kSlice +
                                                      16 * ((8 * u + 2 * g + h) ^ r));
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (u < blocks) {  // wave-uniform
        const int b = 2 * s + u;
        const float sw = ws[b];
#pragma unroll
        for (int f = 0; f < MF; ++f) {
          const v4u x0 = *reinterpret_cast<const v4u*>(xp[f] + (size_t)b * kF8Group);
          const v4u x1 = *reinterpret_cast<const v4u*>(xp[f] + (size_t)b * kF8Group + 16);
          const float sc = xsp[f][b] * sw;
#pragma unroll
          for (int t = 0; t < T; ++t) {
            const v4f p = mfma_f8(wf[t][u][0], wf[t][u][1], x0, x1);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[f][t][i] = __builtin_fmaf(p[i], sc, acc[f][t][i]);
          }
        }
      }
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the slice has been read before its slot is refilled
    asm volatile("" ::: "memory");
    if (j + kRing < mine) fetch(j + kRing);
  }

  // The partial sums of output fragment q = f T + t meet in the order of the waves, summed by wave q.
  v4f* red = reinterpret_cast<v4f*>(area);
#pragma unroll
  for (int f = 0; f < MF; ++f)
#pragma unroll
    for (int t = 0; t < T; ++t) red[(f * T + t) * 64 + lane] = acc[f][t];
  __syncthreads();
  if (wave >= MF * T) return;
  const int f = wave / T, t = wave % T;
  v4f sum = reinterpret_cast<const v4f*>(lds)[wave * 64 + lane];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) sum += reinterpret_cast<const v4f*>(lds + w * area_bytes)[wave * 64 + lane];
  store4(Y, M, N, m0 + 16 * f + r, nb + 16 * t + 4 * g, sum);
}

template <int T, int MF>
hipError_t launch(const uint8_t* Xq, const float* Xs, const uint8_t* Wq, const float* Ws, int64_t M, int N, int K,
                  uint16_t* Y, hipStream_t st) {
  static std::atomic<int> ready[64];
  constexpr int lds = kWaves * kRing * T * kSliceBytes;
  auto kern = gemm_fp8_decode<T, MF>;
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const bool cached = dev >= 0 && dev < 64;
  if (!cached || !ready[dev].load(std::memory_order_acquire)) {
    e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
    if (cached) ready[dev].store(1, std::memory_order_release);
  }
  const dim3 grid((unsigned)((N + 16 * T - 1) / (16 * T)), (unsigned)((M + 16 * MF - 1) / (16 * MF)));
  hipLaunchKernelGGL(kern, grid, dim3(kThreads), lds, st, Xq, Xs, Wq, Ws, Y, M, N, K);
  return hipGetLastError();
}

}  // namespace
}  // namespace fp4

hipError_t fp8_launch_linear(const uint8_t* Xq, const float* Xs, const uint8_t* Wq, const float* Ws, int64_t M,
                             int64_t N, int64_t K, uint16_t* Y, hipStream_t st) {
  auto go = [&](auto mf) {
    return fp4::launch<1, decltype(mf)::value>(Xq, Xs, Wq, Ws, M, (int)N, (int)K, Y, st);
  };
  if (M > 64) return fp8_launch_linear_ring(Xq, Xs, Wq, Ws, M, N, K, Y, st);
  switch ((int)((M + 15) / 16)) {
    case 1: return go(std::integral_constant<int, 1>{});
    case 2: return go(std::integral_constant<int, 2>{});
    case 3: return go(std::integral_constant<int, 3>{});
    default: return go(std::integral_constant<int, 4>{});
  }
}
