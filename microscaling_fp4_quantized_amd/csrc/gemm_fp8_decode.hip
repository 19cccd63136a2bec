// Blockwise-scaled E4M3 GEMM for few rows of X (gfx950): Y[m, n] = sum over blocks b of 128 along K of
// xs[m, b] * ws[n / 128, b] * sum over k in b of xq[m, k] * wq[n, k].
//
// For up to 16 rows W (N x K bytes) is the only large operand, so the product is bound by streaming it from HBM:
//  * One workgroup owns 16 output features and all of K; its 8 waves split K into slices
//    of 256 bytes (two scale blocks), slice s going to wave s % 8. Each wave fetches its slices into its
//    own LDS ring of kRing slices with the LDS DMA (one instruction: 4 rows x 256 contiguous bytes), 16-byte
//    chunks XOR-swizzled by the row so that the fragment reads hit distinct banks, and multiplies a
//    slice when its own loads have landed: no barrier stands between a wave's data and its products.
//  * v_mfma_f32_16x16x128_f8f6f4 with W as the row operand and X as the column operand: one
//    instruction is one scale block, and its 16x16 result gives each lane 4 features of ONE token, so
//    the block's scale xs * ws is one value per lane and acc += p * s is four float32 FMAs.
//  * X is read per lane from L2, a slice ahead.
//  * The waves' float32 sums meet through LDS in a fixed order: the result does not depend on timing.
// Measured: 1 row, K = 4096: N = 4096 5.8 us, N = 14336 12.2 us (58.7 MB of W, 4.8 TB/s); N = 28672, K = 8192 43.0 us (5.5
// TB/s; a plain read of as much reaches 5.9-6.2). 4 waves 15.2, 16 waves 15.5 us at N = 14336.
#include <atomic>

#include "fp8_device.hpp"

namespace fp4 {
namespace {

typedef __attribute__((address_space(3))) void lds_void;

constexpr int kWaves = 8;
constexpr int kSlice = 256;            // bytes of K of a slice: two scale blocks
constexpr int kSliceBytes = 16 * kSlice;  // of 16 rows
constexpr int kRing = 2;               // slices a wave holds or has in flight

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_rsrc(const void* base, unsigned bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00020000);
}

// Y[m][n .. n+3] = a rounded to bf16, bounds-checked.
__device__ __forceinline__ void store4(uint16_t* __restrict__ Y, int M, int N, int m, int n, v4f a) {
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

__global__ __launch_bounds__(kWaves * 64) void gemm_fp8_decode(const uint8_t* __restrict__ Xq,
                                                               const float* __restrict__ Xs,
                                                               const uint8_t* __restrict__ Wq,
                                                               const float* __restrict__ Ws, uint16_t* __restrict__ Y,
                                                               int M, int N, int K) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  constexpr int area_bytes = kRing * kSliceBytes;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int nb = blockIdx.x * 16;
  const int kb = K / kF8Group, nsl = (kb + 1) / 2;
  const int mine = nsl > wave ? (nsl - wave + kWaves - 1) / kWaves : 0;  // this wave's slices
  uint8_t* area = lds + wave * area_bytes;
  const float* ws = Ws + (size_t)(nb / kF8Group) * kb;

  // W slice j of this wave into ring slot j % kRing. Chunk q of row i sits at slot q ^ i of the row;
  // rows past N and bytes past the operand read as zero. The second half of the last slice of an odd
  // number of blocks holds other data, which no product reads.
  const __amdgpu_buffer_rsrc_t rw = buffer_rsrc(Wq + (size_t)nb * K, (unsigned)min(16, N - nb) * (unsigned)K);
  auto fetch = [&](int j) {
    const unsigned at = (unsigned)(wave + kWaves * j) * kSlice;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 4 * i + g;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)(area + (j % kRing) * kSliceBytes + i * 1024), 16,
                                               (unsigned)row * (unsigned)K + at + 16u * (unsigned)(r ^ row), 0, 0, 0);
    }
  };
  const int m = min(r, M - 1);  // rows past M repeat the last one and are not stored
  const uint8_t* xp = Xq + (size_t)m * K + 32 * g;
  const float* xsp = Xs + (size_t)m * kb;
  v4u x[2][2][2];  // [slice % 2][block of it][16 bytes]
  float sc[2][2];
  auto load_x = [&](int j, int h) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int b = min(2 * (wave + kWaves * j) + u, kb - 1);
      x[h][u][0] = *reinterpret_cast<const v4u*>(xp + (size_t)b * kF8Group);
      x[h][u][1] = *reinterpret_cast<const v4u*>(xp + (size_t)b * kF8Group + 16);
      sc[h][u] = xsp[b];
    }
  };

  v4f acc = {0.f, 0.f, 0.f, 0.f};
  // X of a slice is requested before the W of the slice after it, so waiting for it leaves that W in flight.
  if (mine > 0) {
    fetch(0);
    load_x(0, 0);
  }
  if (mine > 1) fetch(1);
  for (int jj = 0; jj < mine; jj += 2) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int j = jj + h;
      if (j >= mine) break;  // uniform in the wave
      const int s = wave + kWaves * j;
      // the slice has landed: at most the next slice's loads are younger
      if (j + 1 < mine) __builtin_amdgcn_s_waitcnt(0x0F70 | 4);
      else __builtin_amdgcn_s_waitcnt(0x0F70);
      asm volatile("" ::: "memory");
      if (j + 1 < mine) load_x(j + 1, h ^ 1);
      v4u w[2][2];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int q = 0; q < 2; ++q)
          w[u][q] = *reinterpret_cast<const v4u*>(area + (j % kRing) * kSliceBytes + r * kSlice +
                                                  16 * ((8 * u + 2 * g + q) ^ r));
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (2 * s + u < kb) {  // uniform in the wave
          const float scale = sc[h][u] * ws[2 * s + u];
          const v4f p = mfma_f8(w[u][0], w[u][1], x[h][u][0], x[h][u][1]);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(p[i], scale, acc[i]);
        }
      }
      __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the slice has been read before its slot is refilled
      asm volatile("" ::: "memory");
      if (j + kRing < mine) fetch(j + kRing);
    }
  }

  // The partial sums meet in the order of the waves.
  *reinterpret_cast<v4f*>(area + lane * 16) = acc;
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int w = 1; w < kWaves; ++w) acc += *reinterpret_cast<const v4f*>(lds + w * area_bytes + lane * 16);
  store4(Y, M, N, r, nb + 4 * g, acc);
}

hipError_t launch(const uint8_t* Xq, const float* Xs, const uint8_t* Wq, const float* Ws, int M, int N, int K, uint16_t* Y,
                  int dev, hipStream_t st) {
  static std::atomic<int> ready[64];
  constexpr int lds = kWaves * kRing * kSliceBytes;
  const bool cached = dev >= 0 && dev < 64;
  if (!cached || !ready[dev].load(std::memory_order_acquire)) {
    const hipError_t e = hipFuncSetAttribute((const void*)gemm_fp8_decode, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
    if (cached) ready[dev].store(1, std::memory_order_release);
  }
  hipLaunchKernelGGL(gemm_fp8_decode, dim3((unsigned)((N + 15) / 16)), dim3(kWaves * 64), lds, st, Xq, Xs, Wq, Ws, Y, M, N, K);
  return hipGetLastError();
}

}  // namespace
}  // namespace fp4

// Up to 16 rows go to this kernel where it has at most one workgroup a CU, or where rows times workgroups stay
// below 8 a CU: every workgroup reads all of X, in a pattern that costs the cache four times what a tile's DMA does (16
// rows of 64 bytes an instruction). Against the 64 x 64 or 32 x 32 tiles, K = 4096: 16 x 4096 7.0 against 8.7 us, 4 x
// 14336 13.0 against 12.1, 16 x 14336 17.8 against 12.3; K = 8192: 4 x 8192 14.0 against 14.9, 16 x 8192 19.0 against 15.2.
hipError_t fp8_launch_linear(const uint8_t* Xq, const float* Xs, const uint8_t* Wq, const float* Ws, int64_t M,
                             int64_t N, int64_t K, uint16_t* Y, hipStream_t st) {
  int dev = 0, cus = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e == hipSuccess) e = fp4_device_cus(dev, &cus);
  if (e != hipSuccess) return e;
  const int64_t tiles = (N + 15) / 16;
  if (M <= 16 && (tiles <= cus || M * tiles <= 8 * (int64_t)cus))
    return fp4::launch(Xq, Xs, Wq, Ws, (int)M, (int)N, (int)K, Y, dev, st);
  return fp8_launch_linear_ring(Xq, Xs, Wq, Ws, M, N, K, Y, dev, cus, st);
}
