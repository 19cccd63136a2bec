// Blockwise-scaled E4M3 GEMM on small tiles, K split over the waves of a workgroup (gfx950): Y[m, n] = sum over blocks b
// of 128 along K of xs[m, b] * ws[n / 128, b] * sum over k in b of xq[m, k] * wq[n, k].
//
// Where the output has few tiles, a workgroup that walks K a stage at a time is bound by the latency of its stages, and
// few rows of X need all of W from HBM. So:
//  * A workgroup of four waves takes a tile of 16 or 32 rows of X by 16 or 32 of W; block b of K goes to wave b % 4,
//    which streams its blocks of X, W and their scales through its own LDS ring with the LDS DMA (one instruction: 8 rows
//    x 128 bytes; 16-byte chunks XOR-swizzled by the row, so that fragment reads hit distinct banks). No barrier stands
//    between a wave's data and its products, and with two to four workgroups on a CU 100 KB and more are in flight.
//  * v_mfma_f32_16x16x128_f8f6f4 with W as the row operand and X as the column operand: one instruction is one block,
//    and its result gives each lane 4 features of ONE token: acc += p * (xs * ws) is four float32 FMAs.
//  * The waves' float32 sums meet once, through LDS, in the order of the waves: the result does not depend on timing.
//  * Rows past M and N read as zero and are not stored.
// Bound by W's bytes from HBM where N is large (K = 4096, N = 14336: 1 row 10.7 us, 16 rows 10.6, 58.7 MB, 5.5 TB/s, and 10.1 a
// call among others; K = 8192, N = 28672: 1 row 40.5 us, 5.8 TB/s), by what a CU reads from L2 and by latency where it is small (K = 4096, N =
// 4096: 1 row 4.9 us, 64 rows 6.5 us; 37 x 4100 7.2 us (6.6 among others), and 12.1 through 32 x 32 tiles of the ring, a stage at
// a time). Eight waves a tile 5.3, 16 waves 5.7 us at 16 x 4096 (four 5.2); three slots a wave no faster.
#include <atomic>

#include "fp8_device.hpp"

namespace fp4 {
namespace {

typedef __attribute__((address_space(3))) void lds_void;
typedef const __attribute__((address_space(1))) void global_void;

constexpr int BKB = 128;    // bytes of K per row and block: one scale block
constexpr int WAVES = 4;
constexpr int SLOTS = 2;    // blocks a wave holds or has in flight

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_rsrc(const void* base, unsigned bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00020000);
}

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 0xF) | (0x7 << 4) | (0xF << 8) | (((N >> 4) & 3) << 14));
}

// 16 MF rows of X by 16 NF of W.
template <int MF, int NF>
struct Split {
  static constexpr int BM = 16 * MF, BN = 16 * NF, LOADS = 2 * (MF + NF) + 1;
  static constexpr int SLOT = (BM + BN) * BKB + 256, AREA = SLOTS * SLOT, LDS = WAVES * AREA;
  static_assert(BM < 64, "one load takes the scales of X's rows and W's");
  static_assert(128 % BN == 0, "a tile's features share a scale block");
  static_assert(MF * NF * 1024 <= AREA, "the sums meet in the ring");
};

template <int MF, int NF>
__device__ __forceinline__ void split_tile(uint8_t* smem, const uint8_t* __restrict__ Xq, const float* __restrict__ Xs,
                                           const uint8_t* __restrict__ Wq, const float* __restrict__ Ws,
                                           uint16_t* __restrict__ Y, int M, int N, int K, int m0, int n0) {
  using C = Split<MF, NF>;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4, kb = K / BKB;
  const int mine = kb > wave ? (kb - wave + WAVES - 1) / WAVES : 0;  // this wave's blocks
  uint8_t* area = smem + wave * C::AREA;
  const __amdgpu_buffer_rsrc_t rx = buffer_rsrc(Xq + (size_t)m0 * K, (unsigned)min(C::BM, M - m0) * (unsigned)K);
  const __amdgpu_buffer_rsrc_t rw = buffer_rsrc(Wq + (size_t)n0 * K, (unsigned)min(C::BN, N - n0) * (unsigned)K);
  // lanes 0 .. BM - 1 fetch the scales of X's rows, the others W's
  const float* sp = lane < C::BM ? Xs + (size_t)(m0 + min(lane, M - 1 - m0)) * kb : Ws + (size_t)(n0 / 128) * kb;
  const unsigned at = (unsigned)(lane >> 3) * (unsigned)K + 16u * (unsigned)((lane & 7) ^ (lane >> 3));
  auto fetch = [&](int j, int slot) {
    const int b = wave + WAVES * j;
    uint8_t* to = area + slot * C::SLOT;
#pragma unroll
    for (int i = 0; i < 2 * NF; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)(to + C::BM * BKB + i * 1024), 16, at + (unsigned)b * BKB + 8u * i * (unsigned)K, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 2 * MF; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_void*)(to + i * 1024), 16, at + (unsigned)b * BKB + 8u * i * (unsigned)K, 0, 0, 0);
    __builtin_amdgcn_global_load_lds((global_void*)(sp + b),
                                     (lds_void*)(to + (C::BM + C::BN) * BKB), 4, 0, 0);
  };
  v4f acc[NF][MF];
#pragma unroll
  for (int i = 0; i < NF; ++i)
#pragma unroll
    for (int f = 0; f < MF; ++f) acc[i][f] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < SLOTS; ++j)
    if (j < mine) fetch(j, j);
  for (int j = 0, slot = 0; j < mine; ++j, slot = slot + 1 == SLOTS ? 0 : slot + 1) {
    // the block has landed: at most those after it are in flight
    if (j + SLOTS - 1 < mine) wait_vmcnt<(SLOTS - 1) * C::LOADS>();
    else wait_vmcnt<0>();
    asm volatile("" ::: "memory");
    const uint8_t* from = area + slot * C::SLOT;
    v4u x[MF][2], w[NF][2];
    float s[MF];
    const float* sl = reinterpret_cast<const float*>(from + (C::BM + C::BN) * BKB);
#pragma unroll
    for (int f = 0; f < MF; ++f) {
      s[f] = sl[16 * f + r] * sl[C::BM];
#pragma unroll
      for (int q = 0; q < 2; ++q)
        x[f][q] = *reinterpret_cast<const v4u*>(from + (16 * f + r) * BKB + 16 * ((4 * q + g) ^ (r & 7)));
    }
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
      for (int q = 0; q < 2; ++q)
        w[i][q] = *reinterpret_cast<const v4u*>(from + (C::BM + 16 * i + r) * BKB + 16 * ((4 * q + g) ^ (r & 7)));
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the block has been read before its slot is refilled
    asm volatile("" ::: "memory");
    if (j + SLOTS < mine) fetch(j + SLOTS, slot);
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
      for (int f = 0; f < MF; ++f) {
        const v8i a = {(int)w[i][0][0], (int)w[i][0][1], (int)w[i][0][2], (int)w[i][0][3],
                       (int)w[i][1][0], (int)w[i][1][1], (int)w[i][1][2], (int)w[i][1][3]};
        const v8i b = {(int)x[f][0][0], (int)x[f][0][1], (int)x[f][0][2], (int)x[f][0][3],
                       (int)x[f][1][0], (int)x[f][1][1], (int)x[f][1][2], (int)x[f][1][3]};
        const v4f p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[i][f][q] = __builtin_fmaf(p[q], s[f], acc[i][f][q]);
      }
  }
  // The partial sums meet in the order of the waves.
#pragma unroll
  for (int i = 0; i < NF; ++i)
#pragma unroll
    for (int f = 0; f < MF; ++f) *reinterpret_cast<v4f*>(area + (i * MF + f) * 1024 + lane * 16) = acc[i][f];
  __syncthreads();
  for (int q = wave; q < MF * NF; q += WAVES) {
    const uint8_t* p = smem + q * 1024 + lane * 16;
    v4f v = *reinterpret_cast<const v4f*>(p);
#pragma unroll
    for (int w = 1; w < WAVES; ++w) v += *reinterpret_cast<const v4f*>(p + w * C::AREA);
    const int m = m0 + 16 * (q % MF) + r, n = n0 + 16 * (q / MF) + 4 * g;
    if (m >= M) continue;
    uint16_t* dst = Y + (size_t)m * N + n;
    uint16_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = __builtin_bit_cast(uint16_t, (__bf16)v[e]);
    if (n + 3 < N) {
      *reinterpret_cast<v2u_any*>(dst) = v2u{o[0] | ((unsigned)o[1] << 16), o[2] | ((unsigned)o[3] << 16)};
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < N) dst[e] = o[e];
    }
  }
}

template <int MF, int NF>
__global__ __launch_bounds__(64 * WAVES) void gemm_fp8_split(const uint8_t* __restrict__ Xq, const float* __restrict__ Xs,
                                                             const uint8_t* __restrict__ Wq,
                                                             const float* __restrict__ Ws, uint16_t* __restrict__ Y,
                                                             int M, int N, int K, int tiles_m, unsigned T) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  // workgroup i runs on XCD i % 8; each takes a contiguous range of tiles, X's fastest, so that tiles of the same W
  // share it in that XCD's L2
  const unsigned b = blockIdx.y * gridDim.x + blockIdx.x, xcd = b & 7;
  if (b >= T) return;
  const unsigned L = xcd * (T >> 3) + min(xcd, T & 7) + (b >> 3);
  split_tile<MF, NF>(smem, Xq, Xs, Wq, Ws, Y, M, N, K, (int)(L % tiles_m) * 16 * MF, (int)(L / tiles_m) * 16 * NF);
}

template <int MF, int NF>
hipError_t launch(const uint8_t* Xq, const float* Xs, const uint8_t* Wq, const float* Ws, int M, int N, int K,
                        uint16_t* Y, int dev, hipStream_t st) {
  using C = Split<MF, NF>;
  static std::atomic<int> ready[64];
  auto kern = gemm_fp8_split<MF, NF>;
  const bool cached = dev >= 0 && dev < 64;
  if (!cached || !ready[dev].load(std::memory_order_acquire)) {
    const hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, C::LDS);
    if (e != hipSuccess) return e;
    if (cached) ready[dev].store(1, std::memory_order_release);
  }
  const int tiles_m = (M - 1) / C::BM + 1, tiles_n = (N - 1) / C::BN + 1;
  const Grid grid = grid_of((int64_t)tiles_m * tiles_n, 64 * WAVES);
  hipLaunchKernelGGL(kern, dim3(grid.x, grid.y), dim3(64 * WAVES), C::LDS, st, Xq, Xs, Wq, Ws, Y, M, N, K, tiles_m,
                     (unsigned)(tiles_m * tiles_n));
  return hipGetLastError();
}

}  // namespace
}  // namespace fp4

// Tiles of bm x bn (16 x 16, 16 x 32 or 32 x 32), chosen by fp8_launch_linear.
hipError_t fp8_launch_linear_split(int bm, int bn, const uint8_t* Xq, const float* Xs, const uint8_t* Wq, const float* Ws,
                                   int64_t M, int64_t N, int64_t K, uint16_t* Y, int dev, hipStream_t st) {
  const int m = (int)M, n = (int)N, k = (int)K;
  if (bm == 32) return fp4::launch<2, 2>(Xq, Xs, Wq, Ws, m, n, k, Y, dev, st);
  if (bn == 32) return fp4::launch<1, 2>(Xq, Xs, Wq, Ws, m, n, k, Y, dev, st);
  return fp4::launch<1, 1>(Xq, Xs, Wq, Ws, m, n, k, Y, dev, st);
}
