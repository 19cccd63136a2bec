// Large-tile blockwise-scaled E4M3 GEMM (gfx950): Y[m, n] = sum over blocks b of 128 along K of
// xs[m, b] * ws[n / 128, b] * sum over k in b of xq[m, k] * wq[n, k].
//
//  * One v_mfma_f32_16x16x128_f8f6f4 is one scale block: its 16x16 result p starts from zero and enters
//    the accumulators as acc += p * (xs * ws), four float32 FMAs. W is the row operand and X the column
//    operand, so a lane's four values belong to ONE token and the block's scale is one value per lane and
//    16 tokens. The matrix pipe alone sustains 4.0 PFLOP/s on random E4M3 data (power-limited; 16x16x128
//    and 32x32x64 alike), 3.5 with these FMAs beside it; 32x32x64, which takes two instructions and 16
//    FMAs a block, 3.3.
//  * K advances one block (128 bytes of a row) per stage. The stages live in an LDS ring filled with
//    buffer_load ... lds (no register staging), 16-byte chunks XOR-swizzled by the row so the 16 rows
//    of a fragment read hit distinct banks; X's scales of the stage come the same way, 4 bytes a row. W's
//    scales are one number per stage and 128 features: lane l holds those of stages 64 i + l, and a
//    stage's comes from v_readlane.
//  * The barrier of the ring waits for LDS reads only, so the DMA of the next stage stays in flight.
//  * Output tiles go through LDS as bf16, so Y is written as whole row segments.
//  * Workgroup i runs on XCD i % 8; each XCD takes a contiguous range of tiles, M fastest within groups
//    of 8 tile rows, so tiles running together share X and W in that XCD's L2.
#include <atomic>
#include <type_traits>

#include "fp8_device.hpp"

namespace fp4 {
namespace {

typedef __attribute__((address_space(3))) void lds_void;

constexpr int WAVES = 8, NT = WAVES * 64;
constexpr int BKB = 128;  // bytes of K per row and stage: one scale block

// BM rows of X by BN rows of W, WGM x WGN waves, an NS-deep ring.
template <int BM_, int BN_, int WGM_, int WGN_, int NS_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WGM = WGM_, WGN = WGN_, NS = NS_;
  static constexpr int WM = BM / WGM, WN = BN / WGN, FM = WM / 16, FN = WN / 16;
  static constexpr int A_WL = BM / 8 / WAVES, B_WL = BN / 8 / WAVES;  // 1 KB DMA wave-loads per wave
  static constexpr int SC_LOADS = BM / 64;                             // 64-row loads of X's scales
  static constexpr int STAGE = (BM + BN) * BKB + BM * 4;
  static constexpr int RING = NS * STAGE;
  static constexpr int EP = WN * 2 + 16;                               // epilogue row pitch (bytes)
  static constexpr int LDS = RING > WAVES * WM * EP ? RING : WAVES * WM * EP;
  static_assert(WGM * WGN == WAVES && WM % 16 == 0 && WN % 16 == 0, "whole fragments");
  static_assert(A_WL * 8 * WAVES == BM && B_WL * 8 * WAVES == BN, "whole wave-loads");
  static_assert(SC_LOADS >= 1 && SC_LOADS <= WAVES, "at most one scale load per wave");
  static_assert(128 % WN == 0 && BN % 64 == 0, "a wave's features share a scale block");
  static_assert(NS >= 2 && LDS <= 160 * 1024, "the ring fits");
};
using T256 = Tile<256, 256, 4, 2, 2>;
using T128 = Tile<128, 128, 4, 2, 2>;
using T64 = Tile<128, 64, 4, 2, 3>;

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 0xF) | (0x7 << 4) | (0xF << 8) | (((N >> 4) & 3) << 14));
}

// Barrier of the LDS ring: wait for this wave's LDS reads (lgkmcnt(0)) but not for its DMA in flight.
__device__ __forceinline__ void ring_barrier() {
  __builtin_amdgcn_s_waitcnt(0xC07F);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_rsrc(const void* base, unsigned bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00020000);
}

// 16-byte chunk q of row r sits at slot q ^ swz(r), which depends on r % 16 only: over 16 consecutive rows each slot is taken twice,
// once on even and once on odd rows.
__device__ __forceinline__ int swz(int r) { return (r ^ ((r >> 3) & 1)) & 7; }

__device__ __forceinline__ v4f mfma_f8(v4u a0, v4u a1, v4u b0, v4u b1) {
  const v8i a = {(int)a0[0], (int)a0[1], (int)a0[2], (int)a0[3], (int)a1[0], (int)a1[1], (int)a1[2], (int)a1[3]};
  const v8i b = {(int)b0[0], (int)b0[1], (int)b0[2], (int)b0[3], (int)b1[0], (int)b1[1], (int)b1[2], (int)b1[3]};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

// One output tile [m0, m0 + BM) x [n0, n0 + BN) over all of K.
template <class C>
__device__ __forceinline__ void ring_tile(uint8_t* smem, const uint8_t* __restrict__ Xq, const float* __restrict__ Xs,
                                          const uint8_t* __restrict__ Wq, const float* __restrict__ Ws,
                                          uint16_t* __restrict__ Y, int M, int N, int K, int m0, int n0) {
  constexpr int BM = C::BM, WM = C::WM, WN = C::WN, FM = C::FM, FN = C::FN, A_WL = C::A_WL, B_WL = C::B_WL;
  constexpr int NS = C::NS, D = NS - 1;  // D: stages fetched ahead
  constexpr int A_ST = BM * BKB, B_ST = C::BN * BKB, B_BASE = NS * A_ST, S_BASE = B_BASE + NS * B_ST;
  auto slot = [](int s) { return NS == 2 ? (s & 1) : (int)((unsigned)s % NS); };
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm0 = (wave / C::WGN) * WM, wn0 = (wave % C::WGN) * WN;
  const int nst = K / BKB;

  // DMA sources: 8 rows x 128 bytes per wave-load; rows past M / N repeat the last one. 32-bit offsets
  // below BM * K <= 2^31 (K <= 2^23).
  const int rows_a = min(M - m0, BM), rows_b = min(N - n0, C::BN);
  const __amdgpu_buffer_rsrc_t rsA = buffer_rsrc(Xq + (size_t)m0 * K, (unsigned)rows_a * (unsigned)K);
  const __amdgpu_buffer_rsrc_t rsB = buffer_rsrc(Wq + (size_t)n0 * K, (unsigned)rows_b * (unsigned)K);
  const __amdgpu_buffer_rsrc_t rsS = buffer_rsrc(Xs + (size_t)m0 * nst, (unsigned)rows_a * (unsigned)nst * 4u);
  unsigned offA[A_WL], offB[B_WL];
#pragma unroll
  for (int i = 0; i < A_WL; ++i) {
    const int r = (wave * A_WL + i) * 8 + (lane >> 3), q = lane & 7;
    offA[i] = (unsigned)min(r, rows_a - 1) * (unsigned)K + ((q ^ swz(r)) << 4);
  }
#pragma unroll
  for (int i = 0; i < B_WL; ++i) {
    const int r = (wave * B_WL + i) * 8 + (lane >> 3), q = lane & 7;
    offB[i] = (unsigned)min(r, rows_b - 1) * (unsigned)K + ((q ^ swz(r)) << 4);
  }
  const unsigned offS = (unsigned)min(wave * 64 + lane, rows_a - 1) * (unsigned)nst * 4u;

  constexpr int PARTS = 4;  // of a stage's DMA, issued over the stage before it
  auto issue_part = [&](int s, int p) {
    uint8_t* bufa = smem + slot(s) * A_ST;
    uint8_t* bufb = smem + B_BASE + slot(s) * B_ST;
#pragma unroll
    for (int i = 0; i < A_WL; ++i)
      if (i % PARTS == p)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsA, (lds_void*)(bufa + (wave * A_WL + i) * 1024), 16, offA[i],
                                                 (unsigned)s * BKB, 0, 0);
#pragma unroll
    for (int i = 0; i < B_WL; ++i)
      if (i % PARTS == p)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsB, (lds_void*)(bufb + (wave * B_WL + i) * 1024), 16, offB[i],
                                                 (unsigned)s * BKB, 0, 0);
    if (p == 0 && wave < C::SC_LOADS)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsS, (lds_void*)(smem + S_BASE + slot(s) * BM * 4 + wave * 256), 4, offS,
                                               (unsigned)s * 4, 0, 0);
  };

  // W's scales: the row of the wave's features (WN divides 128, so they share one)
  const float* wsp = Ws + (size_t)(min(n0 + wn0, N - 1) / kF8Group) * nst;
  float wsl = 0.f;

  v4f acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  const int fr = lane & 15, g = lane >> 4;
  // lane group g takes chunks g and g + 4 of its row, of both operands
  const int c0 = (g ^ swz(fr)) << 4, c1 = ((g + 4) ^ swz(fr)) << 4;

  auto wait_stage = [&](auto with_dma) {
    if constexpr (!decltype(with_dma)::value || D == 1) {
      wait_vmcnt<0>();
    } else {  // stages s + 1 .. s + D - 1 may be in flight
      if (wave < C::SC_LOADS) wait_vmcnt<(D - 1) * (A_WL + B_WL + 1)>();
      else wait_vmcnt<(D - 1) * (A_WL + B_WL)>();
    }
  };
  auto run_stage = [&](int s, auto with_dma) {
    wait_stage(with_dma);
    ring_barrier();
    if ((s & 63) == 0) wsl = wsp[min(s + lane, nst - 1)];
    const uint8_t* pa = smem + slot(s) * A_ST + (wm0 + fr) * BKB;
    const uint8_t* pb = smem + B_BASE + slot(s) * B_ST + (wn0 + fr) * BKB;
    const float* ps = reinterpret_cast<const float*>(smem + S_BASE + slot(s) * BM * 4) + wm0 + fr;
    v4u x0[FM], x1[FM];
    float sc[FM];
    const float sw = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(wsl), s & 63));
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      x0[j] = *reinterpret_cast<const v4u*>(pa + j * 16 * BKB + c0);
      x1[j] = *reinterpret_cast<const v4u*>(pa + j * 16 * BKB + c1);
      sc[j] = ps[j * 16] * sw;
    }
#pragma unroll
    for (int i = 0; i < FN; ++i) {
      if constexpr (decltype(with_dma)::value) {
        if constexpr (FN >= PARTS) {
          if (i % (FN / PARTS) == 0) issue_part(s + D, i / (FN / PARTS));
        } else {
#pragma unroll
          for (int p = 0; p < PARTS / FN; ++p) issue_part(s + D, i * (PARTS / FN) + p);
        }
      }
      const v4u w0 = *reinterpret_cast<const v4u*>(pb + i * 16 * BKB + c0);
      const v4u w1 = *reinterpret_cast<const v4u*>(pb + i * 16 * BKB + c1);
      v4f p[FM];
#pragma unroll
      for (int j = 0; j < FM; ++j) p[j] = mfma_f8(w0, w1, x0[j], x1[j]);
#pragma unroll
      for (int j = 0; j < FM; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[i][j][q] = __builtin_fmaf(p[j][q], sc[j], acc[i][j][q]);
    }
  };
  for (int t = 0; t < D && t < nst; ++t)
#pragma unroll
    for (int p = 0; p < PARTS; ++p) issue_part(t, p);
  int s = 0;
  for (; s + D < nst; ++s) run_stage(s, std::true_type{});
  for (; s < nst; ++s) run_stage(s, std::false_type{});

  // Epilogue: each wave stages its WM x WN outputs as bf16 in its own LDS region, then writes whole
  // 16-byte pieces of rows.
  constexpr int EP = C::EP, CPR = WN / 8;
  __syncthreads();  // every wave is done with the ring
  uint8_t* ep = smem + wave * WM * EP;
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      unsigned b[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) b[q] = __builtin_bit_cast(uint16_t, (__bf16)acc[i][j][q]);
      *reinterpret_cast<v2u*>(ep + (j * 16 + fr) * EP + (i * 16 + 4 * g) * 2) = v2u{b[0] | b[1] << 16, b[2] | b[3] << 16};
    }
  __builtin_amdgcn_s_waitcnt(0xC07F);  // the wave's own region: no barrier
  asm volatile("" ::: "memory");
  const bool vec = N % 8 == 0;  // every piece of Y starts 16-byte aligned
#pragma unroll
  for (int k = 0; k < WM * CPR / 64; ++k) {
    const int at = k * 64 + lane, rr = at / CPR, cc = at % CPR;
    const v4u v = *reinterpret_cast<const v4u*>(ep + rr * EP + cc * 16);
    const int row = m0 + wm0 + rr, col = n0 + wn0 + cc * 8;
    if (row >= M) continue;
    uint16_t* dst = Y + (size_t)row * N + col;
    if (vec && col + 8 <= N) {
      __builtin_nontemporal_store(v, reinterpret_cast<v4u*>(dst));
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (col + q < N) dst[q] = (uint16_t)(v[q >> 1] >> (16 * (q & 1)));
    }
  }
}

// Tile index L of a tiles_m x tiles_n grid -> (tm, tn): groups of 8 tile rows, M fastest.
__device__ __forceinline__ void map_tile(int L, int tiles_m, int tiles_n, int& tm, int& tn) {
  constexpr int GM = 8;
  const int first_m = (L / (GM * tiles_n)) * GM;
  const int gsize = min(tiles_m - first_m, GM);
  const int in = L % (GM * tiles_n);
  tm = first_m + in % gsize;
  tn = in / gsize;
}

template <class C>
__global__ __launch_bounds__(NT) void gemm_fp8_ring(const uint8_t* __restrict__ Xq, const float* __restrict__ Xs,
                                                    const uint8_t* __restrict__ Wq, const float* __restrict__ Ws,
                                                    uint16_t* __restrict__ Y, int M, int N, int K, int tiles_m,
                                                    int tiles_n) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  const int T = tiles_m * tiles_n, b = blockIdx.x;
  const int L = T % 8 == 0 ? (b & 7) * (T >> 3) + (b >> 3) : b;
  int tm, tn;
  map_tile(L, tiles_m, tiles_n, tm, tn);
  ring_tile<C>(smem, Xq, Xs, Wq, Ws, Y, M, N, K, tm * C::BM, tn * C::BN);
}

template <class C>
hipError_t launch(const uint8_t* Xq, const float* Xs, const uint8_t* Wq, const float* Ws, int M, int N, int K,
                  uint16_t* Y, int dev, hipStream_t st) {
  static std::atomic<int> ready[64];
  auto kern = gemm_fp8_ring<C>;
  const bool cached = dev >= 0 && dev < 64;
  if (!cached || !ready[dev].load(std::memory_order_acquire)) {
    const hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, C::LDS);
    if (e != hipSuccess) return e;
    if (cached) ready[dev].store(1, std::memory_order_release);
  }
  const int tiles_m = (M + C::BM - 1) / C::BM, tiles_n = (N + C::BN - 1) / C::BN;
  hipLaunchKernelGGL(kern, dim3((unsigned)(tiles_m * tiles_n)), dim3(NT), C::LDS, st, Xq, Xs, Wq, Ws, Y, M, N, K,
                     tiles_m, tiles_n);
  return hipGetLastError();
}

}  // namespace
}  // namespace fp4

hipError_t fp8_launch_linear_ring(const uint8_t* Xq, const float* Xs, const uint8_t* Wq, const float* Ws, int64_t M,
                                  int64_t N, int64_t K, uint16_t* Y, hipStream_t st) {
  int dev = 0, cus = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e == hipSuccess) e = fp4_device_cus(dev, &cus);
  if (e != hipSuccess) return e;
  auto tiles = [&](int64_t bm, int64_t bn) { return ((M + bm - 1) / bm) * ((N + bn - 1) / bn); };
  const int m = (int)M, n = (int)N, k = (int)K;
  if (tiles(256, 256) >= cus) return fp4::launch<fp4::T256>(Xq, Xs, Wq, Ws, m, n, k, Y, dev, st);
  if (tiles(128, 128) >= cus) return fp4::launch<fp4::T128>(Xq, Xs, Wq, Ws, m, n, k, Y, dev, st);
  return fp4::launch<fp4::T64>(Xq, Xs, Wq, Ws, m, n, k, Y, dev, st);
}
