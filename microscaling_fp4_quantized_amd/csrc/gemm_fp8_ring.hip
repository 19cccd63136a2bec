// Large-tile blockwise-scaled E4M3 GEMM (gfx950): Y[m, n] = sum over blocks b of 128 along K of
// xs[m, b] * ws[n / 128, b] * sum over k in b of xq[m, k] * wq[n, k].
//
//  * One v_mfma_f32_16x16x128_f8f6f4 is one scale block: its 16x16 result p starts from zero and enters
//    the accumulators as acc += p * (xs * ws), four float32 FMAs. W is the row operand and X the column
//    operand, so a lane's four values belong to ONE token and the block's scale is one value per lane and
//    16 tokens. The matrix pipe alone sustains 4.0 PFLOP/s on random E4M3 data (power-limited; 16x16x128
//    and 32x32x64 alike), 3.5 with these FMAs beside it; 32x32x64, which takes two instructions and 16
//    FMAs a block, 3.3.
//  * K advances in stages of one to four blocks (128 bytes of a row each). The stages live in an LDS ring filled with
//    buffer_load ... lds (no register staging), 16-byte chunks XOR-swizzled by the row so the 16 rows
//    of a fragment read hit distinct banks; X's scales of a block come the same way, 4 bytes a row. W's
//    scales are one number per block and 128 features: lane l holds those of blocks 64 i + l, and a
//    block's comes from v_readlane.
//  * The barrier of the ring waits for LDS reads only, so the DMA of the next stage stays in flight.
//  * Output tiles go through LDS as bf16, so Y is written as whole row segments, in 16-byte pieces also where N is no
//    multiple of 8 (2048 x 14340, K = 4096: 126 us, 155 in elements of two bytes; 2048 x 14336 113-115 beside them).
//  * Workgroup i runs on XCD i % 8; each XCD takes a contiguous range of tiles, M fastest within groups
//    of 4 tile rows, so tiles running together share X and W in that XCD's L2.
//
// Measured, us of a call among others: 2048 x 14336, K = 4096: 104 (2.31 PFLOP/s); 8192 x 28672, K = 8192: 1533 (2.51
// PFLOP/s; the library's product with ONE scale for each operand, so without the FMAs, 1185, and 97 at the first size).
#include <atomic>
#include <type_traits>

#include "fp8_device.hpp"

namespace fp4 {
namespace {

typedef __attribute__((address_space(3))) void lds_void;

constexpr int BKB = 128;  // bytes of K per row and stage: one scale block

// BM rows of X by BN rows of W, WGM x WGN waves, an NS-deep ring of stages of KB scale blocks (128 bytes of a row
// each; the workgroup meets at a barrier once per stage).
template <int BM_, int BN_, int WGM_, int WGN_, int NS_, int KB_ = 1>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WGM = WGM_, WGN = WGN_, NS = NS_, KB = KB_, WAVES = WGM_ * WGN_, NT = 64 * WAVES;
  static constexpr int WM = BM / WGM, WN = BN / WGN, FM = WM / 16, FN = WN / 16;
  static constexpr int A_WL = BM / 8 / WAVES, B_WL = BN / 8 / WAVES;  // 1 KB DMA wave-loads per wave
  static constexpr int SC_LOADS = (BM + 63) / 64;                      // 64-row loads of X's scales
  static constexpr int BLOCK = (BM + BN) * BKB + SC_LOADS * 256;       // LDS of one scale block
  static constexpr int RING = NS * KB * BLOCK;
  static constexpr int EP = WN * 2 + 16;                               // epilogue row pitch (bytes)
  static constexpr int LDS = RING > WAVES * WM * EP ? RING : WAVES * WM * EP;
  static_assert(WM % 16 == 0 && WN % 16 == 0, "whole fragments");
  static_assert(A_WL * 8 * WAVES == BM && B_WL * 8 * WAVES == BN, "whole wave-loads");
  static_assert(SC_LOADS >= 1 && SC_LOADS <= WAVES, "at most one scale load per wave");
  static_assert(128 % WN == 0 && (128 % BN == 0 || BN % 128 == 0), "a wave's features share a scale block");
  static_assert((NS - 2) * KB * (A_WL + B_WL + 1) < 64, "the ring's loads in flight can be counted");
  static_assert(NS >= 2 && LDS <= 160 * 1024, "the ring fits");
};
using T64 = Tile<64, 64, 4, 2, 4, 2>;
using T128x64 = Tile<128, 64, 4, 2, 3, 2>;
using T128 = Tile<128, 128, 4, 2, 2, 2>;     // one workgroup on a CU
using T128Two = Tile<128, 128, 4, 2, 2, 1>;  // two

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

// 16-byte chunk q of row r sits at slot q ^ swz(r). ds_read_b128 serves lanes 0-3, 12-15 and 20-27 together (then 4-11,
// 16-19, 28-31, and the same of the upper half), over 64 banks: with the rows on lanes % 16 and the chunk by lane
// group, each of those 16 lanes gets its own four banks (4.0 cycles an instruction measured; a swizzle made for
// consecutive lanes, 6.4).
__device__ __forceinline__ int swz(int r) { return r & 7; }

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
  constexpr int KB = C::KB, D = C::NS - 1, SLOTS = C::NS * KB;  // D: stages fetched ahead; a slot holds a block
  constexpr int A_ST = BM * BKB, B_ST = C::BN * BKB, S_ST = C::SC_LOADS * 256;
  constexpr int B_BASE = SLOTS * A_ST, S_BASE = B_BASE + SLOTS * B_ST;
  auto slot = [](int b) { return (SLOTS & (SLOTS - 1)) == 0 ? (b & (SLOTS - 1)) : (int)((unsigned)b % SLOTS); };
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm0 = (wave / C::WGN) * WM, wn0 = (wave % C::WGN) * WN;
  const int nst = K / BKB, nsup = (nst + KB - 1) / KB;  // blocks and stages

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

  constexpr int PARTS = 4;  // of a block's DMA, issued over the block D stages before it
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
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsS, (lds_void*)(smem + S_BASE + slot(s) * S_ST + wave * 256), 4, offS,
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
      if (wave < C::SC_LOADS) wait_vmcnt<(D - 1) * KB * (A_WL + B_WL + 1)>();
      else wait_vmcnt<(D - 1) * KB * (A_WL + B_WL)>();
    }
  };
  // Block s (of X and W along K); with_dma: the block D stages on is requested meanwhile, if there is one.
  auto run_block = [&](int s, auto with_dma) {
    const int ahead = s + D * KB;
    if ((s & 63) == 0) {
      wsl = wsp[min(s + lane, nst - 1)];
      asm volatile("" : "+v"(wsl));  // wait for it here, or every block waits for the DMA in flight at its use
    }
    const uint8_t* pa = smem + slot(s) * A_ST + (wm0 + fr) * BKB;
    const uint8_t* pb = smem + B_BASE + slot(s) * B_ST + (wn0 + fr) * BKB;
    const float* ps = reinterpret_cast<const float*>(smem + S_BASE + slot(s) * S_ST) + wm0 + fr;
    v4u x0[FM], x1[FM];
    float sc[FM];
    const float sw = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(wsl), s & 63));
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      x0[j] = *reinterpret_cast<const v4u*>(pa + j * 16 * BKB + c0);
      x1[j] = *reinterpret_cast<const v4u*>(pa + j * 16 * BKB + c1);
      sc[j] = ps[j * 16] * sw;
    }
    // The FN x FM products in order, each one's FMAs LAG products after it, so that no FMA waits for the matrix
    // pipe; W's next fragment is read, and a part of the DMA issued, at the first product of a fragment.
    constexpr int LAG = FM * FN >= 4 ? 3 : FM * FN - 1;
    v4u w0[2], w1[2];
    v4f p[LAG + 1];
    auto load_w = [&](int i) {
      w0[i & 1] = *reinterpret_cast<const v4u*>(pb + i * 16 * BKB + c0);
      w1[i & 1] = *reinterpret_cast<const v4u*>(pb + i * 16 * BKB + c1);
    };
    auto add = [&](int m) {
      const int i = m / FM, j = m % FM;
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[i][j][q] = __builtin_fmaf(p[m % (LAG + 1)][q], sc[j], acc[i][j][q]);
    };
    load_w(0);
#pragma unroll
    for (int m = 0; m < FN * FM; ++m) {
      const int i = m / FM, j = m % FM;
      if (j == 0) {
        if (i + 1 < FN) load_w(i + 1);
        if constexpr (decltype(with_dma)::value) {
          if (KB == 1 || ahead < nst) {
            if constexpr (FN >= PARTS) {
              if (i % (FN / PARTS) == 0) issue_part(ahead, i / (FN / PARTS));
            } else {
#pragma unroll
              for (int p = 0; p < PARTS / FN; ++p) issue_part(ahead, i * (PARTS / FN) + p);
            }
          }
        }
      }
      p[m % (LAG + 1)] = mfma_f8(w0[i & 1], w1[i & 1], x0[j], x1[j]);
      if (m >= LAG) add(m - LAG);
    }
#pragma unroll
    for (int m = FN * FM - LAG; m < FN * FM; ++m) add(m);
  };
  auto run_stage = [&](int s, auto with_dma) {
    wait_stage(with_dma);
    ring_barrier();
#pragma unroll
    for (int b = 0; b < KB; ++b)
      if (KB == 1 || s * KB + b < nst) run_block(s * KB + b, with_dma);
  };
  for (int t = 0; t < D * KB && t < nst; ++t)
#pragma unroll
    for (int p = 0; p < PARTS; ++p) issue_part(t, p);
  int s = 0;
  for (; s + D < nsup; ++s) run_stage(s, std::true_type{});
  for (; s < nsup; ++s) run_stage(s, std::false_type{});

  // Epilogue: each wave stages its WM x WN outputs as bf16 in its own LDS region, then writes whole
  // 16-byte pieces of rows.
  constexpr int EP = C::EP, CPR = WN / 8;
  __syncthreads();  // every wave is done with the ring
  uint8_t* ep = smem + wave * (WM * EP);
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
  for (int k = 0; k < (WM * CPR + 63) / 64; ++k) {
    const int at = k * 64 + lane, rr = at / CPR, cc = at % CPR;
    if (WM * CPR % 64 != 0 && at >= WM * CPR) break;
    const v4u v = *reinterpret_cast<const v4u*>(ep + rr * EP + cc * 16);
    const int row = m0 + wm0 + rr, col = n0 + wn0 + cc * 8;
    if (row >= M) continue;
    uint16_t* dst = Y + (size_t)row * N + col;
    if (vec && col + 8 <= N) {
      __builtin_nontemporal_store(v, reinterpret_cast<v4u*>(dst));
    } else if (col + 8 <= N) {  // pieces share lines with their neighbours: through the caches
      *reinterpret_cast<v4u_any*>(dst) = v;
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (col + q < N) dst[q] = (uint16_t)(v[q >> 1] >> (16 * (q & 1)));
    }
  }
}

// Tile index L of a tiles_m x tiles_n grid -> (tm, tn): groups of 4 tile rows, M fastest.
__device__ __forceinline__ void map_tile(int L, int tiles_m, int tiles_n, int& tm, int& tn) {
  constexpr int GM = 4;
  const int first_m = (L / (GM * tiles_n)) * GM;
  const int gsize = min(tiles_m - first_m, GM);
  const int in = L % (GM * tiles_n);
  tm = first_m + in % gsize;
  tn = in / gsize;
}

// A 256 x 256 tile in which two groups of four waves (one wave of each group per SIMD)
// take turns: group 1 runs half a stage behind group 0, so that while one group's waves read the next fragments from
// LDS and wait for them, the other group's are multiplying. In the time between two barriers group 0 reads stage s and
// multiplies it; group 1 multiplies the second half of stage s - 1, whose fragments it has in registers, then
// reads stage s and multiplies its first half. By the barrier every fragment of stage s has been read, so its
// buffer is refilled with stage s + 2 after it. Needs K >= 512.
// With all eight waves reading, then multiplying, between the same barriers (ring_tile's order): 2048 x 14336 x 4096 115 us and
// 8192 x 28672 x 8192 1780, against 106 and 1570 at that time; without any DMA the latter took 1180, without the scales' FMAs
// 1455. At the large size the matrix pipe is busy 63% of the time at 1.88 GHz, the clock that power leaves
// (profiles/gemm_fp8_turns_sq_counters.txt).
// (Covering what is left after whole rounds of tiles with 192-wide ones, so that the last round is full, changed nothing
// at 2048 x 14336: with fewer CUs at work the others' clock rises.)
constexpr int PBM = 256, PBN = 256, PWM = 64, PWN = 128, PFM = PWM / 16, PFN = PWN / 16;
constexpr int P_ST = PBM * BKB;                  // bytes of one operand's stage
constexpr int P_SC = 4 * P_ST;                   // two windows of X's scales: 16 bytes (4 stages) a row
constexpr int P_LDS = P_SC + 2 * PBM * 16;
constexpr int P_EP = PWN * 2 + 16;
static_assert(8 * PWM * P_EP <= P_LDS, "the epilogue's staging fits");

__global__ __launch_bounds__(512) void gemm_fp8_turns(const uint8_t* __restrict__ Xq, const float* __restrict__ Xs,
                                                      const uint8_t* __restrict__ Wq, const float* __restrict__ Ws,
                                                      uint16_t* __restrict__ Y, int M, int N, int K, int tiles_m,
                                                      int tiles_n) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  int tm, tn;
  {
    const int T = tiles_m * tiles_n, b = (int)(blockIdx.y * gridDim.x + blockIdx.x);
    if (b >= T) return;
    map_tile(T % 8 == 0 ? (b & 7) * (T >> 3) + (b >> 3) : b, tiles_m, tiles_n, tm, tn);
  }
  const int m0 = tm * PBM, n0 = tn * PBN;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  // group wave / 4; the four waves of a group and of both groups cover 4 x 2 wave tiles
  const int wm0 = (wave >> 1) * PWM, wn0 = (wave & 1) * PWN;
  const int nst = K / BKB;

  // DMA: wave-load i of a wave carries rows (4 wave + i) * 8 .. + 7 of an operand; rows past M / N read as zero.
  const int rows_a = min(M - m0, PBM), rows_b = min(N - n0, PBN);
  const __amdgpu_buffer_rsrc_t rsA = buffer_rsrc(Xq + (size_t)m0 * K, (unsigned)rows_a * (unsigned)K);
  const __amdgpu_buffer_rsrc_t rsB = buffer_rsrc(Wq + (size_t)n0 * K, (unsigned)rows_b * (unsigned)K);
  const __amdgpu_buffer_rsrc_t rsS = buffer_rsrc(Xs + (size_t)m0 * nst, (unsigned)rows_a * (unsigned)nst * 4u);
  const unsigned off = (unsigned)(wave * 32 + (lane >> 3)) * (unsigned)K + (((lane & 7) ^ swz(lane >> 3)) << 4);
  const unsigned offS = (unsigned)(wave * 64 + lane) * (unsigned)nst * 4u;
  auto window = [&](int w) { return min(4 * w, nst - 4); };  // first stage of a window of scales
  // Part p (0..3) of the DMA of stage s.
  auto issue = [&](int s, int p) {
    const unsigned at = (unsigned)s * BKB + (unsigned)p * 8u * (unsigned)K;
    uint8_t* a = smem + (s & 1) * P_ST + (wave * 4 + p) * 1024;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsA, (lds_void*)a, 16, off + at, 0, 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsB, (lds_void*)(a + 2 * P_ST), 16, off + at, 0, 0, 0);
    if (p == 0 && (s & 3) == 0 && wave < 4)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsS, (lds_void*)(smem + P_SC + ((s >> 2) & 1) * PBM * 16 + wave * 1024), 16,
                                               offS + 4u * (unsigned)window(s >> 2), 0, 0, 0);
  };

  // W's scales of the wave's 128 features; lane l holds those of stages 64 i + l.
  const float* wsp = Ws + (size_t)(min(n0 + wn0, N - 1) / kF8Group) * nst;
  float wsl = 0.f;
  v4f acc[PFN][PFM];
#pragma unroll
  for (int i = 0; i < PFN; ++i)
#pragma unroll
    for (int j = 0; j < PFM; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  const int fr = lane & 15, g = lane >> 4;
  const int c0 = (g ^ swz(fr)) << 4, c1 = ((g + 4) ^ swz(fr)) << 4;

  constexpr int HF = PFN / 2, LAG = 4;  // W's fragments of a half stage
  v4u x0[PFM], x1[PFM], w0[HF], w1[HF];
  float sc[PFM], sw = 0.f;
  auto load_w = [&](int s, int i) __attribute__((always_inline)) {
    const uint8_t* pb = smem + 2 * P_ST + (s & 1) * P_ST + (wn0 + i * 16 + fr) * BKB;
    w0[i % HF] = *reinterpret_cast<const v4u*>(pb + c0);
    w1[i % HF] = *reinterpret_cast<const v4u*>(pb + c1);
  };
  // X, its scales and the first half of W's fragments of stage s into registers.
  auto read = [&](int s) __attribute__((always_inline)) {
    if ((s & 63) == 0) {
      wsl = wsp[min(s + lane, nst - 1)];
      asm volatile("" : "+v"(wsl));  // wait here, not for the DMA in flight at every use
    }
    const uint8_t* pa = smem + (s & 1) * P_ST + (wm0 + fr) * BKB;
    const float* ps =
        reinterpret_cast<const float*>(smem + P_SC + ((s >> 2) & 1) * PBM * 16 + (wm0 + fr) * 16) + (s - window(s >> 2));
    sw = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(wsl), s & 63));
#pragma unroll
    for (int j = 0; j < PFM; ++j) {
      x0[j] = *reinterpret_cast<const v4u*>(pa + j * 16 * BKB + c0);
      x1[j] = *reinterpret_cast<const v4u*>(pa + j * 16 * BKB + c1);
      sc[j] = ps[j * 16 * 4];
    }
#pragma unroll
    for (int i = 0; i < HF; ++i) load_w(s, i);
  };
  // Half a stage's products, each one's FMAs LAG products after it, so that no FMA waits for the matrix pipe; during
  // the first half the second's fragments of W replace those that are used up, and with DMA the requests for stage
  // s + 1 go out between the products. The order is held (the scheduler would move products and FMAs out of the phase
  // they are for, and sink the FMAs past the barrier).
  auto multiply = [&](auto half, auto dma, int s) __attribute__((always_inline)) {
    constexpr int h = decltype(half)::value;
    v4f p[LAG + 1];
    auto add = [&](int m) __attribute__((always_inline)) {
      const int i = h * HF + m / PFM, j = m % PFM;
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[i][j][q] = __builtin_fmaf(p[m % (LAG + 1)][q], sc[j], acc[i][j][q]);
      asm volatile("" : "+v"(acc[i][j]));
    };
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (h == 0) {
#pragma unroll
      for (int j = 0; j < PFM; ++j) sc[j] *= sw;
    }
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int m = 0; m < HF * PFM; ++m) {
      if constexpr (decltype(dma)::value)
        if (m % (HF * PFM / 4) == 0) issue(s + 1, m / (HF * PFM / 4));
      p[m % (LAG + 1)] = mfma_f8(w0[m / PFM], w1[m / PFM], x0[m % PFM], x1[m % PFM]);
      if (m >= LAG) add(m - LAG);
      if (h == 0 && m % PFM == PFM - 1) load_w(s, HF + m / PFM);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int m = HF * PFM - LAG; m < HF * PFM; ++m) add(m);
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
  };
  using H0 = std::integral_constant<int, 0>;
  using H1 = std::integral_constant<int, 1>;
  using True = std::true_type;
  using False = std::false_type;
  auto issue_all = [&](int s) {
#pragma unroll
    for (int p = 0; p < 4; ++p) issue(s, p);
  };

  issue_all(0);
  wait_vmcnt<0>();
  ring_barrier();
  if (wave < 4) {
    auto stage = [&](int s, auto dma) __attribute__((always_inline)) {
      read(s);
      multiply(H0{}, dma, s);
      multiply(H1{}, False{}, s);
      wait_vmcnt<0>();
      ring_barrier();
    };
    for (int s = 0; s + 1 < nst; ++s) stage(s, True{});
    stage(nst - 1, False{});
  } else {
    auto first = [&](int s) __attribute__((always_inline)) {
      read(s);
      multiply(H0{}, False{}, s);
      wait_vmcnt<0>();
      ring_barrier();
    };
    issue_all(1);  // nst >= 4
    first(0);
    for (int s = 1; s + 1 < nst; ++s) {
      multiply(H1{}, True{}, s);
      first(s);
    }
    multiply(H1{}, False{}, 0);
    first(nst - 1);
    multiply(H1{}, False{}, 0);
  }

  // Epilogue: each wave stages its outputs as bf16 in its own LDS region (every stage has been read), then writes
  // whole 16-byte pieces of rows.
  constexpr int CPR = PWN / 8;
  uint8_t* ep = smem + wave * (PWM * P_EP);
#pragma unroll
  for (int i = 0; i < PFN; ++i)
#pragma unroll
    for (int j = 0; j < PFM; ++j) {
      unsigned b[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) b[q] = __builtin_bit_cast(uint16_t, (__bf16)acc[i][j][q]);
      *reinterpret_cast<v2u*>(ep + (j * 16 + fr) * P_EP + (i * 16 + 4 * g) * 2) =
          v2u{b[0] | b[1] << 16, b[2] | b[3] << 16};
    }
  __builtin_amdgcn_s_waitcnt(0xC07F);
  asm volatile("" ::: "memory");
  const bool vec = N % 8 == 0;
  static_assert(PWM * CPR % 64 == 0, "whole instructions");
#pragma unroll
  for (int k = 0; k < PWM * CPR / 64; ++k) {
    const int at = k * 64 + lane, rr = at / CPR, cc = at % CPR;
    const v4u v = *reinterpret_cast<const v4u*>(ep + rr * P_EP + cc * 16);
    const int row = m0 + wm0 + rr, col = n0 + wn0 + cc * 8;
    if (row >= M) continue;
    uint16_t* dst = Y + (size_t)row * N + col;
    if (vec && col + 8 <= N) {
      __builtin_nontemporal_store(v, reinterpret_cast<v4u*>(dst));
    } else if (col + 8 <= N) {  // pieces share lines with their neighbours: through the caches
      *reinterpret_cast<v4u_any*>(dst) = v;
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (col + q < N) dst[q] = (uint16_t)(v[q >> 1] >> (16 * (q & 1)));
    }
  }
}

template <class C>
__global__ __launch_bounds__(C::NT) void gemm_fp8_ring(const uint8_t* __restrict__ Xq, const float* __restrict__ Xs,
                                                    const uint8_t* __restrict__ Wq, const float* __restrict__ Ws,
                                                    uint16_t* __restrict__ Y, int M, int N, int K, int tiles_m,
                                                    int tiles_n) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  const int T = tiles_m * tiles_n, b = (int)(blockIdx.y * gridDim.x + blockIdx.x);
  if (b >= T) return;
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
  const int tiles_m = (M - 1) / C::BM + 1, tiles_n = (N - 1) / C::BN + 1;
  const Grid grid = grid_of((int64_t)tiles_m * tiles_n, C::NT);
  hipLaunchKernelGGL(kern, dim3(grid.x, grid.y), dim3(C::NT), C::LDS, st, Xq, Xs, Wq, Ws, Y, M, N, K, tiles_m, tiles_n);
  return hipGetLastError();
}

hipError_t launch_turns(const uint8_t* Xq, const float* Xs, const uint8_t* Wq, const float* Ws, int M, int N, int K,
                        uint16_t* Y, int dev, hipStream_t st) {
  static std::atomic<int> ready[64];
  const bool cached = dev >= 0 && dev < 64;
  if (!cached || !ready[dev].load(std::memory_order_acquire)) {
    const hipError_t e =
        hipFuncSetAttribute((const void*)gemm_fp8_turns, hipFuncAttributeMaxDynamicSharedMemorySize, P_LDS);
    if (e != hipSuccess) return e;
    if (cached) ready[dev].store(1, std::memory_order_release);
  }
  const int tiles_m = (M - 1) / PBM + 1, tiles_n = (N - 1) / PBN + 1;
  const Grid grid = grid_of((int64_t)tiles_m * tiles_n, 512);
  hipLaunchKernelGGL(gemm_fp8_turns, dim3(grid.x, grid.y), dim3(512), P_LDS, st, Xq, Xs, Wq, Ws, Y, M, N, K, tiles_m,
                     tiles_n);
  return hipGetLastError();
}

}  // namespace
}  // namespace fp4

hipError_t fp8_launch_linear(const uint8_t* Xq, const float* Xs, const uint8_t* Wq, const float* Ws, int64_t M, int64_t N,
                             int64_t K, uint16_t* Y, hipStream_t st) {
  int dev = 0, cus = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e == hipSuccess) e = fp4_device_cus(dev, &cus);
  if (e != hipSuccess) return e;
  const int m = (int)M, n = (int)N, k = (int)K, shape = fp4::best_shape(M, N, K, cus);
  switch (shape) {
    case 0:
    case 1:
    case 2:
      return fp8_launch_linear_split(fp4::kShapes[shape].bm, fp4::kShapes[shape].bn, Xq, Xs, Wq, Ws, M, N, K, Y, dev, st);
    case 3: return fp4::launch<fp4::T64>(Xq, Xs, Wq, Ws, m, n, k, Y, dev, st);
    case 4: return fp4::launch<fp4::T128x64>(Xq, Xs, Wq, Ws, m, n, k, Y, dev, st);
    case 5: return fp4::launch<fp4::T128>(Xq, Xs, Wq, Ws, m, n, k, Y, dev, st);
    case 6: return fp4::launch<fp4::T128Two>(Xq, Xs, Wq, Ws, m, n, k, Y, dev, st);
    default: return fp4::launch_turns(Xq, Xs, Wq, Ws, m, n, k, Y, dev, st);
  }
}
