// A workgroup on the CPU, as far as the attention kernels need one: lanes are fibers that run one after the other up to the next builtin
// across lanes (the wave's lanes meet there) or __syncthreads (all of them do). What a lane reads from others' LDS without meeting them
// therefore depends on the order in which lanes run, which order_seed changes.
#pragma once
#include <sys/mman.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <functional>
#include <vector>

#define __device__
#define __host__
#define __global__
#define __forceinline__ inline
#define __launch_bounds__(...)
#define __shared__ static

struct dim3 {
  unsigned x, y;
  dim3(unsigned x = 1, unsigned y = 1) : x(x), y(y) {}
};
inline dim3 threadIdx, blockIdx;
using std::max;
using std::min;
typedef int hipError_t;
typedef void* hipStream_t;
constexpr int hipSuccess = 0, hipFuncAttributeMaxDynamicSharedMemorySize = 0;
inline int hipGetLastError() { return 0; }
inline int hipGetDevice(int* device) { return *device = 0; }
inline int hipFuncSetAttribute(const void*, int, int) { return 0; }

extern "C" void host_switch(void** from, void* to);
asm(R"(
.text
.globl host_switch
host_switch:
  push %rbp
  push %rbx
  push %r12
  push %r13
  push %r14
  push %r15
  mov %rsp, (%rdi)
  mov %rsi, %rsp
  pop %r15
  pop %r14
  pop %r13
  pop %r12
  pop %rbx
  pop %rbp
  ret
)");

namespace host {

// Memory with a page that nothing may touch right behind it, or with `front` right before it.
inline unsigned char* guarded(size_t bytes, bool front) {
  const size_t held = (bytes + 4095) / 4096 * 4096;
  auto* p = (unsigned char*)mmap(nullptr, held + 8192, PROT_NONE, MAP_PRIVATE | MAP_ANONYMOUS | MAP_NORESERVE, -1, 0);
  if (p == MAP_FAILED || mprotect(p + 4096, held, PROT_READ | PROT_WRITE) != 0) abort();
  return p + 4096 + (front ? 0 : held - bytes);
}

enum At { kRuns, kInWave, kInGroup, kDone };
struct Fiber {
  void* sp;
  At at;
};
struct Wave {
  int live, arrived;
  unsigned turn;
  uint64_t lanes[2];
  alignas(64) unsigned char slots[2][64][64];
};
constexpr size_t kStack = 64 << 10;
inline std::vector<Fiber> fibers;
inline std::vector<Wave> waves;
inline std::function<void()> body;
inline void* outside;
inline int now, live, arrived;
inline unsigned char *stacks, *lds;
inline bool front;
inline unsigned order_seed = 0, order;

inline int lane() { return now & 63; }
inline Wave& wave() { return waves[now >> 6]; }

inline int next() {
  const int n = (int)fibers.size();
  if (order_seed) order = order * 1664525u + 1013904223u;
  // by waves: one starts at random, the lanes of a wave follow each other
  const int from = order_seed && (order >> 16) % 4 == 0 ? (int)((order >> 20) % (n / 64)) * 64 : now;
  for (int i = 0; i < n; ++i)
    if (fibers[(from + i) % n].at == kRuns) return (from + i) % n;
  fprintf(stderr, "lanes wait for lanes that have ended or wait elsewhere: workgroup %u, %u\n", blockIdx.x, blockIdx.y);
  abort();
}
inline void to(int other) {
  const int me = now;
  now = other;
  threadIdx.x = other;
  if (other != me) host_switch(&fibers[me].sp, fibers[other].sp);
}
inline void release(Wave& w, int index) {
  uint64_t lanes = 0;
  for (int i = 0; i < 64; ++i) {
    Fiber& f = fibers[64 * index + i];
    lanes |= (uint64_t)(f.at != kDone) << i;
    if (f.at == kInWave) f.at = kRuns;
  }
  w.lanes[w.turn++ & 1] = lanes;
  w.arrived = 0;
}
inline void release_group() {
  arrived = 0;
  for (Fiber& f : fibers)
    if (f.at == kInGroup) f.at = kRuns;
}
template <class T>
struct Slots {
  const unsigned char (*slots)[64];
  uint64_t lanes;
  T operator[](int lane) const {
    T t;
    memcpy(&t, slots[lane], sizeof t);
    return t;
  }
};
// The value that every lane of the wave brings.
template <class T>
inline Slots<T> meet(const T& mine) {
  static_assert(sizeof(T) <= 64, "a slot's bytes");
  Wave& w = wave();
  const unsigned turn = w.turn & 1;
  memcpy(w.slots[turn][lane()], &mine, sizeof mine);
  if (++w.arrived == w.live) {
    release(w, now >> 6);
  } else {
    fibers[now].at = kInWave;
    to(next());
  }
  return {w.slots[turn], w.lanes[turn]};
}
inline void meet_group() {
  if (++arrived == live) {
    release_group();
  } else {
    fibers[now].at = kInGroup;
    to(next());
  }
}
inline void lane_main() {
  body();
  fibers[now].at = kDone;
  Wave& w = wave();
  --w.live;
  --live;
  if (w.live && w.arrived == w.live) release(w, now >> 6);
  if (live && arrived == live) release_group();
  void* never;
  if (live == 0) host_switch(&never, outside);
  now = next();
  threadIdx.x = now;
  host_switch(&never, fibers[now].sp);
}
inline void run_group(int threads) {
  if (!stacks) stacks = (unsigned char*)mmap(nullptr, 512 * kStack, PROT_READ | PROT_WRITE, MAP_PRIVATE | MAP_ANONYMOUS | MAP_NORESERVE, -1, 0);
  fibers.assign(threads, {});
  waves.assign(threads / 64, {});
  for (Wave& w : waves) w.live = 64;
  live = threads;
  arrived = 0;
  for (int i = 0; i < threads; ++i) {
    auto** sp = (void**)(stacks + (i + 1) * kStack - 64);
    *--sp = nullptr;
    *--sp = (void*)&lane_main;
    fibers[i].sp = sp - 6;
  }
  now = threadIdx.x = 0;
  host_switch(&outside, fibers[0].sp);
}
template <class K, class... A>
inline void run_grid(K kernel, dim3 grid, dim3 block, size_t shared, const A&... args) {
  static size_t have = 0;
  if (shared && shared != have) lds = guarded(have = shared, front);
  body = [&] { kernel(args...); };
  order = order_seed;
  for (blockIdx.y = 0; blockIdx.y < grid.y; ++blockIdx.y)
    for (blockIdx.x = 0; blockIdx.x < grid.x; ++blockIdx.x) run_group(block.x);
}

inline float bf16(unsigned bits) {
  const unsigned u = bits << 16;
  float f;
  memcpy(&f, &u, 4);
  return f;
}
inline float e4m3(unsigned c) {
  const int e = (c >> 3) & 15, m = c & 7;
  const float x = e == 15 && m == 7 ? NAN : e ? ldexpf(1.f + m / 8.f, e - 7) : ldexpf(m / 8.f, -6);
  return (c & 0x80) ? -x : x;
}
typedef __bf16 v2 __attribute__((ext_vector_type(2)));
typedef __bf16 v8 __attribute__((ext_vector_type(8)));
struct Operands {
  uint16_t a[8], b[8];
};
// D[row, column] += A[row, k] B[k, column]: a lane's operands are row (column) lane % side, k from 8 (lane / side) on.
template <int SIDE, class Acc, class Row>
inline Acc product(v8 a, v8 b, Acc c, int n, Row row) {
  Operands x;
  memcpy(x.a, &a, 16);
  memcpy(x.b, &b, 16);
  const auto s = meet(x);
  for (int i = 0; i < n; ++i) {
    float sum = c[i];
    for (int k = 0; k < 64 / SIDE; ++k) {
      const auto* ra = (const Operands*)s.slots[row(i) + SIDE * k];
      const auto* rb = (const Operands*)s.slots[lane() % SIDE + SIDE * k];
      for (int e = 0; e < 8; ++e) sum += bf16(ra->a[e]) * bf16(rb->b[e]);
    }
    c[i] = sum;
  }
  return c;
}

}  // namespace host

#define hipLaunchKernelGGL(kernel, grid, block, shared, stream, ...) host::run_grid(kernel, grid, block, shared, __VA_ARGS__)

inline void __syncthreads() { host::meet_group(); }
inline unsigned long long __ballot(bool p) {
  const auto s = host::meet((unsigned char)p);
  unsigned long long r = 0;
  for (int i = 0; i < 64; ++i)
    if ((s.lanes >> i) & 1) r |= (unsigned long long)s[i] << i;
  return r;
}
inline bool __any(bool p) { return __ballot(p) != 0; }
inline bool __all(bool p) { return __ballot(!p) == 0; }
inline int __popcll(unsigned long long x) { return __builtin_popcountll(x); }
inline float __uint_as_float(unsigned u) { return __builtin_bit_cast(float, u); }
inline unsigned __float_as_uint(float f) { return __builtin_bit_cast(unsigned, f); }
inline float __int_as_float(int u) { return __builtin_bit_cast(float, u); }
inline int __float_as_int(float f) { return __builtin_bit_cast(int, f); }
inline float __shfl_xor(float v, int by) { return host::meet(v)[host::lane() ^ by]; }
inline unsigned long long atomicOr(unsigned long long* p, unsigned long long v) {
  const unsigned long long old = *p;
  *p |= v;
  return old;
}
inline float __builtin_amdgcn_exp2f(float x) { return exp2f(x); }
inline unsigned max(unsigned a, int b) { return std::max(a, (unsigned)b); }
struct Swapped {
  unsigned r[2];
  unsigned operator[](int i) const { return r[i]; }
};
inline Swapped __builtin_amdgcn_permlane32_swap(unsigned v, unsigned, bool, bool) {
  const auto s = host::meet(v);
  return {{s[host::lane() & 31], s[host::lane() | 32]}};
}
inline Swapped __builtin_amdgcn_permlane16_swap(unsigned v, unsigned, bool, bool) {
  const auto s = host::meet(v);
  return {{s[host::lane() & ~16], s[host::lane() | 16]}};
}
inline int __builtin_amdgcn_readlane(int v, int lane) { return host::meet(v)[lane]; }
inline int __builtin_amdgcn_readfirstlane(int v) { return v; }  // of values that all lanes have alike
inline int __builtin_amdgcn_update_dpp(int old, int v, int ctrl, int rows, int, bool) {
  const auto s = host::meet(v);
  const int l = host::lane(), row = l / 16, i = l % 16;
  if (!((rows >> row) & 1)) return old;
  if (ctrl >= 0x111 && ctrl <= 0x11F) return i >= ctrl - 0x110 ? s[l - (ctrl - 0x110)] : old;
  if (ctrl >= 0x121 && ctrl <= 0x12F) return s[16 * row + (i - (ctrl - 0x120) + 16) % 16];
  if (ctrl == 0x142) return row >= 1 ? s[row * 16 - 1] : old;
  if (ctrl == 0x143) return l >= 32 ? s[31] : old;
  abort();
}
inline unsigned __builtin_amdgcn_perm(unsigned high, unsigned low, unsigned take) {
  const uint64_t w = (uint64_t)high << 32 | low;
  unsigned r = 0;
  for (int i = 0; i < 32; i += 8) r |= (unsigned)(w >> (8 * ((take >> i) & 7)) & 0xFF) << i;
  return r;
}
inline unsigned __builtin_amdgcn_bitop3_b32(unsigned a, unsigned b, unsigned c, unsigned table) {
  unsigned r = 0;
  for (int k = 0; k < 8; ++k)
    if ((table >> k) & 1) r |= (k & 4 ? a : ~a) & (k & 2 ? b : ~b) & (k & 1 ? c : ~c);
  return r;
}
inline host::v2 __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(unsigned codes, float, bool high) {
  const unsigned w = high ? codes >> 16 : codes;
  return __builtin_bit_cast(host::v2, __float_as_uint(host::e4m3(w & 0xFF)) >> 16 | (__float_as_uint(host::e4m3(w >> 8 & 0xFF)) & 0xFFFF0000u));
}
inline float __builtin_amdgcn_fdot2_f32_bf16(host::v2 a, host::v2 b, float c, bool) {
  const unsigned x = __builtin_bit_cast(unsigned, a), y = __builtin_bit_cast(unsigned, b);
  return host::bf16(x & 0xFFFF) * host::bf16(y & 0xFFFF) + host::bf16(x >> 16) * host::bf16(y >> 16) + c;
}
template <class Acc>
inline Acc __builtin_amdgcn_mfma_f32_32x32x16_bf16(host::v8 a, host::v8 b, Acc c, int, int, int) {
  return host::product<32>(a, b, c, 16, [](int i) { return 8 * (i / 4) + 4 * (host::lane() / 32) + i % 4; });
}
template <class Acc>
inline Acc __builtin_amdgcn_mfma_f32_16x16x32_bf16(host::v8 a, host::v8 b, Acc c, int, int, int) {
  return host::product<16>(a, b, c, 4, [](int i) { return 4 * (host::lane() / 16) + i; });
}
#define __builtin_amdgcn_sched_group_barrier(...) ((void)0)
#define __builtin_amdgcn_s_setprio(...) ((void)0)
#define __builtin_amdgcn_fence(...) ((void)0)
inline void __builtin_amdgcn_wave_barrier() { host::meet(0); }
inline int __builtin_amdgcn_cvt_pk_fp8_f32(float, float, int, bool) { abort(); }
