// The attention kernels' own source on the CPU (see hip/hip_runtime.h here): a call on buffers of just their bytes, each with a page
// behind it (or before it) that ends the program when touched; sampled rows against float64; a checksum of Out.
//
// Arguments: prompt?, waves (0: as the rule has it), splits, dim, 8 bits, query heads, heads, page size, tokens side by side?, window, sinks,
// columns past the longest sequence, guards in front?, order of lanes, rows to check, rows of nobody, batch, lengths ..., new rows ...
#include <hip/hip_runtime.h>
#include <signal.h>
#include <unistd.h>

#include "attention_prompt.hip"
// two kernels' sources in one: the second one's names of its own
#define kSlack kDecodeSlack
#define Ids DecodeIds
#define ids_of decode_ids_of
#define launch decode_launch
#define join decode_join
#include "attention_decode.hip"
#undef launch
#undef join

hipError_t fp4_device_cus(int, int* cus) {
  *cus = 256;
  return 0;
}

static void on_fault(int, siginfo_t* info, void*) {
  char text[200];
  const int n = snprintf(text, sizeof text, "out of range: %p by workgroup %u, %u thread %d\n", info->si_addr, blockIdx.x, blockIdx.y, host::now);
  (void)!write(2, text, n);
  _exit(3);
}
static uint64_t state = 1;
static unsigned draw() { return (state = state * 6364136223846793005ull + 1442695040888963407ull) >> 33; }
static float normal() {
  float s = 0;
  for (int i = 0; i < 4; ++i) s += draw() / 2147483648.f - 0.5f;
  return 1.7f * s;
}

template <int D, bool E4M3>
static void forced(const Fp4AttentionArgs& a, const fp4::PromptWay& way) {
  if constexpr (fp4::prompt_eight(D, E4M3, false))
    if (way.waves == 8 && way.splits == 1) return (void)fp4::launch<D, E4M3, 8, false>(a, way, 0, nullptr);
  if constexpr (fp4::prompt_eight(D, E4M3, true))
    if (way.waves == 8) return (void)fp4::launch<D, E4M3, 8, true>(a, way, 0, nullptr);
  if (way.splits > 1) fp4::launch<D, E4M3, 4, true>(a, way, 0, nullptr);
  else fp4::launch<D, E4M3, 4, false>(a, way, 0, nullptr);
}

int main(int argc, char** argv) {
  int at = 1;
  auto arg = [&] { return at < argc ? (int)atoll(argv[at++]) : 0; };
  const bool prompt = arg();
  const int waves = arg(), splits = arg(), D = arg();
  const bool e4m3 = arg();
  const int Hq = arg(), H = arg(), page = arg();
  const bool tokens = arg();
  const int window = arg(), sinks = arg(), more = arg();
  const bool front = host::front = arg();
  host::order_seed = arg();
  const int check = arg(), pad = arg(), B = arg();
  std::vector<int> len(B), news(B, 1);
  for (int& n : len) n = arg();
  if (prompt)
    for (int& n : news) n = arg();

  struct sigaction act {};
  act.sa_sigaction = on_fault;
  act.sa_flags = SA_SIGINFO | SA_ONSTACK;
  stack_t alt{};
  alt.ss_size = 1 << 16;
  alt.ss_sp = malloc(alt.ss_size);
  sigaltstack(&alt, nullptr);
  sigaction(SIGSEGV, &act, nullptr);
  sigaction(SIGBUS, &act, nullptr);

  int cols = 0, P = 1;
  for (int n : len) cols = std::max(cols, (n + page - 1) / page), P += (n + page - 1) / page;
  cols = std::max(cols + more, 1);
  const int64_t size = e4m3 ? 1 : 2, page_bytes = (int64_t)H * page * D * size;
  uint8_t* kv[2];
  float* scales[2] = {nullptr, nullptr};
  for (int i = 0; i < 2; ++i) {
    kv[i] = host::guarded(P * page_bytes, front);
    if (!e4m3) {
      for (int64_t n = 0; n < P * page_bytes / 2; ++n) ((uint16_t*)kv[i])[n] = __float_as_uint(normal()) >> 16;
      continue;
    }
    for (int64_t n = 0; n < P * page_bytes; ++n) kv[i][n] = draw() & 0xBF;  // magnitudes below 2
    scales[i] = (float*)host::guarded((size_t)P * H * page * 4, front);
    for (int n = 0; n < P * H * page; ++n) scales[i][n] = 0.5f + draw() % 1000 * 1e-3f;
  }
  std::vector<int> order(P);
  for (int i = 0; i < P; ++i) order[i] = i;
  for (int i = P - 1; i > 0; --i) std::swap(order[i], order[draw() % (i + 1)]);
  int* table = (int*)host::guarded((size_t)B * cols * 4, front);
  int* lengths = (int*)host::guarded(B * 4, front);
  int* starts = (int*)host::guarded((B + 1) * 4, front);
  starts[0] = 0;
  for (int b = 0, p = 0; b < B; ++b) {
    for (int c = 0; c < cols; ++c) table[b * cols + c] = c < (len[b] + page - 1) / page ? order[p++] : c % 2 ? -1 : P;
    lengths[b] = len[b];
    starts[b + 1] = starts[b] + news[b];
  }
  const int T = starts[B] + (prompt ? pad : 0);
  const size_t out_bytes = (size_t)T * Hq * D * 2;
  uint16_t* q = (uint16_t*)host::guarded(out_bytes, front);
  uint16_t* out = (uint16_t*)host::guarded(out_bytes, front);
  for (size_t n = 0; n < out_bytes / 2; ++n) q[n] = __float_as_uint(normal()) >> 16;
  memset(out, 0x55, out_bytes);
  const size_t room = FP4_ATTENTION_WORKSPACE_BYTES(T, B, Hq, H, D);

  int shift = 4;
  while ((1 << shift) < page) ++shift;
  Fp4AttentionArgs a{};
  a.cache = fp4::Paged{kv[0], kv[1], scales[0], scales[1], page_bytes, (tokens ? 1 : page) * D * size, (tokens ? H : 1) * D * size,
                       (int64_t)H * page, tokens ? 1 : page, tokens ? H : 1, table, cols, lengths, P, shift, cols, B, H};
  a.starts = starts;
  a.q = q;
  a.out = out;
  a.q_token = (int64_t)Hq * D;
  a.q_head = D;
  a.scale = 1.f / sqrtf((float)D);
  a.T = T;
  a.q_heads = Hq;
  a.window = window;
  a.sinks = sinks;
  a.workspace = host::guarded((room + 15) / 16 * 16, front);
  if (!prompt) fp4_launch_attention_decode(a, D, e4m3, nullptr);
  else if (!waves) fp4_launch_attention_prompt(a, D, e4m3, nullptr);
  else {
    const fp4::PromptWay way{waves, splits, 1024 / D};
    if (D == 64) e4m3 ? forced<64, true>(a, way) : forced<64, false>(a, way);
    else if (D == 128) e4m3 ? forced<128, true>(a, way) : forced<128, false>(a, way);
    else e4m3 ? forced<256, true>(a, way) : forced<256, false>(a, way);
  }

  // p and the result are rounded to bf16: 2^-8 of sum p |v| / sum p, and 2^-8 of the result; float32 scores are far below that here
  double worst = 0;
  for (int n = 0; n < check; ++n) {
    const int b = draw() % B;
    if (!news[b]) continue;
    const int t = starts[b] + draw() % news[b], h = draw() % Hq, i = len[b] - (starts[b + 1] - t), head = h / (Hq / H);
    auto value = [&](int which, int j, int d) -> double {
      const int64_t p = table[b * cols + j / page], in = j % page;
      const uint8_t* x = kv[which] + p * page_bytes + head * a.cache.head_stride + in * a.cache.token_stride;
      if (!e4m3) return host::bf16(((const uint16_t*)x)[d]);
      return (double)host::e4m3(x[d]) * scales[which][p * a.cache.spage_stride + head * a.cache.shead_stride + in * a.cache.stoken_stride];
    };
    const uint16_t* x = q + ((size_t)t * Hq + h) * D;
    std::vector<double> score;
    std::vector<int> seen;
    double top = -1e300, sum = 0;
    for (int j = 0; j <= i; ++j) {
      if (window && i - j >= window && j >= sinks) continue;
      double z = 0;
      for (int d = 0; d < D; ++d) z += (double)host::bf16(x[d]) * value(0, j, d);
      seen.push_back(j);
      score.push_back(z * a.scale);
      top = std::max(top, score.back());
    }
    for (double& z : score) sum += z = exp(z - top);
    for (int d = 0; d < D; ++d) {
      double o = 0, size = 0;
      for (size_t k = 0; k < seen.size(); ++k) {
        const double v = score[k] / sum * value(1, seen[k], d);
        o += v;
        size += std::fabs(v);
      }
      const double off = std::fabs(host::bf16(out[((size_t)t * Hq + h) * D + d]) - o) / (1.05 / 256 * (size + std::fabs(o)) + 1e-30);
      if (!(off <= worst)) worst = off;
    }
  }
  uint64_t sum = 0;
  for (size_t n = 0; n < out_bytes / 2; ++n) sum = sum * 1099511628211ull + out[n];
  bool left = true;
  for (size_t n = (size_t)starts[B] * Hq * D; n < out_bytes / 2; ++n) left &= out[n] == 0x5555;
  printf("%d %.3f %llx\n", left, worst, (unsigned long long)sum);
}
