// C ABI of the gfx950 FP4 library: argument validation, then kernel launches.
// Declarations and the contract of every call are in include/fp4.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "../../include/fp4.h"
#include "common.hpp"
#include "operators.hpp"
#include "paged.hpp"

namespace {

thread_local char g_err[512] = "";

int fail(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int fail(int status, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof g_err, fmt, ap);
  va_end(ap);
  return status;
}

int ok() {
  g_err[0] = '\0';
  return FP4_OK;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int check_quantize(const char* who, const void* X, int64_t M, int64_t K, int64_t ld, int block, int fmt,
                   const uint8_t* codes, const uint8_t* scales, const float* ts) {
  if (fmt != FP4_MXFP4 && fmt != FP4_NVFP4) return fail(FP4_E_FORMAT, "%s: unknown format %d", who, fmt);
  if (block != 16 && block != 32 && block != 64 && block != 128)
    return fail(FP4_E_BLOCK, "%s: Hadamard block %d not in {16, 32, 64, 128}", who, block);
  if (!X || !codes || !scales) return fail(FP4_E_NULLPTR, "%s: input, codes and scales must be non-NULL", who);
  if (fmt == FP4_NVFP4 && !ts) return fail(FP4_E_NULLPTR, "%s: NVFP4 needs a tensor_scale buffer", who);
  if (fmt == FP4_MXFP4 && ts) return fail(FP4_E_NULLPTR, "%s: tensor_scale must be NULL for MXFP4", who);
  if (M < 1 || K < 1) return fail(FP4_E_SHAPE, "%s: rows (%lld) and K (%lld) must be >= 1", who, (long long)M,
                                  (long long)K);
  if (K % 32 || K % block)
    return fail(FP4_E_SHAPE, "%s: K=%lld must be a multiple of 32 and of the block %d", who, (long long)K, block);
  if (ld < K) return fail(FP4_E_SHAPE, "%s: leading dimension %lld < K=%lld", who, (long long)ld, (long long)K);
  if (M > 0x7FFFFFFFLL / (K / 32) || ld > (int64_t)1 << 40)  // K >= 32 here; no product can overflow
    return fail(FP4_E_SHAPE, "%s: tensor too large (rows*K/32 must fit in 31 bits)", who);
  if (!aligned(X, 16) || ld % 8) return fail(FP4_E_ALIGN, "%s: input must be 16-byte aligned, ld %% 8 == 0", who);
  if (!aligned(codes, 16)) return fail(FP4_E_ALIGN, "%s: codes must be 16-byte aligned", who);
  if (fmt == FP4_NVFP4 && (!aligned(scales, 2) || !aligned(ts, 4)))
    return fail(FP4_E_ALIGN, "%s: NVFP4 scales must be 2-byte aligned, tensor_scale 4-byte aligned", who);
  return FP4_OK;
}

int launched(const char* who, hipError_t e) {
  if (e != hipSuccess) return fail(FP4_E_HIP, "%s: HIP error at launch: %s", who, hipGetErrorString(e));
  return ok();
}

int quantize(const char* who, const void* X, int64_t M, int64_t K, int64_t ld, int block, int fmt, int rule,
             const int8_t* signs, uint8_t* codes, uint8_t* scales, float* ts, void* stream) {
  int st = check_quantize(who, X, M, K, ld, block, fmt, codes, scales, ts);
  if (st != FP4_OK) return st;
  const bool given_ts = (rule & FP4_TENSOR_SCALE_IN) != 0;
  rule &= ~FP4_TENSOR_SCALE_IN;
  if (given_ts && fmt != FP4_NVFP4) return fail(FP4_E_FORMAT, "%s: a given tensor scale applies to NVFP4 only", who);
  if (rule != FP4_SCALE_STANDARD && rule != FP4_SCALE_OCP_FLOOR && rule != FP4_SCALE_OAS && rule != FP4_SCALE_FIT)
    return fail(FP4_E_FORMAT, "%s: unknown scale rule %d", who, rule);
  if (fmt == FP4_NVFP4 && (rule == FP4_SCALE_OCP_FLOOR || rule == FP4_SCALE_OAS))
    return fail(FP4_E_FORMAT, "%s: scale rule %d applies to MXFP4 only", who, rule);
  if (signs && !aligned(signs, 16)) return fail(FP4_E_ALIGN, "%s: signs must be 16-byte aligned", who);
  return launched(who, fp4_launch_rotate_quantize(static_cast<const uint16_t*>(X), M, K, ld, block, fmt, rule,
                                                  given_ts, signs, codes, scales, ts,
                                                  static_cast<hipStream_t>(stream)));
}

int check_decode_step(const char* who, const void* X, int64_t M, int64_t K, int64_t ldx, int block,
                      const uint8_t* Wq, const uint8_t* Ws, int64_t N, void* Y, int y_dtype) {
  if (block != 16 && block != 32 && block != 64 && block != 128)
    return fail(FP4_E_BLOCK, "%s: Hadamard block %d not in {16, 32, 64, 128}", who, block);
  if (y_dtype != FP4_OUT_F32 && y_dtype != FP4_OUT_BF16)
    return fail(FP4_E_FORMAT, "%s: unknown output dtype %d", who, y_dtype);
  if (!X || !Wq || !Ws || !Y) return fail(FP4_E_NULLPTR, "%s: X, Wq, Ws and Y must be non-NULL", who);
  if (M < 1 || M > 16 || N < 1 || K < 512 || K % 512 || N > 0x7FFFFFFF || K > 0x7FFFFFFF)
    return fail(FP4_E_SHAPE, "%s: need 1 <= M <= 16, N >= 1 and K a positive multiple of 512 (M=%lld N=%lld K=%lld)",
                who, (long long)M, (long long)N, (long long)K);
  if (!fp4_decode_fused_fits(M, N, K))
    return fail(FP4_E_SHAPE, "%s: M * K too large for the workgroup's LDS; use fp4_rotate_quantize + fp4_linear", who);
  if (ldx < K || ldx > (int64_t)1 << 40) return fail(FP4_E_SHAPE, "%s: leading dimension %lld < K", who, (long long)ldx);
  if (!aligned(X, 16) || ldx % 8) return fail(FP4_E_ALIGN, "%s: X must be 16-byte aligned, ldx %% 8 == 0", who);
  if (!aligned(Wq, 16) || !aligned(Ws, 16) || !aligned(Y, 16))
    return fail(FP4_E_ALIGN, "%s: Wq, Ws and Y must be 16-byte aligned", who);
  return FP4_OK;
}

// The validated decode step: one fused launch, or, with a workspace and more rows of X per CU
// than the fused kernel quantizes profitably, the quantizer into the workspace (codes, then the
// E8M0 scales at the next 256-byte boundary) followed by the decode GEMM. Both give the same bits.
int decode_step(const char* who, const void* X, int64_t M, int64_t K, int64_t ldx, int block, const uint8_t* Wq,
                const uint8_t* Ws, int64_t N, void* Y, int y_dtype, uint8_t* ws, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  const bool bf16 = y_dtype == FP4_OUT_BF16;
  bool fused = true;
  if (ws) {
    const hipError_t e = fp4_decode_fused_preferred(M, N, K, &fused);
    if (e != hipSuccess) return launched(who, e);
  }
  if (fused)
    return launched(who, fp4_launch_decode_fused(static_cast<const uint16_t*>(X), ldx, block, Wq, Ws, M, N, K, Y, bf16,
                                                 st));
  uint8_t* xq = ws;
  uint8_t* xs = ws + FP4_LINEAR_WORKSPACE_CODES((size_t)M, (size_t)K);
  hipError_t e = fp4_launch_rotate_quantize(static_cast<const uint16_t*>(X), M, K, ldx, block, FP4_MXFP4,
                                            FP4_SCALE_STANDARD, false, nullptr, xq, xs, nullptr, st);
  if (e == hipSuccess) e = fp4_launch_gemm_mxfp4_decode(xq, xs, Wq, Ws, M, N, K, Y, bf16, st);
  return launched(who, e);
}

// Checks shared by the 8-bit quantizers and the norm: X [M, ld] bf16 -> codes [M, K], scales.
int check_fp8_rows(const char* who, const void* X, int64_t M, int64_t K, int64_t ld, const uint8_t* codes,
                   const float* scales) {
  if (!X || !codes || !scales) return fail(FP4_E_NULLPTR, "%s: input, codes and scales must be non-NULL", who);
  if (M < 1 || K < 128 || K % 128)
    return fail(FP4_E_SHAPE, "%s: need rows >= 1 and K a positive multiple of 128 (rows=%lld K=%lld)", who,
                (long long)M, (long long)K);
  if (ld < K || ld > (int64_t)1 << 40)
    return fail(FP4_E_SHAPE, "%s: leading dimension %lld < K=%lld, or too large", who, (long long)ld, (long long)K);
  if (M > 0x7FFFFFFFLL / (K / 8)) return fail(FP4_E_SHAPE, "%s: tensor too large (rows*K/8 must fit in 31 bits)", who);
  if (!aligned(X, 16) || ld % 8) return fail(FP4_E_ALIGN, "%s: input must be 16-byte aligned, ld %% 8 == 0", who);
  if (!aligned(codes, 16) || !aligned(scales, 4))
    return fail(FP4_E_ALIGN, "%s: codes must be 16-byte aligned, scales 4-byte aligned", who);
  return FP4_OK;
}

// The cache of the attention calls and the shapes that go with it, as the kernels take them.
int check_cache(const char* who, const fp4_kv_cache* c, int64_t q_heads, fp4::Paged* out) {
  if (!c || !c->k || !c->v || !c->table || !c->lengths) return fail(FP4_E_NULLPTR, "%s: cache pointers must be non-NULL", who);
  if (c->dtype != FP4_KV_BF16 && c->dtype != FP4_KV_E4M3) return fail(FP4_E_FORMAT, "%s: unknown cache dtype %d", who, c->dtype);
  const bool e4m3 = c->dtype == FP4_KV_E4M3;
  if ((c->k_scales != nullptr) != e4m3 || (c->v_scales != nullptr) != e4m3)
    return fail(FP4_E_NULLPTR, "%s: k_scales and v_scales belong to an E4M3 cache, and only there", who);
  if (c->heads < 1 || c->heads > 1024 || (c->dim != 64 && c->dim != 128 && c->dim != 256))
    return fail(FP4_E_SHAPE, "%s: need 1 to 1024 heads of 64, 128 or 256 (heads=%d dim=%d)", who, c->heads, c->dim);
  if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)))
    return fail(FP4_E_SHAPE, "%s: page_size=%d is no power of two from 16 to 1024", who, c->page_size);
  if (c->pages < 1 || c->pages > 0x7FFFFFFF) return fail(FP4_E_SHAPE, "%s: pages=%lld not in 1 .. 2^31 - 1", who, (long long)c->pages);
  const int64_t far = (int64_t)1 << 40;
  for (const int64_t s : {c->page_stride, c->head_stride, c->token_stride})
    if (s < c->dim || s > far) return fail(FP4_E_SHAPE, "%s: cache stride %lld below dim or too large", who, (long long)s);
  // a granule's tokens are addressed by 32-bit offsets from its first
  if (c->token_stride > (1 << 25)) return fail(FP4_E_SHAPE, "%s: token stride %lld above 2^25", who, (long long)c->token_stride);
  if (e4m3)
    for (const int64_t s : {c->scale_page_stride, c->scale_head_stride, c->scale_token_stride})
      if (s < 1 || s > far) return fail(FP4_E_SHAPE, "%s: scale stride %lld not positive or too large", who, (long long)s);
  if (c->cols < 1 || c->cols > ((int64_t)1 << 30) / c->page_size || c->table_stride < c->cols || c->table_stride > far)
    return fail(FP4_E_SHAPE, "%s: need cols >= 1, cols * page_size <= 2^30 and table_stride >= cols (cols=%lld stride=%lld)", who,
                (long long)c->cols, (long long)c->table_stride);
  if (c->batch < 1 || c->batch > 65535 || c->batch * q_heads > (1 << 22))
    return fail(FP4_E_SHAPE, "%s: need 1 <= batch <= 65535 and batch * query heads <= 2^22 (batch=%lld)", who, (long long)c->batch);
  if (c->batch * c->cols > ((int64_t)1 << 35) / c->page_size)
    return fail(FP4_E_SHAPE, "%s: batch * cols * page_size above 2^35", who);
  const int64_t unit = e4m3 ? 16 : 8;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || c->page_stride % unit || c->head_stride % unit || c->token_stride % unit)
    return fail(FP4_E_ALIGN, "%s: pages must be 16-byte aligned, their strides multiples of %d", who, (int)unit);
  if (!aligned(c->table, 4) || !aligned(c->lengths, 4) || (e4m3 && (!aligned(c->k_scales, 4) || !aligned(c->v_scales, 4))))
    return fail(FP4_E_ALIGN, "%s: table, lengths and scales must be 4-byte aligned", who);
  const int64_t bytes = e4m3 ? 1 : 2;
  int shift = 4;
  while ((1 << shift) < c->page_size) ++shift;
  *out = fp4::Paged{static_cast<const uint8_t*>(c->k), static_cast<const uint8_t*>(c->v), c->k_scales, c->v_scales,
                    c->page_stride * bytes, c->head_stride * bytes, c->token_stride * bytes, c->scale_page_stride,
                    c->scale_head_stride, c->scale_token_stride, c->table, c->table_stride, c->lengths, (int)c->pages, shift,
                    (int)c->cols, (int)c->batch, c->heads};
  return FP4_OK;
}

// Rows of heads of dim bf16 numbers.
int check_heads(const char* who, const char* what, const void* X, int64_t row, int64_t head, int dim) {
  if (row < dim || head < dim || row > (int64_t)1 << 40 || head > (int64_t)1 << 40)
    return fail(FP4_E_SHAPE, "%s: strides of %s (rows %lld, heads %lld) below dim or too large", who, what, (long long)row, (long long)head);
  if (!aligned(X, 16) || row % 8 || head % 8)
    return fail(FP4_E_ALIGN, "%s: %s must be 16-byte aligned, its strides multiples of 8", who, what);
  return FP4_OK;
}

int attention(const char* who, const fp4_kv_cache* cache, const int* starts, int64_t T, const void* Q, int64_t q_row, int64_t q_head,
              int q_heads, float scale, int64_t window, int64_t sinks, void* Out, void* workspace, size_t workspace_bytes,
              bool decode, void* stream) {
  if (!Q || !Out || !workspace || (!decode && !starts)) return fail(FP4_E_NULLPTR, "%s: pointers must be non-NULL", who);
  Fp4AttentionArgs a{};
  int st = check_cache(who, cache, q_heads, &a.cache);
  if (st != FP4_OK) return st;
  if (decode) T = cache->batch;
  if (q_heads < 1 || q_heads > 1024 || q_heads % cache->heads)
    return fail(FP4_E_SHAPE, "%s: q_heads=%d is no multiple of the cache's %d heads up to 1024", who, q_heads, cache->heads);
  if (T < 1 || T > (1 << 24) || T * q_heads > (1 << 30))
    return fail(FP4_E_SHAPE, "%s: need 1 <= T <= 2^24 and T * q_heads <= 2^30 (T=%lld)", who, (long long)T);
  if (!(scale > 0.f) || !__builtin_isfinite(scale)) return fail(FP4_E_SHAPE, "%s: scale must be finite and positive", who);
  if (window < 0 || sinks < 0) return fail(FP4_E_SHAPE, "%s: window and sinks must not be negative", who);
  const size_t need = FP4_ATTENTION_WORKSPACE_BYTES(T, cache->batch, q_heads, cache->heads, cache->dim);
  if (workspace_bytes < need) return fail(FP4_E_SHAPE, "%s: workspace of %zu bytes, %zu needed", who, workspace_bytes, need);
  st = check_heads(who, "Q", Q, q_row, q_head, cache->dim);
  if (st != FP4_OK) return st;
  if (!aligned(Out, 16) || !aligned(workspace, 16) || !aligned(starts, 4))
    return fail(FP4_E_ALIGN, "%s: Out and workspace must be 16-byte aligned, starts 4-byte aligned", who);
  const int64_t most = (int64_t)1 << 30;
  a.starts = starts;
  a.q = static_cast<const uint16_t*>(Q);
  a.out = static_cast<uint16_t*>(Out);
  a.q_token = q_row;
  a.q_head = q_head;
  a.scale = scale;
  a.T = (int)T;
  a.q_heads = q_heads;
  a.window = (int)(window < most ? window : most);
  a.sinks = (int)(sinks < most ? sinks : most);
  a.workspace = workspace;
  const bool e4m3 = cache->dtype == FP4_KV_E4M3;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return launched(who, decode ? fp4_launch_attention_decode(a, cache->dim, e4m3, s) : fp4_launch_attention_prompt(a, cache->dim, e4m3, s));
}

}  // namespace

extern "C" {

int fp4_rotate_quantize(const void* X, int64_t M, int64_t K, int64_t ldx, int block, int fmt, uint8_t* codes,
                        uint8_t* scales, float* tensor_scale, void* stream) {
  return quantize("fp4_rotate_quantize", X, M, K, ldx, block, fmt, FP4_SCALE_STANDARD, nullptr, codes, scales,
                  tensor_scale, stream);
}

int fp4_quantize_weights(const void* W, int64_t N, int64_t K, int64_t ldw, int block, int fmt, uint8_t* codes,
                         uint8_t* scales, float* tensor_scale, void* stream) {
  return quantize("fp4_quantize_weights", W, N, K, ldw, block, fmt, FP4_SCALE_STANDARD, nullptr, codes, scales,
                  tensor_scale, stream);
}

int fp4_rotate_quantize_ex(const void* X, int64_t M, int64_t K, int64_t ldx, int block, int fmt, int scale_rule,
                           const int8_t* signs, uint8_t* codes, uint8_t* scales, float* tensor_scale, void* stream) {
  return quantize("fp4_rotate_quantize_ex", X, M, K, ldx, block, fmt, scale_rule, signs, codes, scales, tensor_scale,
                  stream);
}

int fp4_quantize_weights_ex(const void* W, int64_t N, int64_t K, int64_t ldw, int block, int fmt, int scale_rule,
                            const int8_t* signs, uint8_t* codes, uint8_t* scales, float* tensor_scale, void* stream) {
  return quantize("fp4_quantize_weights_ex", W, N, K, ldw, block, fmt, scale_rule, signs, codes, scales,
                  tensor_scale, stream);
}

int fp4_linear(const uint8_t* Xq, const uint8_t* Xs, const float* x_ts, const uint8_t* Wq, const uint8_t* Ws,
               const float* w_ts, int64_t M, int64_t N, int64_t K, int fmt, void* Y, int y_dtype,
               void* stream) {
  const char* who = "fp4_linear";
  if (fmt != FP4_MXFP4 && fmt != FP4_NVFP4) return fail(FP4_E_FORMAT, "%s: unknown format %d", who, fmt);
  if (y_dtype != FP4_OUT_F32 && y_dtype != FP4_OUT_BF16)
    return fail(FP4_E_FORMAT, "%s: unknown output dtype %d", who, y_dtype);
  if (!Xq || !Xs || !Wq || !Ws || !Y) return fail(FP4_E_NULLPTR, "%s: operand pointers must be non-NULL", who);
  if (fmt == FP4_NVFP4 && (!x_ts || !w_ts))
    return fail(FP4_E_NULLPTR, "%s: NVFP4 needs both tensor scales", who);
  if (fmt == FP4_MXFP4 && (x_ts || w_ts))
    return fail(FP4_E_NULLPTR, "%s: tensor scales must be NULL for MXFP4", who);
  if (fmt == FP4_NVFP4 && (!aligned(x_ts, 4) || !aligned(w_ts, 4)))
    return fail(FP4_E_ALIGN, "%s: tensor scales must be 4-byte aligned", who);
  if (M < 1 || N < 1 || K < 128 || K % 128)
    return fail(FP4_E_SHAPE, "%s: need M, N >= 1 and K a positive multiple of 128 (M=%lld N=%lld K=%lld)", who,
                (long long)M, (long long)N, (long long)K);
  if (M > 0x7FFFFFFF || N > 0x7FFFFFFF || K > 0x7FFFFFFF || M * (K / 2) > ((int64_t)1 << 40) ||
      N * (K / 2) > ((int64_t)1 << 40))
    return fail(FP4_E_SHAPE, "%s: problem too large", who);
  if (((M + 127) / 128) * ((N + 127) / 128) > 0x7FFFFFFF)
    return fail(FP4_E_SHAPE, "%s: too many output tiles", who);
  if (!aligned(Xq, 16) || !aligned(Wq, 16) || !aligned(Xs, 4) || !aligned(Ws, 4) || !aligned(Y, 16))
    return fail(FP4_E_ALIGN, "%s: codes and Y must be 16-byte aligned, scales 4-byte aligned", who);
  hipStream_t st = static_cast<hipStream_t>(stream);
  hipError_t e = fmt == FP4_MXFP4
                     ? fp4_launch_gemm_mxfp4(Xq, Xs, Wq, Ws, M, N, K, Y, y_dtype == FP4_OUT_BF16, st)
                     : fp4_launch_gemm_nvfp4(Xq, Xs, x_ts, Wq, Ws, w_ts, M, N, K, Y, y_dtype == FP4_OUT_BF16, st);
  return launched(who, e);
}

int fp4_rotate_quantize_linear(const void* X, int64_t M, int64_t K, int64_t ldx, int block, const uint8_t* Wq,
                               const uint8_t* Ws, int64_t N, void* Y, int y_dtype, void* workspace,
                               size_t workspace_bytes, void* stream) {
  const char* who = "fp4_rotate_quantize_linear";
  int st = check_decode_step(who, X, M, K, ldx, block, Wq, Ws, N, Y, y_dtype);
  if (st != FP4_OK) return st;
  const size_t need = FP4_LINEAR_WORKSPACE_BYTES((size_t)M, (size_t)K);
  if (workspace && !aligned(workspace, 16)) return fail(FP4_E_ALIGN, "%s: workspace must be 16-byte aligned", who);
  if (workspace && workspace_bytes < need)
    return fail(FP4_E_SHAPE, "%s: workspace of %zu bytes, %zu needed", who, workspace_bytes, need);
  return decode_step(who, X, M, K, ldx, block, Wq, Ws, N, Y, y_dtype, static_cast<uint8_t*>(workspace), stream);
}

int fp4_rotate_quantize_linear_noalloc(const void* X, int64_t M, int64_t K, int64_t ldx, int block,
                                       const uint8_t* Wq, const uint8_t* Ws, int64_t N, void* Y, int y_dtype,
                                       void* stream) {
  const char* who = "fp4_rotate_quantize_linear_noalloc";
  int st = check_decode_step(who, X, M, K, ldx, block, Wq, Ws, N, Y, y_dtype);
  if (st != FP4_OK) return st;
  const size_t need = FP4_LINEAR_WORKSPACE_BYTES((size_t)M, (size_t)K);
  if (need > (size_t)FP4_DECODE_SCRATCH_BYTES)
    return fail(FP4_E_SHAPE, "%s: needs %zu bytes of workspace, the library's array holds %zu", who, need,
                (size_t)FP4_DECODE_SCRATCH_BYTES);
  uint8_t* ws = nullptr;
  const hipError_t e = fp4_decode_scratch(&ws);
  if (e != hipSuccess) return launched(who, e);
  return decode_step(who, X, M, K, ldx, block, Wq, Ws, N, Y, y_dtype, ws, stream);
}

int fp8_quantize(const void* X, int64_t M, int64_t K, int64_t ldx, uint8_t* codes, float* scales, void* stream) {
  const char* who = "fp8_quantize";
  const int st = check_fp8_rows(who, X, M, K, ldx, codes, scales);
  if (st != FP4_OK) return st;
  return launched(who, fp8_launch_quantize(static_cast<const uint16_t*>(X), M, K, ldx, codes, scales,
                                           static_cast<hipStream_t>(stream)));
}

int fp8_quantize_weights(const void* W, int64_t N, int64_t K, int64_t ldw, uint8_t* codes, float* scales,
                         void* stream) {
  const char* who = "fp8_quantize_weights";
  const int st = check_fp8_rows(who, W, N, K, ldw, codes, scales);
  if (st != FP4_OK) return st;
  return launched(who, fp8_launch_quantize_weights(static_cast<const uint16_t*>(W), N, K, ldw, codes, scales,
                                                   static_cast<hipStream_t>(stream)));
}

int fp8_add_rmsnorm_quantize(const void* X, int64_t M, int64_t K, int64_t ldx, const void* residual, int64_t ldr,
                             const void* weight, float eps, uint8_t* codes, float* scales, void* residual_out,
                             void* normed, void* stream) {
  const char* who = "fp8_add_rmsnorm_quantize";
  const int st = check_fp8_rows(who, X, M, K, ldx, codes, scales);
  if (st != FP4_OK) return st;
  if (!weight) return fail(FP4_E_NULLPTR, "%s: weight must be non-NULL", who);
  if ((residual == nullptr) != (residual_out == nullptr))
    return fail(FP4_E_NULLPTR, "%s: residual and residual_out go together", who);
  if (K > 65536) return fail(FP4_E_SHAPE, "%s: K=%lld above 65536", who, (long long)K);
  if (residual && (ldr < K || ldr > (int64_t)1 << 40))
    return fail(FP4_E_SHAPE, "%s: residual leading dimension %lld < K=%lld, or too large", who, (long long)ldr,
                (long long)K);
  if (residual && residual == residual_out && ldr != K)
    return fail(FP4_E_SHAPE, "%s: a residual written in place needs ldr == K", who);
  if (!(eps >= 0.f) || !__builtin_isfinite(eps)) return fail(FP4_E_SHAPE, "%s: eps must be finite and not negative", who);
  if (!aligned(weight, 16) || (residual && (!aligned(residual, 16) || ldr % 8 || !aligned(residual_out, 16))) ||
      (normed && !aligned(normed, 16)))
    return fail(FP4_E_ALIGN, "%s: weight, residual and outputs must be 16-byte aligned, ldr %% 8 == 0", who);
  return launched(who, fp8_launch_add_rmsnorm_quantize(
                           static_cast<const uint16_t*>(X), M, K, ldx, static_cast<const uint16_t*>(residual), ldr,
                           static_cast<const uint16_t*>(weight), eps, codes, scales,
                           static_cast<uint16_t*>(residual_out), static_cast<uint16_t*>(normed),
                           static_cast<hipStream_t>(stream)));
}

int fp8_linear(const uint8_t* Xq, const float* Xs, const uint8_t* Wq, const float* Ws, int64_t M, int64_t N, int64_t K,
               void* Y, void* stream) {
  const char* who = "fp8_linear";
  if (!Xq || !Xs || !Wq || !Ws || !Y) return fail(FP4_E_NULLPTR, "%s: operand pointers must be non-NULL", who);
  if (M < 1 || N < 1 || K < 128 || K % 128)
    return fail(FP4_E_SHAPE, "%s: need M, N >= 1 and K a positive multiple of 128 (M=%lld N=%lld K=%lld)", who,
                (long long)M, (long long)N, (long long)K);
  if (M > 0x7FFFFFFF || N > 0x7FFFFFFF || K > (1 << 23) || M * K > ((int64_t)1 << 40) || N * K > ((int64_t)1 << 40) ||
      ((M + 127) / 128) * ((N + 63) / 64) > 0x7FFFFFFF)
    return fail(FP4_E_SHAPE, "%s: problem too large", who);
  if (!aligned(Xq, 16) || !aligned(Wq, 16) || !aligned(Xs, 4) || !aligned(Ws, 4) || !aligned(Y, 16))
    return fail(FP4_E_ALIGN, "%s: codes and Y must be 16-byte aligned, scales 4-byte aligned", who);
  return launched(who, fp8_launch_linear(Xq, Xs, Wq, Ws, M, N, K, static_cast<uint16_t*>(Y),
                                         static_cast<hipStream_t>(stream)));
}

int fp4_moe_route(const void* X, int64_t T, int64_t D, int64_t ldx, const void* Wr, int64_t E, int k, int renormalize,
                  int* ids, float* weights, void* workspace, size_t workspace_bytes, void* stream) {
  const char* who = "fp4_moe_route";
  if (!X || !Wr || !ids || !weights || !workspace) return fail(FP4_E_NULLPTR, "%s: pointers must be non-NULL", who);
  if (T < 1 || T > FP4_MOE_ROUTE_MAX_TOKENS || D < 128 || D % 128 || D > (1 << 24) || E < 1 || E > 1024)
    return fail(FP4_E_SHAPE, "%s: need 1 <= T <= %d, D a positive multiple of 128 up to %d, 1 <= E <= 1024 (T=%lld D=%lld E=%lld)",
                who, FP4_MOE_ROUTE_MAX_TOKENS, 1 << 24, (long long)T, (long long)D, (long long)E);
  if (k < 1 || k > FP4_MOE_MAX_TOPK || k > E)
    return fail(FP4_E_SHAPE, "%s: k=%d not in 1 .. min(E, %d)", who, k, FP4_MOE_MAX_TOPK);
  if (ldx < D || ldx > (int64_t)1 << 40) return fail(FP4_E_SHAPE, "%s: leading dimension %lld < D", who, (long long)ldx);
  if (workspace_bytes < FP4_MOE_ROUTE_WORKSPACE_BYTES(T, E))
    return fail(FP4_E_SHAPE, "%s: workspace of %zu bytes, %zu needed", who, workspace_bytes,
                FP4_MOE_ROUTE_WORKSPACE_BYTES(T, E));
  if (!aligned(X, 16) || ldx % 8 || !aligned(Wr, 16) || !aligned(workspace, 16) || !aligned(ids, 4) || !aligned(weights, 4))
    return fail(FP4_E_ALIGN, "%s: X, Wr and workspace must be 16-byte aligned, ldx %% 8 == 0, ids and weights 4-byte aligned",
                who);
  return launched(who, fp4_launch_moe_route(static_cast<const uint16_t*>(X), T, D, ldx, static_cast<const uint16_t*>(Wr), E,
                                            k, renormalize, static_cast<float*>(workspace), ids, weights,
                                            static_cast<hipStream_t>(stream)));
}

int fp4_moe_experts(const void* X, int64_t T, int64_t D, int64_t ldx, const int* ids, const float* weights, int k,
                    int64_t E, int64_t I, int block, const uint8_t* W13q, const uint8_t* W13s, const uint8_t* W2q,
                    const uint8_t* W2s, void* Y, void* workspace, size_t workspace_bytes, void* stream) {
  const char* who = "fp4_moe_experts";
  if (block != 16 && block != 32 && block != 64 && block != 128)
    return fail(FP4_E_BLOCK, "%s: Hadamard block %d not in {16, 32, 64, 128}", who, block);
  if (!X || !ids || !weights || !W13q || !W13s || !W2q || !W2s || !Y || !workspace)
    return fail(FP4_E_NULLPTR, "%s: pointers must be non-NULL", who);
  if (T < 1 || T > FP4_MOE_MAX_TOKENS || k < 1 || k > FP4_MOE_MAX_TOPK)
    return fail(FP4_E_SHAPE, "%s: need 1 <= T <= %d and 1 <= k <= %d (T=%lld k=%d)", who, FP4_MOE_MAX_TOKENS,
                FP4_MOE_MAX_TOPK, (long long)T, k);
  if (E < 1 || E > 1024 || D < 128 || D % 128 || D > 65536 || I < 128 || I % 128 || I > 65536)
    return fail(FP4_E_SHAPE, "%s: need 1 <= E <= 1024, D and I multiples of 128 up to 65536 (E=%lld D=%lld I=%lld)", who,
                (long long)E, (long long)D, (long long)I);
  if (ldx < D || ldx > (int64_t)1 << 40) return fail(FP4_E_SHAPE, "%s: leading dimension %lld < D", who, (long long)ldx);
  if (workspace_bytes < FP4_MOE_WORKSPACE_BYTES(T, k, D, I))
    return fail(FP4_E_SHAPE, "%s: workspace of %zu bytes, %zu needed", who, workspace_bytes,
                FP4_MOE_WORKSPACE_BYTES(T, k, D, I));
  if (!aligned(X, 16) || ldx % 8 || !aligned(W13q, 16) || !aligned(W13s, 16) || !aligned(W2q, 16) || !aligned(W2s, 16) ||
      !aligned(Y, 16) || !aligned(workspace, 16) || !aligned(ids, 4) || !aligned(weights, 4))
    return fail(FP4_E_ALIGN, "%s: X, matrices, Y and workspace must be 16-byte aligned, ldx %% 8 == 0, ids and weights 4-byte "
                "aligned", who);
  return launched(who, fp4_launch_moe_experts(static_cast<const uint16_t*>(X), T, D, ldx, ids, weights, k, E, I, block,
                                              W13q, W13s, W2q, W2s, static_cast<uint16_t*>(Y),
                                              static_cast<uint8_t*>(workspace), static_cast<hipStream_t>(stream)));
}

int fp4_kv_append(const fp4_kv_cache* cache, const int* starts, int64_t T, const void* K, int64_t k_row, int64_t k_head,
                  const void* V, int64_t v_row, int64_t v_head, const void* Q, int64_t q_row, int64_t q_head, int q_heads,
                  void* Q_out, int64_t out_row, int64_t out_head, const float* freqs, int rotated, int interleaved,
                  const int* positions, const int* axes, int n_axes, void* stream) {
  const char* who = "fp4_kv_append";
  if (!K || !V) return fail(FP4_E_NULLPTR, "%s: K and V must be non-NULL", who);
  if ((Q != nullptr) != (Q_out != nullptr)) return fail(FP4_E_NULLPTR, "%s: Q and Q_out go together", who);
  if (!freqs && (rotated || positions || axes || Q))
    return fail(FP4_E_NULLPTR, "%s: rotated, positions, axes and Q need freqs", who);
  if (axes && !positions) return fail(FP4_E_NULLPTR, "%s: axes need positions", who);
  Fp4AppendArgs a{};
  int st = check_cache(who, cache, Q ? q_heads : 1, &a.cache);
  if (st != FP4_OK) return st;
  if (Q ? q_heads < 1 || q_heads > 1024 : q_heads != 0) return fail(FP4_E_SHAPE, "%s: q_heads=%d not in 1 .. 1024, or 0 without Q", who, q_heads);
  if (T < 1 || T > (1 << 24) || T * (q_heads + 2 * cache->heads) > (1 << 30))
    return fail(FP4_E_SHAPE, "%s: need 1 <= T <= 2^24 and T * (q_heads + 2 * heads) <= 2^30 (T=%lld)", who, (long long)T);
  if (!starts && T != cache->batch)
    return fail(FP4_E_SHAPE, "%s: without starts T must be the batch, got %lld and %lld", who, (long long)T, (long long)cache->batch);
  if (rotated < 0 || rotated > cache->dim || rotated % 16 || (freqs && !rotated))
    return fail(FP4_E_SHAPE, "%s: rotated=%d is no positive multiple of 16 up to dim (0 without freqs)", who, rotated);
  if (positions ? n_axes < 1 || n_axes > 16 : n_axes != 0)
    return fail(FP4_E_SHAPE, "%s: n_axes=%d not in 1 .. 16, or 0 without positions", who, n_axes);
  st = check_heads(who, "K", K, k_row, k_head, cache->dim);
  if (st == FP4_OK) st = check_heads(who, "V", V, v_row, v_head, cache->dim);
  if (st == FP4_OK && Q) st = check_heads(who, "Q", Q, q_row, q_head, cache->dim);
  if (st == FP4_OK && Q) st = check_heads(who, "Q_out", Q_out, out_row, out_head, cache->dim);
  if (st != FP4_OK) return st;
  if (Q && Q == Q_out && (q_row != out_row || q_head != out_head))
    return fail(FP4_E_SHAPE, "%s: queries rotated in place need the same strides", who);
  if (!aligned(starts, 4) || !aligned(freqs, 4) || !aligned(positions, 4) || !aligned(axes, 4))
    return fail(FP4_E_ALIGN, "%s: starts, freqs, positions and axes must be 4-byte aligned", who);
  a.starts = starts;
  a.q = static_cast<const uint16_t*>(Q);
  a.k = static_cast<const uint16_t*>(K);
  a.v = static_cast<const uint16_t*>(V);
  a.q_out = static_cast<uint16_t*>(Q_out);
  a.q_token = q_row;
  a.q_head = q_head;
  a.k_token = k_row;
  a.k_head = k_head;
  a.v_token = v_row;
  a.v_head = v_head;
  a.out_token = out_row;
  a.out_head = out_head;
  a.freqs = freqs;
  a.positions = positions;
  a.axes = axes;
  a.T = (int)T;
  a.q_heads = q_heads;
  a.half = rotated / 2;
  a.naxes = n_axes;
  a.interleaved = interleaved != 0;
  return launched(who, fp4_launch_kv_append(a, cache->dim, cache->dtype == FP4_KV_E4M3, static_cast<hipStream_t>(stream)));
}

int fp4_attention_decode(const fp4_kv_cache* cache, const void* Q, int64_t q_row, int64_t q_head, int q_heads, float scale,
                         int64_t window, int64_t sinks, void* Out, void* workspace, size_t workspace_bytes, void* stream) {
  return attention("fp4_attention_decode", cache, nullptr, 0, Q, q_row, q_head, q_heads, scale, window, sinks, Out, workspace,
                   workspace_bytes, true, stream);
}

int fp4_attention_prompt(const fp4_kv_cache* cache, const int* starts, int64_t T, const void* Q, int64_t q_row, int64_t q_head,
                         int q_heads, float scale, int64_t window, int64_t sinks, void* Out, void* workspace,
                         size_t workspace_bytes, void* stream) {
  return attention("fp4_attention_prompt", cache, starts, T, Q, q_row, q_head, q_heads, scale, window, sinks, Out, workspace,
                   workspace_bytes, false, stream);
}

const char* fp4_last_error(void) { return g_err; }

int fp4_abi_version(void) { return FP4_ABI_VERSION; }

}  // extern "C"
