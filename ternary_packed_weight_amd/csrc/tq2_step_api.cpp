// C ABI of the feed-forward half of a decode step and of the model's answer
// (declared in include/tq2.h): argument validation, then launches on the
// caller's stream.  Every check happens before any launch.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "tq2.h"
#include "tq2_step.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

// A byte range of device memory; empty where the pointer is null.  Or rows of
// one, `row` bytes long and `stride` apart: two of the same stride may lie
// between each other's rows (columns of one matrix).
struct Span {
  uintptr_t at = 0;
  uint64_t bytes = 0, row = 0, stride = 0;
  Span() = default;
  Span(const void* p, uint64_t n, uint64_t row = 0, uint64_t stride = 0)
      : at((uintptr_t)p), bytes(p ? n : 0), row(row), stride(stride) {}
  bool meets(const Span& o) const {
    if (!bytes || !o.bytes || at >= o.at + o.bytes || o.at >= at + bytes) return false;
    if (!stride || stride != o.stride) return true;
    // a place of the other's rows in the period that begins with a row of these
    const uint64_t d = o.at >= at ? (o.at - at) % stride : (stride - (at - o.at) % stride) % stride;
    return d < row || d + o.row > stride;
  }
};

// No output meets another or an input.
template <int O, int I>
bool apart(const Span (&outs)[O], const Span (&ins)[I]) {
  for (int o = 0; o < O; ++o) {
    for (int p = 0; p < o; ++p)
      if (outs[o].meets(outs[p])) return false;
    for (const Span& i : ins)
      if (outs[o].meets(i)) return false;
  }
  return true;
}

bool is_dtype(int32_t d) { return d >= TQ2_F16 && d <= TQ2_F32; }
int64_t size_of(int32_t dtype) { return dtype == TQ2_F32 ? 4 : 2; }
int32_t hip_status(hipError_t e) { return e == hipSuccess ? TQ2_OK : TQ2_ERR_HIP; }

constexpr int64_t kMost = (int64_t)1 << 40;  // elements of an array
constexpr int64_t kMostTokens = 1 << 26;     // rows of a norm
constexpr int64_t kMostGated = 1 << 26;      // rows of a gated matrix
constexpr int64_t kMostRows = 1 << 22;       // rows of logits: a grid holds less than 2^32 threads
constexpr int64_t kMostVocab = 1 << 24;
static_assert(TQ2_MAX_TOP == tq2::kMaxTop, "what the kernels' lists hold");

#define TQ2_TRY(expr)              \
  do {                             \
    const int32_t st_ = (expr);    \
    if (st_ != TQ2_OK) return st_; \
  } while (0)

// Strided rows [T][D] of 16-byte pieces: the checks of pointer and stride, and the bytes they span.
int32_t check_rows(const void* p, int64_t stride, int64_t T, int64_t D, int64_t size, uint64_t* bytes) {
  if (!p || stride < 0) return TQ2_ERR_ARG;
  if (T == 1) stride = 0;
  if (stride > kMost / T) return TQ2_ERR_SHAPE;
  if (!aligned(p, 16) || stride * size % 16) return TQ2_ERR_ALIGN;
  *bytes = (uint64_t)(((T - 1) * stride + D) * size);
  return TQ2_OK;
}

// Both forms of the norm: `q` and `scales` or `s` for int8, `out` else.
int32_t norm(const void* x, int64_t x_stride, int32_t x_dtype, const void* residual, int64_t r_stride, int32_t r_dtype,
             void* h_out, int64_t T, int32_t D, const float* weight, float eps, int32_t out_dtype, void* out,
             float* scales, float s, tq2_stream_t stream) {
  const bool int8 = out_dtype == tq2::kOutI8;
  if (T < 0 || !is_dtype(x_dtype) || (residual && !is_dtype(r_dtype)) || (!int8 && !is_dtype(out_dtype)))
    return TQ2_ERR_ARG;
  if (!(eps >= 0.0f) || isinf(eps) || (!residual && h_out)) return TQ2_ERR_ARG;
  // (no rows: the scales' pointer may be null with a scale for each)
  if (int8 && !scales && !(isfinite(s) && s > 0.0f) && (T || s != 0.0f)) return TQ2_ERR_SCALE;
  if (int8 && scales && s != 0.0f) return TQ2_ERR_ARG;
  if (D < 8 || D > TQ2_MAX_K || D % 8 || T > kMostTokens) return TQ2_ERR_SHAPE;
  if (T == 0) return TQ2_OK;
  if (!out) return TQ2_ERR_ARG;
  uint64_t xb = 0, rb = 0;
  TQ2_TRY(check_rows(x, x_stride, T, D, size_of(x_dtype), &xb));
  if (residual) TQ2_TRY(check_rows(residual, r_stride, T, D, size_of(r_dtype), &rb));
  // rows of the sum may not lie in each other, nor may a row of the residual that a sum replaces be read again
  if (h_out && T > 1 && r_stride < D) return TQ2_ERR_ARG;
  if (!aligned(out, 16) || !aligned(h_out, 16) || !aligned(weight, 16) || !aligned(scales, 4)) return TQ2_ERR_ALIGN;
  const uint64_t xs = size_of(x_dtype), rs = size_of(r_dtype);
  const Span sum(h_out, rb, D * rs, T > 1 ? r_stride * rs : 0);
  const Span outs[3] = {Span(out, (uint64_t)(T * D) * (int8 ? 1 : size_of(out_dtype))), sum, Span(scales, (uint64_t)T * 4)};
  const Span ins[3] = {Span(x, xb, D * xs, T > 1 ? x_stride * xs : 0),
                       Span(h_out == residual ? nullptr : residual, rb, D * rs, T > 1 ? r_stride * rs : 0),
                       Span(weight, (uint64_t)D * 4)};
  if (!apart(outs, ins)) return TQ2_ERR_ARG;
  tq2::NormArgs a{};
  a.x = x, a.residual = residual, a.h_out = h_out, a.weight = weight, a.out = out, a.scales = scales;
  a.x_stride = T == 1 ? 0 : x_stride, a.r_stride = T == 1 ? 0 : r_stride, a.T = T, a.D = D, a.eps = eps, a.s = s;
  (void)hipGetLastError();
  return hip_status(tq2::launch_add_rms_norm(a, x_dtype, r_dtype, out_dtype, (hipStream_t)stream));
}

int32_t gated_shape(int64_t N, int64_t K, int64_t M, int64_t most_k) {
  if (N < 1 || M < 1) return TQ2_ERR_ARG;
  if (K < TQ2_BLOCK || K % TQ2_BLOCK || K > most_k || M > TQ2_MAX_TOKENS) return TQ2_ERR_SHAPE;
  if (N > kMostGated || N > kMost / K || N > kMost / M) return TQ2_ERR_SHAPE;
  return TQ2_OK;
}

int32_t gated(bool int8, const uint8_t* codes_g, const uint16_t* scales_g, const uint8_t* codes_u,
              const uint16_t* scales_u, int64_t N, int64_t K, const void* x, int64_t M, float s, const float* x_scales,
              void* h, int32_t h_dtype, void* ws, size_t ws_bytes, tq2_stream_t stream) {
  TQ2_TRY(gated_shape(N, K, M, int8 ? TQ2_I8_MAX_K : TQ2_MAX_K));
  if (!codes_g || !scales_g || !codes_u || !scales_u || !x || !h || !is_dtype(h_dtype)) return TQ2_ERR_ARG;
  if (int8 && !x_scales && !(isfinite(s) && s > 0.0f)) return TQ2_ERR_SCALE;
  if (int8 && x_scales && s != 0.0f) return TQ2_ERR_ARG;
  if (!aligned(codes_g, 16) || !aligned(codes_u, 16) || !aligned(scales_g, 2) || !aligned(scales_u, 2) ||
      !aligned(x, 16) || !aligned(x_scales, 4) || !aligned(h, 16))
    return TQ2_ERR_ALIGN;
  const uint64_t cb = (uint64_t)(N * (K / 4)), sb = (uint64_t)(N * (K / TQ2_BLOCK) * 2);
  const Span outs[1] = {Span(h, (uint64_t)(M * N * size_of(h_dtype)))};
  const Span ins[6] = {Span(codes_g, cb), Span(codes_u, cb), Span(scales_g, sb), Span(scales_u, sb),
                       Span(x, (uint64_t)(M * K * (int8 ? 1 : 2))), Span(x_scales, (uint64_t)M * 4)};
  if (!apart(outs, ins)) return TQ2_ERR_ARG;
  if (const size_t need = tq2::gated_workspace_bytes(K, M, int8)) {
    if (!ws || ws_bytes < need || !aligned(ws, 256)) return TQ2_ERR_WORKSPACE;
    const Span w[1] = {Span(ws, need)};
    if (!apart(w, ins) || !apart(w, outs)) return TQ2_ERR_WORKSPACE;
  }
  tq2::GatedArgs a{};
  a.codes[0] = codes_g, a.codes[1] = codes_u, a.scales[0] = scales_g, a.scales[1] = scales_u;
  a.x = x, a.x_scales = x_scales, a.s = s, a.h = h, a.N = N, a.K = K, a.M = M, a.pieces = ws;
  (void)hipGetLastError();
  return hip_status(tq2::launch_gated(a, int8, h_dtype, (hipStream_t)stream));
}

}  // namespace

extern "C" {

int32_t tq2_add_rms_norm(const void* x, int64_t x_stride, int32_t x_dtype, const void* residual, int64_t r_stride,
                         int32_t r_dtype, void* h_out, int64_t T, int32_t D, const float* weight, float eps, void* out,
                         int32_t out_dtype, tq2_stream_t stream) {
  if (!is_dtype(out_dtype)) return TQ2_ERR_ARG;
  return norm(x, x_stride, x_dtype, residual, r_stride, r_dtype, h_out, T, D, weight, eps, out_dtype, out, nullptr,
              0.0f, stream);
}

int32_t tq2_add_rms_norm_i8(const void* x, int64_t x_stride, int32_t x_dtype, const void* residual, int64_t r_stride,
                            int32_t r_dtype, void* h_out, int64_t T, int32_t D, const float* weight, float eps, float s,
                            int8_t* x_q, float* x_scales, tq2_stream_t stream) {
  return norm(x, x_stride, x_dtype, residual, r_stride, r_dtype, h_out, T, D, weight, eps, tq2::kOutI8, x_q, x_scales, s,
              stream);
}

size_t tq2_gemm_gate_up_silu_workspace_bytes(int64_t N, int64_t K, int64_t M) {
  return gated_shape(N, K, M, TQ2_MAX_K) == TQ2_OK ? tq2::gated_workspace_bytes(K, M, false) : (size_t)-1;
}

int32_t tq2_gemm_gate_up_silu(const uint8_t* codes_g, const uint16_t* scales_g, const uint8_t* codes_u,
                              const uint16_t* scales_u, int64_t N, int64_t K, const uint16_t* x, int64_t M, void* h,
                              int32_t h_dtype, void* ws, size_t ws_bytes, tq2_stream_t stream) {
  return gated(false, codes_g, scales_g, codes_u, scales_u, N, K, x, M, 1.0f, nullptr, h, h_dtype, ws, ws_bytes, stream);
}

size_t tq2_gemm_i8q_gate_up_silu_workspace_bytes(int64_t N, int64_t K, int64_t M) {
  return gated_shape(N, K, M, TQ2_I8_MAX_K) == TQ2_OK ? tq2::gated_workspace_bytes(K, M, true) : (size_t)-1;
}

int32_t tq2_gemm_i8q_gate_up_silu(const uint8_t* codes_g, const uint16_t* scales_g, const uint8_t* codes_u,
                                  const uint16_t* scales_u, int64_t N, int64_t K, const int8_t* x_q, int64_t M, float s,
                                  const float* x_scales, void* h, int32_t h_dtype, void* ws, size_t ws_bytes,
                                  tq2_stream_t stream) {
  return gated(true, codes_g, scales_g, codes_u, scales_u, N, K, x_q, M, s, x_scales, h, h_dtype, ws, ws_bytes, stream);
}

size_t tq2_token_logprobs_workspace_bytes(int64_t T, int64_t V, int32_t top) {
  if (T < 0 || V < 1 || top < 0 || T > kMostRows || V > kMostVocab || top > TQ2_MAX_TOP || top > V) return (size_t)-1;
  return T ? tq2::logprob_workspace_bytes(T, V, top) : 0;
}

int32_t tq2_token_logprobs(const void* logits, int64_t stride, int32_t dtype, int64_t T, int64_t V, float scale,
                           const int64_t* tokens, float* logprobs, float* entropy, int32_t top, int64_t* top_tokens,
                           float* top_logprobs, void* ws, size_t ws_bytes, tq2_stream_t stream) {
  if (T < 0 || V < 1 || top < 0 || stride < 0 || !is_dtype(dtype)) return TQ2_ERR_ARG;
  if (!(isfinite(scale) && scale > 0.0f)) return TQ2_ERR_SCALE;
  const size_t need = tq2_token_logprobs_workspace_bytes(T, V, top);
  if (need == (size_t)-1) return TQ2_ERR_SHAPE;
  if (T == 0) return TQ2_OK;
  if (!logits || (!tokens != !logprobs) || (!tokens && !entropy && !top)) return TQ2_ERR_ARG;
  if (top ? !top_tokens || !top_logprobs : top_tokens || top_logprobs) return TQ2_ERR_ARG;
  if (T == 1) stride = 0;
  if (stride > kMost / T) return TQ2_ERR_SHAPE;
  if (!aligned(logits, size_of(dtype)) || !aligned(tokens, 8) || !aligned(logprobs, 4) || !aligned(entropy, 4) ||
      !aligned(top_tokens, 8) || !aligned(top_logprobs, 4))
    return TQ2_ERR_ALIGN;
  const Span outs[4] = {Span(logprobs, (uint64_t)T * 4), Span(entropy, (uint64_t)T * 4),
                        Span(top_tokens, (uint64_t)(T * top) * 8), Span(top_logprobs, (uint64_t)(T * top) * 4)};
  const Span ins[2] = {Span(logits, (uint64_t)(((T - 1) * stride + V) * size_of(dtype))), Span(tokens, (uint64_t)T * 8)};
  if (!apart(outs, ins)) return TQ2_ERR_ARG;
  if (need) {
    if (!ws || ws_bytes < need || !aligned(ws, 256)) return TQ2_ERR_WORKSPACE;
    const Span w(ws, need);
    for (const Span& o : outs)
      if (w.meets(o)) return TQ2_ERR_WORKSPACE;
    for (const Span& i : ins)
      if (w.meets(i)) return TQ2_ERR_WORKSPACE;
  }
  tq2::LogprobArgs a{};
  a.logits = logits, a.stride = stride, a.T = T, a.V = V, a.scale = scale, a.tokens = tokens, a.logprobs = logprobs;
  a.entropy = entropy, a.top_tokens = top_tokens, a.top_logprobs = top_logprobs, a.top = top, a.ws = (uint8_t*)ws;
  (void)hipGetLastError();
  return hip_status(tq2::launch_token_logprobs(a, dtype, (hipStream_t)stream));
}

}  // extern "C"
