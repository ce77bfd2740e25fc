// C ABI of the attention half of a decode step (declared in include/tq2.h):
// argument validation, then launches on the caller's stream.  Every check
// happens before any launch.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "tq2.h"
#include "tq2_kv4.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

// A byte range of device memory; empty where the pointer is null.
struct Span {
  uintptr_t at;
  uint64_t bytes;
  Span(const void* p, uint64_t n) : at((uintptr_t)p), bytes(p ? n : 0) {}
  bool meets(const Span& o) const { return bytes && o.bytes && at < o.at + o.bytes && o.at < at + bytes; }
};

int64_t size_of(int32_t dtype) { return dtype == TQ2_F32 ? 4 : 2; }

constexpr int64_t kMost = (int64_t)1 << 40;  // elements of an array
constexpr int64_t kMostTokens = 1 << 26;     // of a call: a grid holds less than 2^32 threads

// Strided heads [T][H][D]: the checks of pointer and strides, and the bytes they span.
int32_t check_heads(const void* p, int64_t ts, int64_t hs, int64_t T, int64_t H, int64_t D, int64_t size,
                    uint64_t* bytes) {
  if (!p) return TQ2_ERR_ARG;
  if (ts < 0 || hs < 0) return TQ2_ERR_ARG;
  if (T == 1) ts = 0;
  if (H == 1) hs = 0;
  if (ts > kMost / T || hs > kMost / H) return TQ2_ERR_SHAPE;
  if (!aligned(p, 16) || ts * size % 16 || hs * size % 16) return TQ2_ERR_ALIGN;
  *bytes = (uint64_t)(((T - 1) * ts + (H - 1) * hs + D) * size);
  return TQ2_OK;
}

int32_t check_cache_shape(int64_t pages, int32_t P, int32_t Hk, int32_t D) {
  if (pages < 1 || Hk < 1) return TQ2_ERR_ARG;
  if (P < 32 || P > 4096 || (P & (P - 1)) || (D != 64 && D != 128 && D != 256)) return TQ2_ERR_SHAPE;
  if (Hk > 4096 || pages > kMost / P || pages > kMost / (tq2::kv4_block_bytes(P, D) * Hk)) return TQ2_ERR_SHAPE;
  return TQ2_OK;
}

uint64_t cache_bytes(int64_t pages, int32_t P, int32_t Hk, int32_t D) {
  return (uint64_t)(pages * Hk * tq2::kv4_block_bytes(P, D));
}

int32_t hip_status(hipError_t e) { return e == hipSuccess ? TQ2_OK : TQ2_ERR_HIP; }

#define TQ2_TRY(expr)              \
  do {                             \
    const int32_t st_ = (expr);    \
    if (st_ != TQ2_OK) return st_; \
  } while (0)

bool attn_sizes_ok(int64_t T, int32_t Hq, int32_t Hk, int32_t D, int32_t P, int32_t width, int32_t B,
                   int32_t max_q) {
  if (T < 0 || T > kMostTokens || Hq < 1 || Hk < 1 || width < 1 || B < 1 || max_q < 1) return false;
  if (check_cache_shape(1, P, Hk, D) != TQ2_OK || Hq % Hk || Hq > 65536) return false;
  if (T > kMost / ((int64_t)Hq * D) || (int64_t)width * P > INT32_MAX) return false;
  const int64_t rows = (int64_t)B * max_q;  // workgroups and rows are counted in 32 bits
  if (rows > INT32_MAX / Hq || T > rows) return false;
  return tq2::plan_kv4_attn(Hq, Hk, D, P, width, B, max_q, 0).grid < ((int64_t)1 << 24);  // workgroups of 256
}

}  // namespace

extern "C" {

int32_t tq2_qk_norm_rope(const void* q, int64_t q_token_stride, int64_t q_head_stride, int32_t Hq, const void* k,
                         int64_t k_token_stride, int64_t k_head_stride, int32_t Hk, int32_t in_dtype, int64_t T,
                         int32_t D, const float* q_weight, const float* k_weight, float eps, const int32_t* positions,
                         const float* inv_freq, int32_t rot, int32_t interleaved, void* q_out, void* k_out,
                         int32_t out_dtype, tq2_stream_t stream) {
  if (Hq < 0 || Hk < 0 || (Hq == 0 && Hk == 0) || T < 0) return TQ2_ERR_ARG;
  if (in_dtype < TQ2_F16 || in_dtype > TQ2_F32 || out_dtype < TQ2_F16 || out_dtype > TQ2_F32) return TQ2_ERR_ARG;
  if (interleaved != 0 && interleaved != 1) return TQ2_ERR_ARG;
  if (!(eps >= 0.0f) || isinf(eps)) return TQ2_ERR_ARG;
  if (D < 16 || D > 512 || D % 16 || rot < 0 || rot > D || rot % 16) return TQ2_ERR_SHAPE;
  if (Hq > 65536 || Hk > 65536 || T > kMostTokens) return TQ2_ERR_SHAPE;
  if (T == 0) return TQ2_OK;
  const int64_t in = size_of(in_dtype), out = size_of(out_dtype);
  uint64_t qb = 0, kb = 0;
  if (Hq) TQ2_TRY(check_heads(q, q_token_stride, q_head_stride, T, Hq, D, in, &qb));
  if (Hk) TQ2_TRY(check_heads(k, k_token_stride, k_head_stride, T, Hk, D, in, &kb));
  if ((Hq && !q_out) || (Hk && !k_out) || (rot && (!positions || !inv_freq))) return TQ2_ERR_ARG;
  if ((Hq && !aligned(q_out, 16)) || (Hk && !aligned(k_out, 16)) || !aligned(q_weight, 4) || !aligned(k_weight, 4) ||
      !aligned(positions, 4) || !aligned(inv_freq, 4))
    return TQ2_ERR_ALIGN;
  const Span outs[2] = {Span(Hq ? q_out : nullptr, (uint64_t)(T * Hq * D * out)),
                        Span(Hk ? k_out : nullptr, (uint64_t)(T * Hk * D * out))};
  const Span ins[6] = {Span(Hq ? q : nullptr, qb),
                       Span(Hk ? k : nullptr, kb),
                       Span(Hq ? q_weight : nullptr, (uint64_t)D * 4),
                       Span(Hk ? k_weight : nullptr, (uint64_t)D * 4),
                       Span(rot ? positions : nullptr, (uint64_t)T * 4),
                       Span(rot ? inv_freq : nullptr, (uint64_t)rot * 2)};
  if (outs[0].meets(outs[1])) return TQ2_ERR_ARG;
  for (const Span& o : outs)
    for (const Span& i : ins)
      if (o.meets(i)) return TQ2_ERR_ARG;
  tq2::RopeArgs a{};
  a.q = q, a.k = k, a.q_out = q_out, a.k_out = k_out;
  a.q_weight = q_weight, a.k_weight = k_weight, a.inv_freq = inv_freq, a.positions = positions;
  a.q_ts = q_token_stride, a.q_hs = q_head_stride, a.k_ts = k_token_stride, a.k_hs = k_head_stride;
  a.T = T, a.Hq = Hq, a.Hk = Hk, a.D = D, a.rot = rot, a.interleaved = interleaved, a.eps = eps;
  (void)hipGetLastError();
  return hip_status(tq2::launch_qk_norm_rope(a, in_dtype, out_dtype, (hipStream_t)stream));
}

size_t tq2_kv4_page_bytes(int32_t P, int32_t Hk, int32_t D) {
  if (check_cache_shape(1, P, Hk, D) != TQ2_OK) return 0;
  return (size_t)cache_bytes(1, P, Hk, D);
}

int32_t tq2_kv4_store(uint8_t* cache, int64_t pages, int32_t P, int32_t Hk, int32_t D, const void* k,
                      int64_t k_token_stride, int64_t k_head_stride, const void* v, int64_t v_token_stride,
                      int64_t v_head_stride, int32_t dtype, const int64_t* slots, int64_t T, tq2_stream_t stream) {
  TQ2_TRY(check_cache_shape(pages, P, Hk, D));
  if (dtype < TQ2_F16 || dtype > TQ2_F32 || T < 0) return TQ2_ERR_ARG;
  if (T > kMostTokens || T * Hk > kMostTokens) return TQ2_ERR_SHAPE;
  if (T == 0) return TQ2_OK;
  if (!cache || !slots) return TQ2_ERR_ARG;
  uint64_t kb = 0, vb = 0;
  TQ2_TRY(check_heads(k, k_token_stride, k_head_stride, T, Hk, D, size_of(dtype), &kb));
  TQ2_TRY(check_heads(v, v_token_stride, v_head_stride, T, Hk, D, size_of(dtype), &vb));
  if (!aligned(cache, 16) || !aligned(slots, 8)) return TQ2_ERR_ALIGN;
  const Span out(cache, cache_bytes(pages, P, Hk, D));
  if (out.meets(Span(k, kb)) || out.meets(Span(v, vb)) || out.meets(Span(slots, (uint64_t)T * 8))) return TQ2_ERR_ARG;
  tq2::Kv4StoreArgs a{};
  a.k = k, a.v = v, a.cache = cache, a.slots = slots;
  a.k_ts = k_token_stride, a.k_hs = k_head_stride, a.v_ts = v_token_stride, a.v_hs = v_head_stride;
  a.T = T, a.pages = pages, a.Hk = Hk, a.D = D, a.P = P;
  (void)hipGetLastError();
  return hip_status(tq2::launch_kv4_store(a, dtype, (hipStream_t)stream));
}

int32_t tq2_kv4_load(const uint8_t* cache, int64_t pages, int32_t P, int32_t Hk, int32_t D, const int64_t* slots,
                     int64_t T, void* k, void* v, int32_t dtype, tq2_stream_t stream) {
  TQ2_TRY(check_cache_shape(pages, P, Hk, D));
  if (dtype < TQ2_F16 || dtype > TQ2_F32 || T < 0) return TQ2_ERR_ARG;
  if (T > kMostTokens || T * Hk > kMostTokens) return TQ2_ERR_SHAPE;
  if (T == 0) return TQ2_OK;
  if (!cache || !slots || (!k && !v)) return TQ2_ERR_ARG;
  if (!aligned(cache, 16) || !aligned(slots, 8) || !aligned(k, 16) || !aligned(v, 16)) return TQ2_ERR_ALIGN;
  const uint64_t bytes = (uint64_t)(T * Hk * D * size_of(dtype));
  const Span ins[2] = {Span(cache, cache_bytes(pages, P, Hk, D)), Span(slots, (uint64_t)T * 8)};
  const Span ks(k, bytes), vs(v, bytes);
  if (ks.meets(vs)) return TQ2_ERR_ARG;
  for (const Span& i : ins)
    if (ks.meets(i) || vs.meets(i)) return TQ2_ERR_ARG;
  tq2::Kv4LoadArgs a{};
  a.cache = cache, a.slots = slots, a.k = k, a.v = v;
  a.T = T, a.pages = pages, a.Hk = Hk, a.D = D, a.P = P;
  (void)hipGetLastError();
  return hip_status(tq2::launch_kv4_load(a, dtype, (hipStream_t)stream));
}

size_t tq2_kv4_attn_workspace_bytes(int64_t T, int32_t Hq, int32_t Hk, int32_t D, int32_t P, int32_t table_width,
                                    int32_t B, int32_t max_q) {
  if (!attn_sizes_ok(T, Hq, Hk, D, P, table_width, B, max_q)) return (size_t)-1;
  return tq2::plan_kv4_attn(Hq, Hk, D, P, table_width, B, max_q, 0).ws_bytes;
}

int32_t tq2_kv4_attn(const void* q, int64_t q_token_stride, int64_t q_head_stride, int64_t T, int32_t Hq, int32_t dtype,
                     const uint8_t* cache, int64_t pages, int32_t P, int32_t Hk, int32_t D, const int32_t* table,
                     int64_t table_stride, int32_t table_width, const int32_t* ctx_len, const int32_t* q_start,
                     int32_t B, int32_t max_q, float scale, int32_t window, void* out, float* lse, void* ws,
                     size_t ws_bytes, tq2_stream_t stream) {
  TQ2_TRY(check_cache_shape(pages, P, Hk, D));
  if (T < 0 || Hq < 1 || B < 1 || max_q < 1 || table_width < 1 || window < 0 || Hq % Hk) return TQ2_ERR_ARG;
  if (dtype != TQ2_F16 && dtype != TQ2_BF16) return TQ2_ERR_ARG;
  if (!isfinite(scale)) return TQ2_ERR_SCALE;
  if (!attn_sizes_ok(T, Hq, Hk, D, P, table_width, B, max_q)) return TQ2_ERR_SHAPE;
  if (table_stride < 0 || table_stride > kMost / B) return TQ2_ERR_SHAPE;
  if (T == 0) return TQ2_OK;
  if (!q_start && T != (int64_t)B * max_q) return TQ2_ERR_SHAPE;
  if (!cache || !table || !ctx_len || !out) return TQ2_ERR_ARG;
  uint64_t qb = 0;
  TQ2_TRY(check_heads(q, q_token_stride, q_head_stride, T, Hq, D, 2, &qb));
  if (!aligned(cache, 16) || !aligned(table, 4) || !aligned(ctx_len, 4) || !aligned(q_start, 4) || !aligned(out, 16) ||
      !aligned(lse, 4))
    return TQ2_ERR_ALIGN;
  const Span outs[2] = {Span(out, (uint64_t)(T * Hq * D * 2)), Span(lse, (uint64_t)(T * Hq * 4))};
  const Span ins[5] = {Span(q, qb), Span(cache, cache_bytes(pages, P, Hk, D)),
                       Span(table, (uint64_t)(((B - 1) * table_stride + table_width) * 4)),
                       Span(ctx_len, (uint64_t)B * 4), Span(q_start, (uint64_t)(B + (int64_t)1) * 4)};
  if (outs[0].meets(outs[1])) return TQ2_ERR_ARG;
  for (const Span& o : outs)
    for (const Span& i : ins)
      if (o.meets(i)) return TQ2_ERR_ARG;
  const tq2::Kv4AttnPlan plan = tq2::plan_kv4_attn(Hq, Hk, D, P, table_width, B, max_q, window);
  if (plan.ws_bytes) {
    if (!ws || ws_bytes < plan.ws_bytes || !aligned(ws, 256)) return TQ2_ERR_WORKSPACE;
    const Span w(ws, plan.ws_bytes);
    for (const Span& o : outs)
      if (w.meets(o)) return TQ2_ERR_WORKSPACE;
    for (const Span& i : ins)
      if (w.meets(i)) return TQ2_ERR_WORKSPACE;
  }
  tq2::Kv4AttnArgs a{};
  a.q = q, a.out = out, a.lse = lse, a.cache = cache, a.table = table, a.ctx = ctx_len, a.q_start = q_start;
  a.part = (float*)ws;
  a.q_ts = q_token_stride, a.q_hs = q_head_stride, a.table_stride = table_stride, a.T = T, a.pages = pages;
  a.B = B, a.max_q = max_q, a.width = table_width, a.Hq = Hq, a.Hk = Hk, a.G = Hq / Hk, a.D = D, a.P = P;
  a.window = window, a.scale = scale;
  (void)hipGetLastError();
  return hip_status(tq2::launch_kv4_attn(a, plan, dtype, (hipStream_t)stream));
}

}  // extern "C"
