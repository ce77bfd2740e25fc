// gfx950 (MI355X, CDNA4) kernels of the model's answer: log probabilities of
// given tokens, the entropy and the likeliest tokens of rows of logits.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "tq2_elem.h"
#include "tq2_step.h"

// Products are rounded before what is added to them, unless an fmaf says
// otherwise: the forms of a kernel give one row the same bits.
#pragma clang fp contract(off)

namespace tq2 {
namespace {

using namespace elem;

constexpr int kWaves = 4;  // of a workgroup
constexpr int kE = 16;     // logits a lane takes at a time
constexpr int kSpan = 64 * kE;

// What a part of a row leaves: the largest logit m so far (at least the type's
// lowest finite number), and with t = rate * (logit - m), rate = scale * log2 e,
// z = sum 2^t and w = sum 2^t t.  The logits' distances are scaled, not the
// logits: nothing passes fp32's range upwards, the largest has t = 0, and what
// is rounded is of the size of t, not of the logits.
struct Stat {
  float m, z, w;
};

__device__ __forceinline__ float exp2_of(float t) { return __builtin_amdgcn_exp2f(t); }

// The sums of s about another m >= s.m.  A term whose 2^t is 0 adds nothing to
// w either: distances are held at -256, where 2^t is 0 in fp32.
constexpr float kFar = -256.0f;
__device__ __forceinline__ Stat moved(Stat s, float m, float rate) {
  const float t = fmaxf((s.m - m) * rate, kFar), c = exp2_of(t);
  return {m, s.z * c, c * fmaf(s.z, t, s.w)};
}
__device__ __forceinline__ Stat joined(Stat a, Stat b, float rate) {
  const float m = fmaxf(a.m, b.m), ta = fmaxf((a.m - m) * rate, kFar), tb = fmaxf((b.m - m) * rate, kFar);
  const float ca = exp2_of(ta), cb = exp2_of(tb);
  return {m, fmaf(a.z, ca, b.z * cb), fmaf(fmaf(a.z, ta, a.w), ca, fmaf(b.z, tb, b.w) * cb)};
}
template <int O = 32>
__device__ __forceinline__ Stat wave_joined(Stat s, int lane, float rate) {
  s = joined(s, {across<O>(s.m, lane), across<O>(s.z, lane), across<O>(s.w, lane)}, rate);
  if constexpr (O > 1) s = wave_joined<O / 2>(s, lane, rate);
  return s;
}

// ---- the likeliest tokens ----
//
// A token's key orders by value, of equal values (0 and -0 are) by the lower
// id: the value's bits in an order of whole numbers above, the id's complement
// below.  0 is no token.  A wave holds the 64 largest keys that it has met, in
// order, one a lane.
typedef uint64_t Key;
static_assert(kMaxTop == 64, "a wave's list");

__device__ __forceinline__ Key key_of(float x, uint32_t id) {
  const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);
  const uint32_t o = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
  return ((Key)o << 32) | (uint32_t)~id;
}
__device__ __forceinline__ float value_of(Key k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return __builtin_bit_cast(float, o ^ ((uint32_t)((int32_t)~o >> 31) | 0x80000000u));
}
__device__ __forceinline__ uint32_t id_of(Key k) { return ~(uint32_t)k; }

// One step of a bitonic network: partners are O lanes apart, the larger goes to the lower lane where `down`.
template <int O, class K>
__device__ __forceinline__ K step_of(K k, int lane, bool down) {
  const K other = across<O>(k, lane);
  const bool larger = ((lane & O) == 0) == down;
  return (k > other) == larger ? k : other;
}
// A bitonic sequence over groups of N lanes into the order of `down`.
template <int N, class K>
__device__ __forceinline__ K merged(K k, int lane, bool down) {
  k = step_of<N / 2>(k, lane, down);
  if constexpr (N > 2) k = merged<N / 2>(k, lane, down);
  return k;
}
// All lanes into falling order.
template <int N = 64, class K>
__device__ __forceinline__ K sorted(K k, int lane) {
  if constexpr (N > 2) k = sorted<N / 2>(k, lane);
  return merged<N>(k, lane, N == 64 || (lane & N) == 0);
}
// The 64 largest of two falling lists.
__device__ __forceinline__ Key best_of(Key a, Key b, int lane) {
  const Key r = across<32>(across<16>(across<8>(across<4>(across<2>(across<1>(b, lane), lane), lane), lane), lane), lane);
  return merged<64>(a > r ? a : r, lane, true);
}
__device__ __forceinline__ Key lane_of(Key k, int lane) {  // `lane` the same in all
  const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)k, lane), hi = __builtin_amdgcn_readlane((uint32_t)(k >> 32), lane);
  return ((Key)hi << 32) | lo;
}

// ---- one part of a row ----

template <int DT>
constexpr int kPer = DT == kF32 ? 4 : 8;  // logits in 16 bytes

// A lane's logits of the span that begins at place v0 of a row (a multiple of
// 16 bytes in memory; it may lie before the row), as floats; -inf outside
// [0, V).  In load u a wave takes 1 KiB: place v0 + u*64*kPer + lane*kPer + i.
template <int DT>
__device__ __forceinline__ void load_span(const typename Elem<DT>::T* row, int64_t v0, int64_t V, int lane, float (&x)[kE]) {
  constexpr int P = kPer<DT>;
#pragma unroll
  for (int u = 0; u < kE / P; ++u) {
    const int64_t at = v0 + u * 64 * P + lane * P;
    if (at >= 0 && at + P <= V) {
      const Vec<DT, P> a = __builtin_nontemporal_load((const Vec<DT, P>*)(row + at));  // read once
#pragma unroll
      for (int i = 0; i < P; ++i) x[u * P + i] = (float)a[i];
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) x[u * P + i] = at + i >= 0 && at + i < V ? (float)row[at + i] : -INFINITY;
    }
  }
}

// A row's results from its sums (the first lane's: a pair's order in `joined`
// is not the same in both of its lanes) and keys; one wave.
struct Finish {
  const LogprobArgs& a;
  int64_t t;
  __device__ __forceinline__ void operator()(Stat s, float given, int lane, Key best) const {
    s.z = __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(uint32_t, s.z)));
    // a row that holds NaN or +inf has no distribution, nor has one whose logits are all -inf
    const bool none = s.z == 0.0f, bad = s.z != s.z;
    const float log_z = logf(s.z);
    const auto logprob = [&](float logit) { return bad ? NAN : none ? -INFINITY : fmaf(logit - s.m, a.scale, -log_z); };
    if (lane == 0) {
      if (a.tokens) {
        const int64_t tok = a.tokens[t];
        a.logprobs[t] = tok < 0 || tok >= a.V ? 0.0f : logprob(given);
      }
      if (a.entropy) a.entropy[t] = none ? 0.0f : log_z - s.w / s.z * 0.693147181f;
    }
    if (lane < a.top) {
      a.top_tokens[t * a.top + lane] = bad ? -1 : (int64_t)id_of(best);
      a.top_logprobs[t * a.top + lane] = logprob(value_of(best));
    }
  }
};

// One pass over a row, or over a share of it (gridDim.y of them): a wave takes
// spans of 1024 logits in turn, holds sums about a running largest value in
// every lane, and offers what is larger than its top-th key so far to its
// list.  Later spans hold higher ids, so a value that equals the top-th is no
// candidate.  Before the list is full the bound is the top-th largest of the
// lanes' own largest of the first span: at least `top` logits are that large.
// 80 scalar registers, 96 with those that the runtime keeps, are what eight
// waves a SIMD have: 2048 rows are then on the GPU all at once (65537 bf16
// logits, none of the likeliest: 54 us, 67 with seven waves).
template <int DT, bool TOP>
__global__ __launch_bounds__(64 * kWaves) __attribute__((amdgpu_num_sgpr(80))) void k_logprobs(LogprobArgs a) {
  typedef typename Elem<DT>::T T;
  __shared__ Stat stats[kWaves];
  __shared__ Key lists[TOP ? kWaves : 1][kMaxTop];
  __shared__ Key wait[TOP ? kWaves : 1][128];  // candidates that are not in the list yet, fewer than 64 at a time
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = blockIdx.x;
  const T* row = (const T*)a.logits + t * a.stride;
  const int shift = (int)((uintptr_t)row / sizeof(T) % kPer<DT>);
  const int spans = (int)((a.V + shift + kSpan - 1) / kSpan);
  const int share = ((spans + (int)gridDim.y - 1) / (int)gridDim.y + kWaves - 1) / kWaves * kWaves;
  const int end = min(spans, ((int)blockIdx.y + 1) * share);
  float given = 0.0f;
  if (a.tokens && threadIdx.x == 0) {
    const int64_t tok = a.tokens[t];
    if (tok >= 0 && tok < a.V) given = (float)row[tok];
  }

  Stat s = {-3.40282347e38f, 0.0f, 0.0f};
  Key best = 0;
  float bound = -INFINITY;
  bool full = false, first = true;
  int waiting = 0;  // wave-uniform
  float next[kE], x[kE];
  int sp = (int)blockIdx.y * share + wave;
  if (sp < end) load_span<DT>(row, (int64_t)sp * kSpan - shift, a.V, lane, next);
  for (; sp < end; sp += kWaves) {
#pragma unroll
    for (int i = 0; i < kE; ++i) x[i] = next[i];
    if (sp + kWaves < end) load_span<DT>(row, (int64_t)(sp + kWaves) * kSpan - shift, a.V, lane, next);
    float most = x[0];
#pragma unroll
    for (int i = 1; i < kE; ++i) most = fmaxf(most, x[i]);
    if (most > s.m) s = moved(s, most, a.rate);
    float z[2] = {0.0f, 0.0f}, w[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kE; ++i) {
      const float d = (x[i] - s.m) * a.rate, e = exp2_of(d);
      z[i & 1] += e;
      w[i & 1] = fmaf(e, fmaxf(d, kFar), w[i & 1]);
    }
    s.z += z[0] + z[1];
    s.w += w[0] + w[1];
    if constexpr (TOP) {
      if (first) {
        const float k = sorted(most, lane);
        bound = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(uint32_t, k), a.top - 1));
        first = false;
      }
      if (__builtin_amdgcn_ballot_w64(full ? most > bound : most >= bound)) {
        const int64_t v0 = (int64_t)sp * kSpan - shift;
#pragma unroll
        for (int i = 0; i < kE; ++i) {
          constexpr int P = kPer<DT>;
          const int64_t at = v0 + (i / P) * 64 * P + lane * P + i % P;
          const bool on = (full ? x[i] > bound : x[i] >= bound) && at >= 0 && at < a.V;
          const uint64_t all = __builtin_amdgcn_ballot_w64(on);
          if (!all) continue;
          if (on) wait[wave][waiting + __builtin_amdgcn_mbcnt_hi((uint32_t)(all >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)all, 0))] = key_of(x[i], (uint32_t)at);
          waiting += __builtin_popcountll(all);
          __builtin_amdgcn_wave_barrier();
          if (waiting >= 64) {
            const Key k = wait[wave][lane], rest = wait[wave][64 + lane];
            __builtin_amdgcn_wave_barrier();
            wait[wave][lane] = rest;
            waiting -= 64;
            best = best_of(best, sorted(k, lane), lane);
          }
        }
        const Key last = lane_of(best, a.top - 1);
        if (last) bound = value_of(last), full = true;
      }
    }
  }
  s = wave_joined(s, lane, a.rate);
  if constexpr (TOP) {
    if (waiting) best = best_of(best, sorted(lane < waiting ? wait[wave][lane] : 0, lane), lane);
    lists[wave][lane] = best;
  }
  if (lane == 0) stats[wave] = s;
  __syncthreads();
  if (wave) return;
#pragma unroll
  for (int o = 1; o < kWaves; ++o) {
    s = joined(s, stats[o], a.rate);
    if constexpr (TOP) best = best_of(best, lists[o][lane], lane);
  }
  if (gridDim.y == 1) {
    Finish{a, t}(s, given, lane, best);
    return;
  }
  // the share's part: 16 bytes of sums, then `top` keys
  const int64_t at = t * gridDim.y + blockIdx.y;
  if (lane == 0) ((float4*)a.ws)[at] = make_float4(s.m, s.z, s.w, 0.0f);
  if (TOP && lane < a.top) ((Key*)(a.ws + a.T * gridDim.y * 16))[at * a.top + lane] = best;
}

// The parts of a row joined.
constexpr int kJoinWaves = 8;
template <int DT, bool TOP>
__global__ __launch_bounds__(64 * kJoinWaves) void k_logprobs_join(LogprobArgs a, int parts) {
  __shared__ Stat stats[kJoinWaves];
  __shared__ Key lists[TOP ? kJoinWaves : 1][kMaxTop];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = blockIdx.x;
  float given = 0.0f;
  if (a.tokens && threadIdx.x == 0) {
    const int64_t tok = a.tokens[t];
    if (tok >= 0 && tok < a.V) given = (float)((const typename Elem<DT>::T*)a.logits)[t * a.stride + tok];
  }
  Stat s = {-3.40282347e38f, 0.0f, 0.0f};
  for (int p = threadIdx.x; p < parts; p += 64 * kJoinWaves) {
    const float4 v = ((const float4*)a.ws)[t * parts + p];
    s = joined(s, {v.x, v.y, v.z}, a.rate);
  }
  Key best = 0;
  if constexpr (TOP) {
    const Key* keys = (const Key*)(a.ws + a.T * parts * 16);
    // (the next list is on its way while one is merged)
    Key next = wave < parts && lane < a.top ? keys[(t * parts + wave) * a.top + lane] : 0;
    for (int p = wave; p < parts; p += kJoinWaves) {
      const Key k = next;
      next = p + kJoinWaves < parts && lane < a.top ? keys[(t * parts + p + kJoinWaves) * a.top + lane] : 0;
      best = best_of(best, k, lane);
    }
    lists[wave][lane] = best;
  }
  s = wave_joined(s, lane, a.rate);
  if (lane == 0) stats[wave] = s;
  __syncthreads();
  for (int n = kJoinWaves / 2; n; n /= 2) {
    if (wave < n) {
      s = joined(s, stats[wave + n], a.rate);
      if (lane == 0) stats[wave] = s;
      if constexpr (TOP) {
        best = best_of(best, lists[wave + n][lane], lane);
        lists[wave][lane] = best;
      }
    }
    __syncthreads();
  }
  if (wave == 0) Finish{a, t}(s, given, lane, best);
}

template <int DT, bool TOP>
hipError_t launch(const LogprobArgs& a, hipStream_t st) {
  const int parts = logprob_splits(a.T, a.V);
  hipLaunchKernelGGL((k_logprobs<DT, TOP>), dim3((unsigned)a.T, (unsigned)parts), dim3(64 * kWaves), 0, st, a);
  if (parts > 1)
    hipLaunchKernelGGL((k_logprobs_join<DT, TOP>), dim3((unsigned)a.T), dim3(64 * kJoinWaves), 0, st, a, parts);
  return hipGetLastError();
}
template <int DT>
hipError_t launch(const LogprobArgs& a, hipStream_t st) {
  return a.top ? launch<DT, true>(a, st) : launch<DT, false>(a, st);
}

}  // namespace

// A row is shared where the rows alone give fewer than 512 workgroups, down to a span for each wave.
int logprob_splits(int64_t T, int64_t V) {
  const int64_t spans = V / kSpan + 1, most = (spans + kWaves - 1) / kWaves, want = (512 + T - 1) / T;
  return (int)(want < most ? want : most);
}
size_t logprob_workspace_bytes(int64_t T, int64_t V, int32_t top) {
  const int64_t parts = logprob_splits(T, V);
  return parts == 1 ? 0 : (size_t)(T * parts * (16 + 8 * (int64_t)top));
}

hipError_t launch_token_logprobs(const LogprobArgs& given, int dtype, hipStream_t st) {
  LogprobArgs a = given;
  // (finite: the distance 0 stays 0.  Scales so large that this holds them back
  // tell logits apart that are less than 2^-120 from each other.)
  a.rate = (float)fmin((double)a.scale * 1.4426950408889634, 3.4028234663852886e38);
  if (dtype == kF16) return launch<kF16>(a, st);
  if (dtype == kBF16) return launch<kBF16>(a, st);
  return launch<kF32>(a, st);
}

}  // namespace tq2
