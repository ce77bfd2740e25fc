// gfx950 (MI355X, CDNA4) kernels of the residual's addition and RMS norm.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "tq2_elem.h"
#include "tq2_step.h"

namespace tq2 {
namespace {

using namespace elem;

constexpr int kNone = -1;  // no residual

// What `join` makes of all lanes' values, from lanes O apart down to neighbours, the same in every lane.
template <int O, class V, class F>
__device__ __forceinline__ V all_lanes(V v, int lane, F join) {
  v = join(v, across<O>(v, lane));
  if constexpr (O > 1) v = all_lanes<O / 2>(v, lane, join);
  return v;
}
// ... of the whole workgroup: the waves' values meet in `red`, `none` stands for waves that are not there.
template <class V, class F>
__device__ __forceinline__ V all_waves(V v, V none, int waves, V* red, F join) {
  const int lane = threadIdx.x & 63;
  v = all_lanes<32>(v, lane, join);
  if (waves == 1) return v;
  if (lane == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return all_lanes<8>(lane % 16 < waves ? red[lane % 16] : none, lane, join);
}

// fp32 of 1/sqrt(v).  Where v is in fp32's range: an fp32 estimate y, whose
// square is exact in fp64, so that e = 1 - v y^2 (at most 2^-21) is rounded once,
// and y (1 - e)^-1/2 = y + y e (1/2 + 3/8 e + ...), which leaves out less than
// e^3 / 3 = 2^-64: within fp64's rounding, as its own root and quotient are.
// (Without the second term, 2^-44, one row in some 10^6 had another fp32 root.)
__device__ __forceinline__ float root(double v) {
  if (v > 1e-30 && v < 1e30) {
    const double y = (double)__builtin_amdgcn_rsqf((float)v), e = fma(-v, y * y, 1.0);
    return (float)fma(y * e, fma(0.375, e, 0.5), y);
  }
  return (float)(1.0 / sqrt(v));
}

// clamp(rint(y / s), -128, 127), 0 for s = 0.  y * (1/s) is within 3 * 2^-24 of
// the division's value relative to it; only next to a half is the division
// needed to tell the code, and beyond 128.5 every value has the same one.
__device__ __forceinline__ int code_of(float y, float s, float inv, bool usual) {
  const float v = y * inv;
  float c = rintf(v);
  const bool near = fabsf(v - c) > 0.5f - 0x1p-14f && fabsf(v) < 130.0f;  // 2^-14 > 3 * 2^-24 * 130
  if (!usual || near) c = s == 0.0f ? 0.0f : rintf(y / s);
  return (int)fminf(fmaxf(c, -128.0f), 127.0f);
}

// h = residual + x, rounded to the residual's type; y = (h * r) * w with r =
// fp32(1/sqrt(sum h^2 / D + eps)), the sum and the root in fp64, so that r
// does not depend on the order of the sum; out: y rounded once, or the code
// clamp(rint(y / s), -128, 127) with s given, or max|y| / 127.  A workgroup
// takes a row at a time and holds it in registers between the sum and the
// scaling: every element is read once and written once.
//
// Memory bounds it where there are many rows (4096 x 4096, fp32 and a bf16
// residual in, fp16 out: 30.3 us, 5.5 TB/s of reads and writes; on the same rows
// again, part of them in the last-level cache, 25.5), else the trip there and two
// meetings of the waves: one row of 4096 takes 2.7 us.  Its lanes' values meet
// through the vector unit's moves; through LDS the same row took 0.4 us more.
template <int SRC, int RES, int V>
__global__ __launch_bounds__(1024) void k_add_rms_norm(NormArgs a, int out_dtype) {
  __shared__ double red_sum[16];
  __shared__ uint32_t red_max[16];
  const int threads = blockDim.x, waves = threads >> 6, D = a.D;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));  // each row's addresses anew: kept from row to row, those of V = 8 took 120 registers
    // all of a row's loads at once where the registers hold them
    constexpr bool kAhead = V <= 2;
    float h[V][8], r[kAhead ? V : 1][8], w[kAhead ? V : 1][8];
    double sum = 0.0;
    const auto add = [&](int v) {
      const int d = 8 * (tid + v * threads);
      if constexpr (RES != kNone) {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[v][i] = rounded<RES>(h[v][i] + r[kAhead ? v : 0][i]);
        if (a.h_out && d < D) store8<RES>(a.h_out, t * a.r_stride + d, h[v]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fma((double)h[v][i], (double)h[v][i], sum);
    };
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int d = 8 * (tid + v * threads);
      float(&rv)[8] = r[kAhead ? v : 0];
#pragma unroll
      for (int i = 0; i < 8; ++i) h[v][i] = rv[i] = 0.0f;
      if (d < D) {
        load8<SRC>(a.x, t * a.x_stride + d, h[v]);
        if constexpr (RES != kNone) load8<RES>(a.residual, t * a.r_stride + d, rv);
        if constexpr (kAhead)
          if (a.weight) load8<kF32>(a.weight, d, w[v]);
      }
      if constexpr (!kAhead) add(v);
    }
    if constexpr (kAhead) {
#pragma unroll
      for (int v = 0; v < V; ++v) add(v);
    }
    sum = all_waves(sum, 0.0, waves, red_sum, [](double p, double q) { return p + q; });
    const float rt = root(sum / D + (double)a.eps);
    uint32_t most = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int d = 8 * (tid + v * threads);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[v][i] *= rt;
      if (d < D) {
        if (a.weight) {
          float(&wv)[8] = w[kAhead ? v : 0];
          if constexpr (!kAhead) load8<kF32>(a.weight, d, wv);
#pragma unroll
          for (int i = 0; i < 8; ++i) h[v][i] *= wv[i];
        }
        if (out_dtype == kF16) store8<kF16>(a.out, t * D + d, h[v]);
        if (out_dtype == kBF16) store8<kBF16>(a.out, t * D + d, h[v]);
        if (out_dtype == kF32) store8<kF32>(a.out, t * D + d, h[v]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t b = __builtin_bit_cast(uint32_t, h[v][i]) & 0x7FFFFFFFu;  // NaN is the largest
          most = b > most ? b : most;
        }
      }
    }
    if (out_dtype == kOutI8) {
      float s = a.s;
      if (a.scales) {
        most = all_waves(most, 0u, waves, red_max, [](uint32_t p, uint32_t q) { return p > q ? p : q; });
        s = __builtin_bit_cast(float, most) / 127.0f;
        if (threadIdx.x == 0) a.scales[t] = s;
      }
      const float inv = 1.0f / s;
      const bool usual = s > 0x1p-100f && s < 0x1p100f;  // (the reciprocal and the products keep 24 bits)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int d = 8 * (tid + v * threads);
        if (d >= D) continue;
        uint32_t q[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = code_of(h[v][i], s, inv, usual);
          q[i >> 2] |= ((uint32_t)c & 0xFFu) << (8 * (i & 3));
        }
        *(uint2*)((uint8_t*)a.out + t * D + d) = make_uint2(q[0], q[1]);
      }
    }
    if (waves > 1) __syncthreads();  // before the next row's sums
  }
}

// Vectors of 8 elements a thread holds.  One row is quickest spread over the
// most waves (1 x 8192 with 1 / 2: 3.8 / 4.5 us); many wide rows with two each,
// since two workgroups then share a unit (4096 x 8192 71 / 61 us, 4096 x 5000
// 28.1 / 25.8).
template <int SRC, int RES>
hipError_t launch_norm(const NormArgs& a, int out_dtype, hipStream_t st) {
  const int vecs = a.D / 8;
  const int per = vecs > 1024 ? (vecs > 2048 ? 8 : 2) : vecs > 512 && a.T >= 512 ? 2 : 1;
  const int threads = ((vecs + per - 1) / per + 63) / 64 * 64;
  const unsigned grid = (unsigned)(a.T < (1 << 20) ? a.T : 1 << 20);
  if (per == 8)
    hipLaunchKernelGGL((k_add_rms_norm<SRC, RES, 8>), dim3(grid), dim3(threads), 0, st, a, out_dtype);
  else if (per == 2)
    hipLaunchKernelGGL((k_add_rms_norm<SRC, RES, 2>), dim3(grid), dim3(threads), 0, st, a, out_dtype);
  else
    hipLaunchKernelGGL((k_add_rms_norm<SRC, RES, 1>), dim3(grid), dim3(threads), 0, st, a, out_dtype);
  return hipGetLastError();
}

template <int SRC>
hipError_t launch_norm(const NormArgs& a, int r_dtype, int out_dtype, hipStream_t st) {
  if (!a.residual) return launch_norm<SRC, kNone>(a, out_dtype, st);
  if (r_dtype == kF16) return launch_norm<SRC, kF16>(a, out_dtype, st);
  if (r_dtype == kBF16) return launch_norm<SRC, kBF16>(a, out_dtype, st);
  return launch_norm<SRC, kF32>(a, out_dtype, st);
}

}  // namespace

hipError_t launch_add_rms_norm(const NormArgs& a, int x_dtype, int r_dtype, int out_dtype, hipStream_t st) {
  if (x_dtype == kF16) return launch_norm<kF16>(a, r_dtype, out_dtype, st);
  if (x_dtype == kBF16) return launch_norm<kBF16>(a, r_dtype, out_dtype, st);
  return launch_norm<kF32>(a, r_dtype, out_dtype, st);
}

}  // namespace tq2
