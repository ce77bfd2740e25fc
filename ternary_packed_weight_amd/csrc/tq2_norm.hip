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

// Sum over the workgroup (`waves` waves), the same in every lane.
__device__ __forceinline__ double wg_sum(double v, int waves, double* red) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o, 64);
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = red[0];
  for (int w = 1; w < waves; ++w) s += red[w];
  return s;
}
// Largest of the workgroup's bit patterns.
__device__ __forceinline__ uint32_t wg_max(uint32_t v, int waves, uint32_t* red) {
#pragma unroll
  for (int o = 32; o; o >>= 1) {
    const uint32_t b = __shfl_xor(v, o, 64);
    v = b > v ? b : v;
  }
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  uint32_t m = red[0];
  for (int w = 1; w < waves; ++w) m = red[w] > m ? red[w] : m;
  return m;
}

// fp32 of 1/sqrt(v): an fp32 estimate and one Newton step in fp64 (relative
// error 2^-44) where v is in fp32's range, else fp64's own.
__device__ __forceinline__ float root(double v) {
  if (v > 1e-30 && v < 1e30) {
    const double y = (double)__builtin_amdgcn_rsqf((float)v);
    return (float)(y * fma(-0.5 * v, y * y, 1.5));
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
template <int SRC, int RES, int V>
__global__ __launch_bounds__(1024) void k_add_rms_norm(NormArgs a, int out_dtype) {
  __shared__ double red_sum[16];
  __shared__ uint32_t red_max[16];
  const int threads = blockDim.x, waves = threads >> 6, D = a.D;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    float h[V][8], r[V][8], w[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int d = 8 * ((int)threadIdx.x + v * threads);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[v][i] = r[v][i] = 0.0f, w[v][i] = 1.0f;
      if (d >= D) continue;
      load8<SRC>(a.x, t * a.x_stride + d, h[v]);
      if constexpr (RES != kNone) load8<RES>(a.residual, t * a.r_stride + d, r[v]);
      if (V <= 2 && a.weight) load8<kF32>(a.weight, d, w[v]);  // on its way during the sum
    }
    double sum = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int d = 8 * ((int)threadIdx.x + v * threads);
      if constexpr (RES != kNone) {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[v][i] = rounded<RES>(h[v][i] + r[v][i]);
        if (a.h_out && d < D) store8<RES>(a.h_out, t * a.r_stride + d, h[v]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fma((double)h[v][i], (double)h[v][i], sum);
    }
    sum = wg_sum(sum, waves, red_sum);
    const float rt = root(sum / D + (double)a.eps);
    uint32_t most = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int d = 8 * ((int)threadIdx.x + v * threads);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[v][i] *= rt;
      if (d < D) {
        if (a.weight) {
          if (V > 2) load8<kF32>(a.weight, d, w[v]);
#pragma unroll
          for (int i = 0; i < 8; ++i) h[v][i] *= w[v][i];
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
        s = __builtin_bit_cast(float, wg_max(most, waves, red_max)) / 127.0f;
        if (threadIdx.x == 0) a.scales[t] = s;
      }
      const float inv = 1.0f / s;
      const bool usual = s > 0x1p-100f && s < 0x1p100f;  // (the reciprocal and the products keep 24 bits)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int d = 8 * ((int)threadIdx.x + v * threads);
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

template <int SRC, int RES>
hipError_t launch_norm(const NormArgs& a, int out_dtype, hipStream_t st) {
  const int vecs = a.D / 8;
  int per = vecs > 1024 ? (vecs > 2048 ? 8 : 2) : vecs > 512 && a.T >= 512 ? 2 : 1;
  int threads = ((vecs + per - 1) / per + 63) / 64 * 64;
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
