// gfx950 (MI355X, CDNA4) kernels of the gated projections: h = silu(Wg x) *
// (Wu x) of two ternary matrices for any number of tokens.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "tq2_elem.h"
#include "tq2_step.h"

namespace tq2 {
namespace {

using namespace elem;

typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

// A buffer of `bytes` bytes from `base` (wave-uniform); reads past it give zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ v4u load16(__amdgpu_buffer_rsrc_t r, int at) {
  return __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
}

// Eight codes (the low 16 bits of c, lowest first) as the fp16 weights d *
// (code - 1), exact.  t holds code 2j at bit 4j and code 2j + 1 at bit 4j +
// 16, so a mask and the exponent of 1024 make the pair 1024 + 16^j code, and
// one fused multiply-add the pair code - 1.  15 operations for 8 weights, and
// the weights come in the order of K: activations go to the matrix cores as
// they lie in memory.
__device__ __forceinline__ v8h weights8(uint32_t c, v2h d) {
  const uint32_t t = c | (c << 14), t8 = t >> 8;
  const v2h p0 = __builtin_bit_cast(v2h, (t & 0x00030003u) | 0x64006400u) - v2h{(_Float16)1025.0f, (_Float16)1025.0f};
  const v2h q = {(_Float16)0.0625f, (_Float16)0.0625f}, q2 = {(_Float16)0.00390625f, (_Float16)0.00390625f};
  const v2h m65 = {(_Float16)-65.0f, (_Float16)-65.0f}, m5 = {(_Float16)-5.0f, (_Float16)-5.0f};
  const v2h p1 = __builtin_elementwise_fma(__builtin_bit_cast(v2h, (t & 0x00300030u) | 0x64006400u), q, m65);
  const v2h p2 = __builtin_elementwise_fma(__builtin_bit_cast(v2h, (t & 0x03000300u) | 0x64006400u), q2, m5);
  const v2h p3 = __builtin_elementwise_fma(__builtin_bit_cast(v2h, (t8 & 0x00300030u) | 0x64006400u), q, m65);
  const v2h w0 = p0 * d, w1 = p1 * d, w2 = p2 * d, w3 = p3 * d;
  return v8h{w0[0], w0[1], w1[0], w1[1], w2[0], w2[1], w3[0], w3[1]};
}
// Eight int8 activations as fp16, exact: a byte with its top bit turned is x + 128, below the exponent of 1024.
__device__ __forceinline__ v8h halves8(uint32_t a, uint32_t b) {
  uint32_t r[4];
  const uint32_t u[2] = {a ^ 0x80808080u, b ^ 0x80808080u};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(v2h, __builtin_amdgcn_perm(0x64646464u, u[i >> 1], i & 1 ? 0x04030402u : 0x04010400u)) -
                                            v2h{(_Float16)1152.0f, (_Float16)1152.0f});
  return __builtin_bit_cast(v8h, v4u{r[0], r[1], r[2], r[3]});
}

// silu(g) * u = g / (1 + e^-g) * u
__device__ __forceinline__ float gate(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504f)) * u;
}

__device__ __forceinline__ void store1(void* h, int64_t at, float v, int dtype) {
  if (dtype == kF32) ((float*)h)[at] = v;
  else if (dtype == kF16) ((_Float16*)h)[at] = (_Float16)v;
  else ((__bf16*)h)[at] = (__bf16)v;
}

// ---- few tokens ----
//
// A workgroup of C waves takes 16*R gate rows, the up rows of the same places
// and TT tiles of 16 tokens; its waves take blocks of 256 along K in turn and
// their sums meet in LDS, added in the order of the waves.  Lane (G, i) = (l /
// 16, l % 16) holds row i's codes of quarter G of a block and token i's
// activations there; matrix instruction s of a block takes the places 64G + 8s
// .. + 7 of all quarters.
template <bool I8, int R, int TT, int C>
__global__ __launch_bounds__(64 * C) void k_gated_few(GatedArgs a, int out_dtype) {
  constexpr int U = 2 * R;
  __shared__ v4f red[C][U][TT][64];
  const int lane = threadIdx.x & 63, G = lane >> 4, i = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * (16 * R), m0 = (int64_t)blockIdx.y * (16 * TT);
  const int rows = (int)(a.N - n0 < 16 * R ? a.N - n0 : 16 * R);
  const int toks = (int)(a.M - m0 < 16 * TT ? a.M - m0 : 16 * TT);
  const int row_bytes = (int)(a.K / 4), blocks = (int)(a.K / 256), xb = (int)a.K * (I8 ? 1 : 2);
  __amdgpu_buffer_rsrc_t rc[2], rs[2];
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    rc[p] = buffer_of(a.codes[p] + n0 * row_bytes, (uint32_t)(rows * row_bytes));
    rs[p] = buffer_of(a.scales[p] + n0 * blocks, (uint32_t)(rows * blocks * 2));
  }
  const __amdgpu_buffer_rsrc_t rx = buffer_of((const uint8_t*)a.x + m0 * xb, (uint32_t)(toks * xb));
  v4f acc[U][TT];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int q = 0; q < TT; ++q) acc[u][q] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  for (int b = wave; b < blocks; b += C) {
    v4u w[U];
    v2h d[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = 16 * (u >> 1) + i;
      w[u] = load16(rc[u & 1], r * row_bytes + 64 * b + 16 * G);
      const _Float16 e = __builtin_bit_cast(_Float16, (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rs[u & 1], (r * blocks + b) * 2, 0, 0));
      d[u] = v2h{e, e};
    }
#pragma unroll
    for (int s = 0; s < 8; s += 2) {
      v8h x[2][TT];
#pragma unroll
      for (int q = 0; q < TT; ++q) {
        const int at = (16 * q + i) * xb + (256 * b + 64 * G + 8 * s) * (I8 ? 1 : 2);
        const v4u e = load16(rx, at);
        if constexpr (I8) {
          x[0][q] = halves8(e[0], e[1]);
          x[1][q] = halves8(e[2], e[3]);
        } else {
          x[0][q] = __builtin_bit_cast(v8h, e);
          x[1][q] = __builtin_bit_cast(v8h, load16(rx, at + 16));
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const v8h wt = weights8((w[u][s / 2] >> (16 * k)) & 0xFFFFu, d[u]);
#pragma unroll
          for (int q = 0; q < TT; ++q) acc[u][q] = __builtin_amdgcn_mfma_f32_16x16x32_f16(wt, x[k][q], acc[u][q], 0, 0, 0);
        }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int q = 0; q < TT; ++q) red[wave][u][q][lane] = acc[u][q];
  __syncthreads();
  // output (row n of the workgroup, token m): lane (n % 16 / 4, m % 16), element n % 4
  for (int o = threadIdx.x; o < 16 * R * 16 * TT; o += 64 * C) {
    const int n = o % (16 * R), m = o / (16 * R);
    if (n >= rows || m >= toks) continue;
    const int l = n % 16 / 4 * 16 + m % 16, u = 2 * (n / 16), q = m / 16;
    float g = red[0][u][q][l][n % 4], p = red[0][u + 1][q][l][n % 4];
#pragma unroll
    for (int c = 1; c < C; ++c) g += red[c][u][q][l][n % 4], p += red[c][u + 1][q][l][n % 4];
    if constexpr (I8) {
      const float s = a.x_scales ? a.x_scales[m0 + m] : a.s;
      g *= s, p *= s;
    }
    store1(a.h, (m0 + m) * a.N + n0 + n, gate(g, p), out_dtype);
  }
}

template <bool I8, int TT>
hipError_t launch_few(const GatedArgs& a, int out_dtype, hipStream_t st) {
  constexpr int R = 2;
  const dim3 grid((unsigned)((a.N + 16 * R - 1) / (16 * R)), (unsigned)((a.M + 16 * TT - 1) / (16 * TT)));
  if (a.K >= 2048)
    hipLaunchKernelGGL((k_gated_few<I8, R, TT, 8>), grid, dim3(64 * 8), 0, st, a, out_dtype);
  else
    hipLaunchKernelGGL((k_gated_few<I8, R, TT, 4>), grid, dim3(64 * 4), 0, st, a, out_dtype);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gated(const GatedArgs& a, bool int8, int out_dtype, hipStream_t st) {
  if (int8) return a.M <= 16 ? launch_few<true, 1>(a, out_dtype, st) : launch_few<true, 2>(a, out_dtype, st);
  return a.M <= 16 ? launch_few<false, 1>(a, out_dtype, st) : launch_few<false, 2>(a, out_dtype, st);
}

}  // namespace tq2
