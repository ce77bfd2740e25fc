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
// `top` is 0x64006400 in a vector register: an and-or takes one scalar.
__device__ __forceinline__ uint32_t exponent_of_1024() {
  uint32_t c;
  asm("v_mov_b32 %0, 0x64006400" : "=v"(c));
  return c;
}
__device__ __forceinline__ v8h weights8(uint32_t c, v2h d, uint32_t top) {
  const uint32_t t = c | (c << 14), t8 = t >> 8;
  const auto half2 = [](float f) { return v2h{(_Float16)f, (_Float16)f}; };
  const auto pair = [&](uint32_t w, uint32_t mask) { return __builtin_bit_cast(v2h, (w & mask) | top); };
  const v2h w0 = (pair(t, 0x00030003u) - half2(1025.0f)) * d;
  const v2h w1 = __builtin_elementwise_fma(pair(t, 0x00300030u), half2(0.0625f), half2(-65.0f)) * d;
  const v2h w2 = __builtin_elementwise_fma(pair(t, 0x03000300u), half2(0.00390625f), half2(-5.0f)) * d;
  const v2h w3 = __builtin_elementwise_fma(pair(t8, 0x00300030u), half2(0.0625f), half2(-65.0f)) * d;
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
  const uint32_t top = exponent_of_1024();
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
          const v8h wt = weights8((w[u][s / 2] >> (16 * k)) & 0xFFFFu, d[u], top);
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

// ---- many tokens ----
//
// A workgroup of WR x WC waves takes 32*WR gate rows with their up rows and
// 16*NT*WC tokens; a wave 32 + 32 rows (two groups of 16 each) and 16*NT
// tokens, whose sums stay in its registers.  K goes in blocks of 128: the
// tokens' activations of a block go straight to LDS (two blocks, one being
// filled while the other is used), the codes to registers, one block ahead.
// Lane (G, i) holds places 32G .. 32G + 31 of the block of row (token) i, of
// which matrix instruction s takes 8s .. 8s + 7.
constexpr int kStage = 128;

// 16 bytes a lane from a buffer straight to LDS, lane l's at lds + 16 l
__device__ __forceinline__ void load_lds(__amdgpu_buffer_rsrc_t r, int at, int scalar, uint8_t* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, at, scalar, 0, 0);
}

template <int WR, int WC, int NT, int DST>
__global__ __launch_bounds__(64 * WR * WC, 2) void k_gated_many(GatedArgs a) {
  constexpr int kWaves = WR * WC, kTok = 16 * NT * WC, kBytes = kTok * kStage * 2;
  __shared__ __attribute__((aligned(16))) uint8_t lds0[kBytes], lds1[kBytes];
  const int lane = threadIdx.x & 63, G = lane >> 4, i = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wr = wave % WR, wc = wave / WR;
  const int64_t n0 = (int64_t)blockIdx.x * (32 * WR), m0 = (int64_t)blockIdx.y * kTok;
  const int rows = (int)(a.N - n0 < 32 * WR ? a.N - n0 : 32 * WR);
  const int toks = (int)(a.M - m0 < kTok ? a.M - m0 : kTok);
  const int row_bytes = (int)(a.K / 4), blocks = (int)(a.K / 256), xb = (int)a.K * 2;
  // a buffer for each group of 16 rows (gate, gate, up, up) and of 16 tokens,
  // none longer than its valid rows.  (What a load adds by its scalar offset
  // stays inside a row; rows past the last one are past the buffer without it,
  // and read as zeros.)
  __amdgpu_buffer_rsrc_t rc[4], rs[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int r0 = 32 * wr + 16 * (u & 1), valid = rows < r0 ? 0 : rows - r0 < 16 ? rows - r0 : 16;
    const int64_t at = valid ? n0 + r0 : 0;
    rc[u] = buffer_of(a.codes[u >> 1] + at * row_bytes, (uint32_t)(valid * row_bytes));
    rs[u] = buffer_of(a.scales[u >> 1] + at * blocks, (uint32_t)(valid * blocks * 2));
  }
  // the wave's share of a block's activations: a load brings 4 tokens' 256
  // bytes; the 16-byte piece c of token t lies at place c ^ (t % 16) of its
  // row, so that a read of 16 tokens' pieces meets every bank once
  constexpr int kGroups = kTok / 16 / kWaves;
  static_assert(kGroups * 16 * kWaves == kTok, "groups of 16 tokens, as many for each wave");
  __amdgpu_buffer_rsrc_t rx[kGroups];
#pragma unroll
  for (int n = 0; n < kGroups; ++n) {
    const int t0 = (wave * kGroups + n) * 16, valid = toks < t0 ? 0 : toks - t0 < 16 ? toks - t0 : 16;
    rx[n] = buffer_of((const uint8_t*)a.x + (valid ? m0 + t0 : 0) * xb, (uint32_t)(valid * xb));
  }
  int xo[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int t = 4 * k + G;
    xo[k] = t * xb + 16 * (i ^ t);
  }
  const auto fill = [&](uint8_t* lds, int kb) {
#pragma unroll
    for (int n = 0; n < kGroups; ++n)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        load_lds(rx[n], xo[k], kb * (kStage * 2), lds + ((wave * kGroups + n) * 4 + k) * 1024);
  };
  typedef uint32_t v2u __attribute__((ext_vector_type(2)));
  const int ro = i * row_bytes + 8 * G, so = i * blocks * 2;
  struct Weights {
    v2u w[4];
    uint32_t d[4];
  };
  const auto fetch = [&](Weights& f, int kb) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      f.w[u] = __builtin_bit_cast(v2u, __builtin_amdgcn_raw_buffer_load_b64(rc[u], ro, kb * 32, 0));
      f.d[u] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rs[u], so, kb / 2 * 2, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };

  const uint32_t top = exponent_of_1024();
  v4f acc[4][NT];
#pragma unroll
  for (int u = 0; u < 4; ++u)
#pragma unroll
    for (int q = 0; q < NT; ++q) acc[u][q] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  const int row = (16 * NT * wc + i) * 256;
  // the weights of matrix instruction s of a block
  const auto decode = [&](v8h (&w)[4], const Weights& f, int s) {
#pragma unroll
    for (int u = 0; u < 4; ++u)
      w[u] = weights8((f.w[u][s >> 1] >> (16 * (s & 1))) & 0xFFFFu, __builtin_bit_cast(v2h, f.d[u] * 0x10001u), top);
  };
  // One block: w holds the weights of its first instruction, and those of the
  // next block's in the end.  Each instruction's weights are made while the one
  // before runs: two vector operations to a matrix instruction.
  const auto multiply = [&](const uint8_t* lds, v8h (&w)[4], const Weights& f, const Weights& next) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      v8h wn[4];
      if (s < 3) decode(wn, f, s + 1);
      else decode(wn, next, 0);
#pragma unroll
      for (int q = 0; q < NT; ++q) {
        const v8h x = *(const v8h*)(lds + row + q * 4096 + 16 * ((4 * G + s) ^ i));
#pragma unroll
        for (int u = 0; u < 4; ++u) acc[u][q] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[u], x, acc[u][q], 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) w[u] = wn[u];
    }
    __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
#pragma unroll
    for (int n = 0; n < 4 * NT; ++n) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);
    }
  };
  // what was asked for a block ago has come, to every wave, and the other buffer has been read by every wave
  const auto ready = [&] {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };

  Weights f0, f1;
  v8h w[4];
  fill(lds0, 0);
  fetch(f0, 0);
  decode(w, f0, 0);
  const int last = 2 * blocks - 1;
  for (int kb = 0; kb < last; kb += 2) {
    ready();
    fill(lds1, kb + 1);
    fetch(f1, kb + 1);
    multiply(lds0, w, f0, f1);
    ready();
    const int next = kb + 2 < last ? kb + 2 : last;  // behind the last block it is read again, and not used
    fill(lds0, next);
    fetch(f0, next);
    multiply(lds1, w, f1, f0);
  }

  // lane (G, i): rows 4G .. 4G + 3 of each group, token i of each tile
#pragma unroll
  for (int q = 0; q < NT; ++q) {
    const int m = 16 * (NT * wc + q) + i;
    if (m >= toks) continue;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int n = 32 * wr + 16 * g + 4 * G;
      typename Elem<DST>::T* h = (typename Elem<DST>::T*)a.h + (m0 + m) * a.N + n0 + n;
      Vec<DST, 4> v;
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = (typename Elem<DST>::T)gate(acc[g][q][r], acc[2 + g][q][r]);
      if (a.N % 4 == 0) {
        if (n < rows) *(Vec<DST, 4>*)h = v;
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (n + r < rows) h[r] = v[r];
      }
    }
  }
}

template <int WR, int WC, int NT>
hipError_t launch_many(const GatedArgs& a, int out_dtype, hipStream_t st) {
  const dim3 grid((unsigned)((a.N + 32 * WR - 1) / (32 * WR)), (unsigned)((a.M + 16 * NT * WC - 1) / (16 * NT * WC)));
  const dim3 block(64 * WR * WC);
  if (out_dtype == kF16) hipLaunchKernelGGL((k_gated_many<WR, WC, NT, kF16>), grid, block, 0, st, a);
  else if (out_dtype == kBF16) hipLaunchKernelGGL((k_gated_many<WR, WC, NT, kBF16>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_gated_many<WR, WC, NT, kF32>), grid, block, 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gated(const GatedArgs& a, bool int8, int out_dtype, hipStream_t st) {
  if (!int8 && a.M > 64) return launch_many<4, 2, 8>(a, out_dtype, st);
  if (int8) return a.M <= 16 ? launch_few<true, 1>(a, out_dtype, st) : launch_few<true, 2>(a, out_dtype, st);
  return a.M <= 16 ? launch_few<false, 1>(a, out_dtype, st) : launch_few<false, 2>(a, out_dtype, st);
}

}  // namespace tq2
