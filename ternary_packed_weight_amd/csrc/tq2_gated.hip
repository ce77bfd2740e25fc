// gfx950 (MI355X, CDNA4) kernels of the gated projections: h = silu(Wg x) *
// (Wu x) of two ternary matrices for any number of tokens.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

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

// 16 bytes a lane from a buffer straight to LDS, lane l's at lds + 16 l
__device__ __forceinline__ void load_lds(__amdgpu_buffer_rsrc_t r, int at, int scalar, uint8_t* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, at, scalar, 0, 0);
}

// Eight codes (the low 16 bits of c, lowest first) as fp16 code - 1, exact.  t
// holds code 2j at bit 4j and code 2j + 1 at bit 4j + 16, so a mask and the
// exponent of 1024 make the pair 1024 + 16^j code, and one fused multiply-add
// the pair code - 1.  11 operations for 8 weights, and the weights come in the
// order of K: activations go to the matrix cores as they lie in memory.  `top`
// is 0x64006400 in a vector register: an and-or takes one scalar.
__device__ __forceinline__ uint32_t exponent_of_1024() {
  uint32_t c;
  asm("v_mov_b32 %0, 0x64006400" : "=v"(c));
  return c;
}
__device__ __forceinline__ v2h both(float f) { return v2h{(_Float16)f, (_Float16)f}; }
struct Signs {
  v2h p[4];
};
__device__ __forceinline__ Signs signs8(uint32_t c, uint32_t top) {
  const uint32_t t = c | (c << 14);
  const auto pair = [&](uint32_t w, uint32_t mask) { return __builtin_bit_cast(v2h, (w & mask) | top); };
  return {{pair(t, 0x00030003u) - both(1025.0f),
           __builtin_elementwise_fma(pair(t, 0x00300030u), both(0.0625f), both(-65.0f)),
           __builtin_elementwise_fma(pair(t, 0x03000300u), both(0.00390625f), both(-5.0f)),
           __builtin_elementwise_fma(pair(t >> 8, 0x00300030u), both(0.0625f), both(-65.0f))}};
}
__device__ __forceinline__ v8h joined(const Signs& s) {
  return v8h{s.p[0][0], s.p[0][1], s.p[1][0], s.p[1][1], s.p[2][0], s.p[2][1], s.p[3][0], s.p[3][1]};
}
// Sixteen codes, inverted (3, 2, 1 for 0, 1, 2), as fp16 2 * (code - 1): the
// two bits are the top of -2, -0 and 2, so nothing is computed, and a shift and
// a mask put two codes in place.  Codes j and j + 8 share a pair; the first
// eight of the result are pairs 0 .. 3, the second eight pairs 4 .. 7.
__device__ __forceinline__ v8h doubles8(uint32_t n, int second) {
  const int j = second ? 6 : 14;
  const auto pair = [&](int shift) { return (shift ? n << shift : n) & 0xC000C000u; };
  return __builtin_bit_cast(v8h, v4u{pair(j), pair(j - 2), pair(j - 4), pair(j - 6)});
}
// Sixteen fp16 activations in the order of these pairs.
__device__ __forceinline__ void paired(v4u& a, v4u& b) {
  const v4u x = a, y = b;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t lo = __builtin_amdgcn_perm(y[k], x[k], 0x05040100u), hi = __builtin_amdgcn_perm(y[k], x[k], 0x07060302u);
    (k < 2 ? a : b)[k % 2 * 2] = lo;
    (k < 2 ? a : b)[k % 2 * 2 + 1] = hi;
  }
}
// ... and sixteen int8 activations as fp16, exact: a byte with its top bit turned is x + 128, below the exponent of 1024.
__device__ __forceinline__ void paired(v4u x, v4u& a, v4u& b) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t lo = x[j / 4] ^ 0x80808080u, hi = x[2 + j / 4] ^ 0x80808080u;
    const uint32_t k = (uint32_t)j % 4, two = __builtin_amdgcn_perm(hi, lo, 0x0C000C00u | (4 + k) << 16 | k) | 0x64006400u;
    (j < 4 ? a : b)[j % 4] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(v2h, two) - v2h{(_Float16)1152.0f, (_Float16)1152.0f});
  }
}
// Eight codes as the weights d * (code - 1), exact: 15 operations.
__device__ __forceinline__ v8h weights8(uint32_t c, v2h d, uint32_t top) {
  Signs s = signs8(c, top);
#pragma unroll
  for (int j = 0; j < 4; ++j) s.p[j] *= d;
  return joined(s);
}
// silu(g) * u = g / (1 + e^-g) * u.  The exponential's argument is -g log2 e
// rounded to t, which alone makes e^-g up to |g| 2^-24 wrong: for fp32 outputs 30
// units in the last place at g = -80, for the others a hundredth of their own
// rounding.  So for fp32 what t leaves, r = -g - t ln 2, goes into the sum: 1 +
// 2^t e^r = 1 + 2^t + 2^t r.  (The constant is the next below log2 e: r > 0 for g
// < 0 then, and an infinite 2^t stays that; beyond 120 the quotient is 0 or 1
// anyway.)  Four operations an output: 77 tokens of 2 x 5461 x 2560 in fp32 19.7
// us without and 20.0 with them, 4096 tokens of 2 x 16384 x 4096 893 and 896.
template <bool EXACT>
__device__ __forceinline__ float gate(float g, float u) {
  if constexpr (EXACT) {
    const float c = __builtin_amdgcn_fmed3f(g, -120.0f, 120.0f), t = c * -0x1.715474p+0f;
    const float r = fmaf(t, 0x1.05c610p-29f, fmaf(t, -0x1.62e430p-1f, -c)), e = __builtin_amdgcn_exp2f(t);
    return g * __builtin_amdgcn_rcpf(fmaf(e, r, 1.0f + e)) * u;
  }
  return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504f)) * u;
}

__device__ __forceinline__ void store_gated(void* h, int64_t at, float g, float u, int dtype) {
  if (dtype == kF32) ((float*)h)[at] = gate<true>(g, u);
  else if (dtype == kF16) ((_Float16*)h)[at] = (_Float16)gate<false>(g, u);
  else ((__bf16*)h)[at] = (__bf16)gate<false>(g, u);
}

// ---- one token ----
//
// A row's 1 KiB of 4096 codes is one load of a wave: lane l takes places 64l ..
// 64l + 63 and holds their activations for all of its R rows.  Half of a
// workgroup's waves take gate rows, half the up rows of the same places, and C
// waves share a row's K.  A pair of weights costs two operations on bits and a
// product of two: `doubles8` makes -2, -0 and 2 of a code, so nothing is
// subtracted afterwards and a sum's error is that of its own terms.  2 x 16384
// rows of 4096 from memory: 11.6 us (3.0 TB/s); by the form for few tokens 12.6.
// The operations behind a wave's last load bound it.  Eight rows a wave took 0.2
// us more.
constexpr int kOneRows = kGatedOneRows;

template <int C>
__global__ __launch_bounds__(kGatedOneThreads, 4) void k_gated_one(GatedArgs a, int out_dtype) {
  constexpr int R = kOneRows, H = 4 / C;  // groups of R gate rows
  constexpr int kOut = 0x40000000;
  __shared__ v4u xs[C][8][64];  // of a chunk: piece, lane
  __shared__ float red[8][R];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = wave % C, slot = wave / C, p = slot / H;
  const int64_t n0 = ((int64_t)blockIdx.x * H + slot % H) * R;
  const int rows = a.N <= n0 ? 0 : a.N - n0 < R ? (int)(a.N - n0) : R;
  const int row_bytes = (int)(a.K / 4), blocks = (int)(a.K / 256), chunks = (blocks + 15) / 16;
  const __amdgpu_buffer_rsrc_t rc = buffer_of(a.codes[p] + (rows ? n0 : 0) * row_bytes, (uint32_t)(rows * row_bytes));
  const __amdgpu_buffer_rsrc_t rs = buffer_of(a.scales[p] + (rows ? n0 : 0) * blocks, (uint32_t)(rows * blocks * 2));
  const __amdgpu_buffer_rsrc_t rx = buffer_of(a.x, (uint32_t)(a.K * 2));
  float out[R];
#pragma unroll
  for (int r = 0; r < R; ++r) out[r] = 0.0f;
  for (int c0 = 0; c0 < chunks; c0 += C) {
    // activations before weights: the staging waits for these alone
    constexpr int kPasses = (C * 256 + 511) / 512;
    v4u x0[kPasses], x1[kPasses];
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
      const int at = (c0 * 256 + (int)threadIdx.x + k * 512) * 32;  // (past the last activation: zeros)
      x0[k] = load16(rx, at), x1[k] = load16(rx, at + 16);
    }
    __builtin_amdgcn_sched_barrier(0);
    v4u w[R];
    uint16_t d[R];
    const int block = (c0 + c) * 16 + lane / 4;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool on = block < blocks;
      w[r] = load16(rc, on ? r * row_bytes + (c0 + c) * 1024 + 16 * lane : kOut);
      d[r] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rs, on ? (r * blocks + block) * 2 : kOut, 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
    if (c0) __syncthreads();  // every wave has read the chunks before
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
      const int m = (int)threadIdx.x + k * 512;  // group of 16 activations
      paired(x0[k], x1[k]);
      if (m < C * 256) xs[m / 256][m % 4 * 2][m / 4 % 64] = x0[k], xs[m / 256][m % 4 * 2 + 1][m / 4 % 64] = x1[k];
    }
    __syncthreads();
    v4u x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = xs[c][k][lane];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float sum[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        sum[k] = 0.0f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const v4u v = __builtin_bit_cast(v4u, doubles8(~w[r][k], e));
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t two = v[j], act = x[2 * k + e][j];
            sum[k] = __builtin_amdgcn_fdot2(__builtin_bit_cast(v2h, two), __builtin_bit_cast(v2h, act), sum[k], false);
          }
        }
      }
      out[r] = fmaf((float)__builtin_bit_cast(_Float16, d[r]), (sum[0] + sum[1]) + (sum[2] + sum[3]), out[r]);
    }
  }
  // over the lanes: half of the rows go each way until one is left, then its sixteen lanes
  static_assert(R == 4, "two steps that halve");
  const bool up = lane & 32, odd = lane & 16;
#pragma unroll
  for (int r = 0; r < 2; ++r) out[r] = (up ? out[r + 2] : out[r]) + across<32>(up ? out[r] : out[r + 2], lane);
  out[0] = (odd ? out[1] : out[0]) + across<16>(odd ? out[0] : out[1], lane);
  out[0] += across<8>(out[0], lane);
  out[0] += across<4>(out[0], lane);
  out[0] += across<2>(out[0], lane);
  out[0] += across<1>(out[0], lane);
  if (lane % 16 == 0) red[wave][lane / 32 * 2 + lane / 16 % 2] = out[0];
  __syncthreads();
  if (threadIdx.x < H * R) {
    const int g = threadIdx.x / R, r = threadIdx.x % R;
    float q = red[g * C][r], u = red[(g + H) * C][r];
#pragma unroll
    for (int k = 1; k < C; ++k) q += red[g * C + k][r], u += red[(g + H) * C + k][r];
    const int64_t n = ((int64_t)blockIdx.x * H + g) * R + r;
    if (n < a.N) store_gated(a.h, n, 0.5f * q, 0.5f * u, out_dtype);
  }
}

// ---- few tokens ----
//
// The weights are streamed once, and a workgroup's C waves share K.  A wave
// takes blocks of 256 along K in turn, for 16*U/2 gate rows, the up rows of the
// same places and TT tiles of 16 tokens; the waves' sums meet in LDS and are
// added in their order.  Codes go straight to LDS, two blocks of them at a time
// (64 bytes of a row, a block, to registers took 3 us longer: a load touched 16
// lines), and no wave waits for another before the sums (with the scales staged
// by all: 1 us).  Activations are the instruction's rows and weights its
// columns: lane (G, i) = (l / 16, l % 16) holds token i's activations and row
// i's codes at places 64G + 16p .. + 15, which instructions 2p and 2p + 1 of a
// block take (in the order of `doubles8`), and gets the sums of tokens 4G .. 4G
// + 3 with row i, which have one scale: sums of x * 2 (code - 1) are scaled when
// a block is whole, so that a weight costs one operation on bits where making it
// of its scale costs 15/8.  What bounds it is the operations behind a wave's
// last load: a SIMD spends some 6 us on 2 x 16384 rows of 4096.
template <bool I8, int U, int TT, int C, int W>
__global__ __launch_bounds__(64 * C, W) void k_gated_few(GatedArgs a, int out_dtype) {
  constexpr int R = U / 2;                   // groups of 16 gate rows
  constexpr int kX = I8 ? 2 : 4;             // 16-byte pieces of a lane's activations of half a block
  constexpr int kRing = 2048 * U;            // a wave's codes of two blocks
  static_assert(TT <= 2, "the waves' sums fit where their codes were");
  // (arrays of their own: reads of one need not wait for loads into the other)
  __shared__ __attribute__((aligned(16))) uint8_t ring[C * kRing];
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  v4f(*red)[U][TT][64] = (v4f(*)[U][TT][64])ring;           // [C]
  const int lane = threadIdx.x & 63, G = lane >> 4, i = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * (16 * R), m0 = (int64_t)blockIdx.y * (16 * TT);
  const int rows = (int)(a.N - n0 < 16 * R ? a.N - n0 : 16 * R);
  const int toks = (int)(a.M - m0 < 16 * TT ? a.M - m0 : 16 * TT);
  const int row_bytes = (int)(a.K / 4), blocks = (int)(a.K / 256), xb = (int)a.K * (I8 ? 1 : 2);
  __amdgpu_buffer_rsrc_t rc[2];
#pragma unroll
  for (int p = 0; p < 2; ++p) rc[p] = buffer_of(a.codes[p] + n0 * row_bytes, (uint32_t)(rows * row_bytes));
  const __amdgpu_buffer_rsrc_t rx = buffer_of((const uint8_t*)a.x + m0 * xb, (uint32_t)(toks * xb));
  // the wave's blocks
  const int share = (blocks + C - 1) / C, first = wave * share;
  const int end = first + share < blocks ? first + share : blocks;
  const int held = 32 - __builtin_clz(share * 2 - 1) - 1;  // log2 of the places of a row's scales
  uint16_t* scale = (uint16_t*)lds + (wave * (32 * R) << held);  // [matrix][row][block of the wave]
  // Places of the lane's rows and tokens; those of rows and tokens past the last
  // one are past every buffer, and read as zeros without a read.
  constexpr int kOut = 0x40000000;
  int ro[2 * R], xo[TT];
#pragma unroll
  for (int g = 0; g < 2 * R; ++g) {
    const int r = 8 * g + lane / 8;
    ro[g] = r < rows ? r * row_bytes + 16 * (lane % 8 ^ lane / 8) : kOut;
  }
#pragma unroll
  for (int q = 0; q < TT; ++q) xo[q] = 16 * q + i < toks ? (16 * q + i) * xb + 64 * G * (I8 ? 1 : 2) : kOut;
  // Codes of blocks b and b + 1 straight to LDS: 128 bytes of 8 rows a load, the
  // 16-byte piece c of row r at place c ^ (r % 8), so that a read of 16 rows'
  // pieces meets every bank once.  (A row's last block alone: nothing behind it is read.)
  const auto fetch = [&](int b) {
    b = __builtin_amdgcn_readfirstlane(b);  // (known to be the same in all lanes)
    const bool off = b + 1 >= blocks && (lane % 8 ^ lane / 8) >= 4;
#pragma unroll
    for (int n = 0; n < 2 * U; ++n) {
      const int u = n / 2, g = u / 2 * 2 + n % 2;
      load_lds(rc[u & 1], off ? kOut : ro[g], 64 * b, ring + wave * kRing + n * 1024);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  struct Codes {
    v4u w[U];
  };
  const auto take = [&](Codes& f, int block) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      f.w[u] = ~*(const v4u*)(ring + wave * kRing + u * 2048 + i * 128 + 16 * ((4 * block + G) ^ (i & 7)));
    }
  };
  struct Half {
    v4u x[TT][kX];
  };
  const auto half = [&](Half& f, int b, int h) {
    if (b >= end) return;
    b = __builtin_amdgcn_readfirstlane(b);
#pragma unroll
    for (int q = 0; q < TT; ++q)
#pragma unroll
      for (int k = 0; k < kX; ++k) {
        const int at = (I8 ? 32 : 64) * h + 16 * k;
        f.x[q][k] = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(rx, xo[q] + at, (I8 ? 256 : 512) * b, 0));
      }
    __builtin_amdgcn_sched_barrier(0);
  };
  v4f acc[U][TT];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int q = 0; q < TT; ++q) acc[u][q] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  v4f sum[U][TT];
  const auto multiply = [&](const Codes& f, const Half& e, int b, int h) {
    const uint16_t* sc = scale + (i << held) + (b - first);
    v4u x[TT][4];
#pragma unroll
    for (int q = 0; q < TT; ++q)
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        if constexpr (I8) {
          paired(e.x[q][p], x[q][2 * p], x[q][2 * p + 1]);
        } else {
          x[q][2 * p] = e.x[q][2 * p], x[q][2 * p + 1] = e.x[q][2 * p + 1];
          paired(x[q][2 * p], x[q][2 * p + 1]);
        }
      }
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const v8h w = doubles8(f.w[u][2 * h + s / 2], s % 2);
#pragma unroll
        for (int q = 0; q < TT; ++q)
          sum[u][q] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, x[q][s]), w, h || s ? sum[u][q] : v4f{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
      }
      if (h) {
        const float d = (float)__builtin_bit_cast(_Float16, sc[((u & 1) * (16 * R) + (u >> 1) * 16) << held]);
#pragma unroll
        for (int q = 0; q < TT; ++q)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[u][q][r] = fmaf(d, sum[u][q][r], acc[u][q][r]);
      }
      // (else weights of many rows are made ahead, and registers spill)
      if constexpr (TT > 1) __builtin_amdgcn_sched_barrier(0);
    }
  };
  Codes f;
  Half e[2];
  // The scales of the wave's blocks go to LDS, where only this wave
  // looks: no wave waits for another's loads.  They are asked for before
  // anything else and taken there once everything else has been: loads come in
  // their order, and a wait for these between would hold the codes up by a trip
  // to memory.
  constexpr int kEarly = 2;  // of each matrix, or of each row
  const int places = 16 * R << held;
  __amdgpu_buffer_rsrc_t rs[2];
  uint16_t early[2][kEarly];
  const auto scale_at = [&](int o) {  // of place o, or past every buffer
    const int r = o >> held, b = first + (o & ((1 << held) - 1));
    return o < places && r < rows && b < end ? (r * blocks + b) * 2 : kOut;
  };
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    rs[p] = buffer_of(a.scales[p] + n0 * blocks, (uint32_t)(rows * blocks * 2));
#pragma unroll
    for (int k = 0; k < kEarly; ++k) early[p][k] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rs[p], scale_at(lane + 64 * k), 0, 0);
  }
  __builtin_amdgcn_sched_barrier(0);
  if (first < end) fetch(first);
#pragma unroll
  for (int n = 0; n < 2; ++n) half(e[n], first, n);
#pragma unroll
  for (int p = 0; p < 2; ++p) {
#pragma unroll
    for (int k = 0; k < kEarly; ++k)
      if (lane + 64 * k < places) scale[p * places + lane + 64 * k] = early[p][k];
    for (int o = lane + 64 * kEarly; o < places; o += 64)
      scale[p * places + o] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rs[p], scale_at(o), 0, 0);
  }
  __builtin_amdgcn_wave_barrier();
  for (int b = first; b < end; b += 2) {
    __builtin_amdgcn_s_waitcnt(0x0f70);  // the two blocks have come
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    take(f, 0);
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      multiply(f, e[n], b, n);
      half(e[n], b + 1, n);
    }
    take(f, 1);
    // Both are read: the next two go out, behind the activations that the
    // second one takes (a wait for those would be one for these too).
    __builtin_amdgcn_s_waitcnt(0xc07f);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    if (b + 2 < end) fetch(b + 2);
    if (b + 1 >= end) break;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      multiply(f, e[n], b + 1, n);
      half(e[n], b + 2, n);
    }
  }
  __syncthreads();  // every wave is done with its codes: its sums go there
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int q = 0; q < TT; ++q) red[wave][u][q][lane] = acc[u][q];
  __syncthreads();
  // output (row n of the workgroup, token m): lane (m % 16 / 4, n % 16), element m % 4
  for (int o = threadIdx.x; o < 16 * R * 16 * TT; o += 64 * C) {
    const int n = o % (16 * R), m = o / (16 * R);
    if (n >= rows || m >= toks) continue;
    const int l = m % 16 / 4 * 16 + n % 16, u = 2 * (n / 16), q = m / 16;
    float g = red[0][u][q][l][m % 4], p = red[0][u + 1][q][l][m % 4];
#pragma unroll
    for (int c = 1; c < C; ++c) g += red[c][u][q][l][m % 4], p += red[c][u + 1][q][l][m % 4];
    float s = 0.5f;  // (weights were doubled)
    if constexpr (I8) s *= a.x_scales ? a.x_scales[m0 + m] : a.s;
    g *= s, p *= s;
    store_gated(a.h, (m0 + m) * a.N + n0 + n, g, p, out_dtype);
  }
}

// ---- many tokens ----
//
// A workgroup of WR waves (KS times as many) takes 32*WR gate rows with their up
// rows and 16*NT tokens; a wave 32 + 32 rows (two groups of 16 each) and all the
// tokens, and the sums stay in its registers.  K goes in blocks of 128: the
// tokens' activations of a block go straight to LDS (two blocks, one being
// filled while the other is used), the codes to registers, one block ahead.
// Where few workgroups would run, KS parts of a workgroup take blocks of K in
// turn, each with its own two blocks in LDS, and their sums are added at the
// end.  Lane (G, i) holds places 32G .. 32G + 31 of the block of row (token) i,
// of which matrix instruction s takes 8s .. 8s + 7.
//
// A weight is made by 15/8 operations, which run beside the matrix
// instructions: a wave's 64 rows by 128 tokens take 32 of those for every 4 x 15
// operations.  What bounds it is the power of the matrix cores: 4096 tokens, 2 x
// 16384 rows of 4096, 860 us = 1280 TFLOP/s at 2.0 to 2.25 of the 2.4 GHz; with
// activations and scales of one value the same code runs at 2.4.
constexpr int kStage = 128;

template <int WR, int NT, int KS, int DST>
__global__ __launch_bounds__(64 * WR * KS, KS > 1 ? 1 : 2) void k_gated_many(GatedArgs a) {
  constexpr int kTok = 16 * NT, kBytes = kTok * kStage * 2;
  // (an array each: reads of one need not wait for loads into another)
  __shared__ __attribute__((aligned(16))) uint8_t lds0[KS * kBytes], lds1[KS * kBytes];
  const int lane = threadIdx.x & 63, G = lane >> 4, i = lane & 15;
  const int index = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wave = index % WR, part = index / WR;
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
    const int r0 = 32 * wave + 16 * (u & 1), valid = rows < r0 ? 0 : rows - r0 < 16 ? rows - r0 : 16;
    const int64_t at = valid ? n0 + r0 : 0;
    rc[u] = buffer_of(a.codes[u >> 1] + at * row_bytes, (uint32_t)(valid * row_bytes));
    rs[u] = buffer_of(a.scales[u >> 1] + at * blocks, (uint32_t)(valid * blocks * 2));
  }
  // the wave's share of a block's activations: a load brings 4 tokens' 256
  // bytes; the 16-byte piece c of token t lies at place c ^ (t % 16) of its
  // row, so that a read of 16 tokens' pieces meets every bank once
  constexpr int kGroups = NT / WR;
  static_assert(kGroups * WR == NT, "groups of 16 tokens, as many for each wave");
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
        load_lds(rx[n], xo[k], kb * (kStage * 2), lds + part * kBytes + ((wave * kGroups + n) * 4 + k) * 1024);
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
  // the weights of matrix instruction s of a block
  const auto decode = [&](v8h (&w)[4], const Weights& f, int s) {
#pragma unroll
    for (int u = 0; u < 4; ++u)
      w[u] = weights8((f.w[u][s >> 1] >> (16 * (s & 1))) & 0xFFFFu, __builtin_bit_cast(v2h, f.d[u] * 0x10001u), top);
  };
  // One block.  (An instruction's operands before its products, and no more of
  // them: made ahead by the compiler they spill.)
  const auto multiply = [&](const uint8_t* lds, const Weights& f) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      v8h w[4], x[NT];
#pragma unroll
      for (int q = 0; q < NT; ++q) x[q] = *(const v8h*)(lds + part * kBytes + i * 256 + q * 4096 + 16 * ((4 * G + s) ^ i));
      decode(w, f, s);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int q = 0; q < NT; ++q)
#pragma unroll
        for (int u = 0; u < 4; ++u) acc[u][q] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[u], x[q], acc[u][q], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // A block has come, to every wave, and the other array has been read by every wave.
  const auto ready = [&] {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0x70);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };

  const int last = 2 * blocks - 1;
  Weights f[2];
  const auto ask = [&](uint8_t* lds, Weights& to, int kb) {
    kb = kb < last ? kb : last;  // behind the last block it is read again, and not used
    fill(lds, kb);
    fetch(to, kb);
  };
  uint8_t* const lds[2] = {lds0, lds1};
  ask(lds0, f[0], part);
  // (parts whose blocks end earlier go on to the last barrier)
  for (int kb = 0; kb <= last; kb += 2 * KS) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int at = kb + k * KS;
      if (k && KS > 1 && at > last) break;
      ready();
      ask(lds[1 - k], f[1 - k], at + part + KS);
      if (KS == 1 || at + part <= last) multiply(lds[k], f[k]);
    }
  }
  __builtin_amdgcn_s_waitcnt(0x0f70);  // nothing comes into LDS that may be another workgroup's then
  if constexpr (KS > 1) {
    // the parts' sums, the upper half of them added to the lower one until one is left
    v4f* red = (v4f*)lds0;
    static_assert(KS / 2 * WR * 4 * NT * 1024 <= KS * kBytes, "half of the parts fit one array");
#pragma unroll
    for (int h = KS / 2; h; h /= 2) {
      __syncthreads();
      v4f* const at = red + ((part % h) * WR + wave) * (4 * NT * 64) + lane;
#pragma unroll
      for (int n = 0; n < 4 * NT; ++n)
        if (part >= h && part < 2 * h) at[n * 64] = acc[n % 4][n / 4];
      __syncthreads();
#pragma unroll
      for (int n = 0; n < 4 * NT; ++n)
        if (part < h) acc[n % 4][n / 4] += at[n * 64];
    }
    if (part) return;
  }

  // lane (G, i): rows 4G .. 4G + 3 of each group, token i of each tile
#pragma unroll
  for (int q = 0; q < NT; ++q) {
    const int m = 16 * q + i;
    if (m >= toks) continue;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int n = 32 * wave + 16 * g + 4 * G;
      typename Elem<DST>::T* h = (typename Elem<DST>::T*)a.h + (m0 + m) * a.N + n0 + n;
      Vec<DST, 4> v;
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = (typename Elem<DST>::T)gate<DST == kF32>(acc[g][q][r], acc[2 + g][q][r]);
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

// ---- many tokens, 8-bit activations ----
//
// The matrix cores multiply numbers of four bits (e2m1) by numbers of six (e2m3)
// at four times their binary16 rate.  An inverted code is the top half of the
// four bits of -2, -0 or 2, so 16 weights are three operations on bits; and x_q
// = 16 hi + lo with lo in -8 .. 7 and hi in -8 .. 8, both exact in six bits (a
// magnitude of 0 .. 15 eighths is its own bits).  The instruction's powers of
// two per 32 places undo the factors.  A block's sums are whole and at most 2^15,
// so they are exact, and these times the row's scale are added in fp32.
//
// k_split_i8 writes the pieces once, in the order in which the product's LDS
// wants them.  Unit (c, G, p) of a token and block is piece p (lo, hi) of places
// 64G + 32c .. + 31: 32 six-bit numbers in the order of the weights' (places 0,
// 2, .. 14, 1, 3, .. 15 of each 16), 24 bytes.  For 16 tokens and a block, 6
// KiB: first 16 bytes of every unit (token t's unit n at t * 256 + 16 * (n ^
// t)), then 8 bytes of every unit (4096 + t * 128 + 8 * (n ^ t)); n = 8c + 2G +
// p.  The exclusive or makes 16 tokens' reads of one unit meet every bank once.
constexpr int kPieces = 6144;  // bytes of 16 tokens and a block
constexpr int kSlab = 128;     // tokens of a workgroup

__global__ __launch_bounds__(256) void k_split_i8(const int8_t* __restrict__ x, int64_t M, int64_t K, uint8_t* __restrict__ to) {
  const int blocks = (int)(K / 256);
  const int64_t job = (int64_t)blockIdx.x * 256 + threadIdx.x;  // (group of 16 tokens, block, half unit, token)
  const int t = (int)(job % 16), cg = (int)(job / 16 % 8), c = cg / 4, G = cg % 4;
  const int64_t gb = job / 128, m = gb / blocks * 16 + t;
  const int b = (int)(gb % blocks);
  uint32_t lo[6] = {0, 0, 0, 0, 0, 0}, hi[6] = {0, 0, 0, 0, 0, 0};
  if (m < M) {
    const uint4* src = (const uint4*)(x + m * K + 256 * b + 64 * G + 32 * c);
    const uint4 v[2] = {src[0], src[1]};
    const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const int k = e / 16 * 16 + e % 8 * 2 + e / 8 % 2;  // the place that element e holds
      const int q = (int)(int8_t)(w[k / 4] >> (8 * (k % 4)));
      const int l = ((q + 8) & 15) - 8, h = (q - l) >> 4;
      const uint32_t le = (uint32_t)(l < 0 ? 32 - l : l), he = (uint32_t)(h < 0 ? 32 - h : h);
      const int at = 6 * e % 32, d = 6 * e / 32;
      lo[d] |= le << at, hi[d] |= he << at;
      if (at > 26) lo[d + 1] |= le >> (32 - at), hi[d + 1] |= he >> (32 - at);
    }
  }
  uint8_t* base = to + gb * kPieces;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const uint32_t* u = p ? hi : lo;
    const int n = (8 * c + 2 * G + p) ^ t;
    *(uint4*)(base + t * 256 + 16 * n) = make_uint4(u[0], u[1], u[2], u[3]);
    *(uint2*)(base + 4096 + t * 128 + 8 * n) = make_uint2(u[4], u[5]);
  }
}

typedef int v8i __attribute__((ext_vector_type(8)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

template <int WR, int NT, int DST>
__global__ __launch_bounds__(64 * WR, 2) void k_gated_many_i8(GatedArgs a) {
  constexpr int kTok = 16 * NT, kBytes = NT * kPieces;
  static_assert(kTok <= 64 * WR, "a thread for each token's scale");
  __shared__ __attribute__((aligned(16))) uint8_t lds0[kBytes], lds1[kBytes];
  const int lane = threadIdx.x & 63, G = lane >> 4, i = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * (32 * WR), m0 = (int64_t)blockIdx.y * kTok;
  const int rows = (int)(a.N - n0 < 32 * WR ? a.N - n0 : 32 * WR);
  const int toks = (int)(a.M - m0 < kTok ? a.M - m0 : kTok);
  const int row_bytes = (int)(a.K / 4), blocks = (int)(a.K / 256);
  __amdgpu_buffer_rsrc_t rc[4], rs[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int r0 = 32 * wave + 16 * (u & 1), valid = rows < r0 ? 0 : rows - r0 < 16 ? rows - r0 : 16;
    const int64_t at = valid ? n0 + r0 : 0;
    rc[u] = buffer_of(a.codes[u >> 1] + at * row_bytes, (uint32_t)(valid * row_bytes));
    rs[u] = buffer_of(a.scales[u >> 1] + at * blocks, (uint32_t)(valid * blocks * 2));
  }
  // the pieces of the workgroup's tokens: whole groups of 16, those past the last token are zeros
  const int pitch = blocks * kPieces;  // of a group
  const __amdgpu_buffer_rsrc_t rx = buffer_of((const uint8_t*)a.pieces + (int64_t)blockIdx.y * NT * pitch, (uint32_t)(NT * pitch));
  constexpr int kLoads = 6 * NT / WR;
  static_assert(kLoads * WR == 6 * NT, "as many loads for each wave");
  const auto fill = [&](uint8_t* lds, int b, int n) {
    const int k = wave * kLoads + n;
    load_lds(rx, lane * 16, k / 6 * pitch + b * kPieces + k % 6 * 1024, lds + k * 1024);
  };
  const int ro = i * row_bytes + 16 * G, so = i * blocks * 2;
  v4u f[4];
  uint16_t fd[4];
  // load n of what a block needs: its codes, its scales, its activations
  const auto ask = [&](uint8_t* lds, int b, int n) {
    if (n < 4) f[n] = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(rc[n % 4], ro, b * 64, 0));
    else if (n < 8) fd[n % 4] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rs[n % 4], so, b * 2, 0);
    else fill(lds, b, n - 8);
  };

  v4f acc[4][NT];
#pragma unroll
  for (int u = 0; u < 4; ++u)
#pragma unroll
    for (int q = 0; q < NT; ++q) acc[u][q] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  // powers of two, exponent + 127: lo counts eighths, hi eighths of 16, a weight is half of -2, 0, 2
  constexpr int kLo = 127 + 3, kHi = 127 + 7, kHalf = 127 - 1;
  const auto block = [&](const uint8_t* lds, uint8_t* other, int b) {
    // this block has come, to every wave, and the other array has been read by every wave
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0x70);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    const int next = b + 1 < blocks ? b + 1 : b;  // behind the last block it is read again, and not used
    v8i w[4][2];
    float d[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      d[u] = (float)__builtin_bit_cast(_Float16, fd[u]);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint32_t v = f[u][2 * c], z = f[u][2 * c + 1], m = 0xCCCCCCCCu;
        w[u][c] = v8i{(int)(~(v << 2) & m), (int)(~v & m), (int)(~(z << 2) & m), (int)(~z & m), 0, 0, 0, 0};
      }
    }
    // Step t takes unit t % 4 of token group t / 4: its pieces are read two steps
    // ahead, and a group's sums are scaled while the next one's are formed.  The
    // next block's loads go out one a step: all at once they held the waves up
    // before they had multiplied anything.
    v8i e[3];
    v4f sum[2][4];
    const auto read = [&](int t) {
      const int q = t / 4, n = (8 * (t / 2 % 2) + 2 * G + t % 2) ^ i;
      const v4u x = *(const v4u*)(lds + q * kPieces + i * 256 + 16 * n);
      const v2u y = *(const v2u*)(lds + q * kPieces + 4096 + i * 128 + 8 * n);
      e[t % 3] = v8i{(int)x[0], (int)x[1], (int)x[2], (int)x[3], (int)y[0], (int)y[1], 0, 0};
    };
    const auto scaled = [&](int q) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[u][q][r] = fmaf(d[u], sum[q % 2][u][r], acc[u][q][r]);
    };
    read(0);
    read(1);
#pragma unroll
    for (int t = 0; t < 4 * NT; ++t) {
      const int q = t / 4, c = t / 2 % 2, p = t % 2;
      if (t + 2 < 4 * NT) read(t + 2);
      if (t < 8 + kLoads) ask(other, next, t);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        sum[q % 2][u] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            e[t % 3], w[u][c], t % 4 ? sum[q % 2][u] : v4f{0.0f, 0.0f, 0.0f, 0.0f}, 2, 4, 0, p ? kHi : kLo, 0, kHalf);
      if (t % 4 == 1 && q) scaled(q - 1);
      __builtin_amdgcn_sched_barrier(0);
    }
    scaled(NT - 1);
  };
#pragma unroll
  for (int n = 0; n < 8 + kLoads; ++n) ask(lds0, 0, n);
  for (int b = 0; b < blocks - 1; b += 2) {
    block(lds0, lds1, b);
    block(lds1, lds0, b + 1);
  }
  if (blocks % 2) block(lds0, lds1, blocks - 1);
  __builtin_amdgcn_s_waitcnt(0x0f70);  // nothing comes into LDS that may be another workgroup's then

  // lane (G, i), element r: token 4G + r of each group, weight row i of each
  // group.  (The tokens' scales through LDS: loaded where they are used, they
  // made every group of 16 tokens wait for memory, a third of the kernel.)
  __syncthreads();
  float* xs = (float*)lds0;
  if (threadIdx.x < kTok) xs[threadIdx.x] = !a.x_scales ? a.s : (int)threadIdx.x < toks ? a.x_scales[m0 + threadIdx.x] : 0.0f;
  __syncthreads();
  typedef typename Elem<DST>::T T;
  T* h = (T*)a.h + (m0 + 4 * G) * a.N + n0 + 32 * wave + i;
#pragma unroll
  for (int q = 0; q < NT; ++q) {
    const v4f s = *(const v4f*)(xs + 16 * q + 4 * G);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (16 * q + 4 * G + r < toks) {
#pragma unroll
        for (int g = 0; g < 2; ++g)
          if (32 * wave + 16 * g + i < rows) h[16 * g] = (T)gate<DST == kF32>(s[r] * acc[g][q][r], s[r] * acc[2 + g][q][r]);
      }
      h += r < 3 ? a.N : 13 * a.N;
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

// ---- the launches ----

#define TQ2_GATED_OF(kernel, ...)                                                                          \
  do {                                                                                                     \
    if (out_dtype == kF16) hipLaunchKernelGGL((kernel<__VA_ARGS__, kF16>), grid, block, 0, st, a);         \
    else if (out_dtype == kBF16) hipLaunchKernelGGL((kernel<__VA_ARGS__, kBF16>), grid, block, 0, st, a);  \
    else hipLaunchKernelGGL((kernel<__VA_ARGS__, kF32>), grid, block, 0, st, a);                           \
  } while (0)

// Compute units of the current device.
int cus() {
  static const int n = [] {
    int dev = 0, v = 0;
    return hipGetDevice(&dev) == hipSuccess && hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) == hipSuccess && v > 0 ? v : 256;
  }();
  return n;
}

constexpr int64_t kMostOf64 = 32768;  // K of which the scales of 64 rows find room beside their codes in LDS

template <bool I8, int U, int TT, int W>
hipError_t launch_few(const GatedArgs& a, int out_dtype, hipStream_t st) {
  constexpr int C = 8;
  const dim3 grid((unsigned)((a.N + 8 * U - 1) / (8 * U)), (unsigned)((a.M + 16 * TT - 1) / (16 * TT)));
  const auto kernel = k_gated_few<I8, U, TT, C, W>;
  const auto bytes = [](int64_t K) {  // a place for each scale of a wave's blocks
    int places = 1;
    while (places * C < K / 256) places *= 2;
    return (int)(C * places * 32 * U);
  };
  const int most = bytes(U == 8 ? kMostOf64 : 65536);
  static std::atomic<uint64_t> allowed{0};  // a bit for each device
  int dev = 0;
  if (const hipError_t e = hipGetDevice(&dev)) return e;
  if (dev >= 64 || !(allowed.load(std::memory_order_relaxed) >> dev & 1)) {
    if (const hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, most)) return e;
    if (dev < 64) allowed.fetch_or((uint64_t)1 << dev, std::memory_order_relaxed);
  }
  hipLaunchKernelGGL(kernel, grid, dim3(64 * C), bytes(a.K), st, a, out_dtype);
  return hipGetLastError();
}

// Gate rows of a workgroup (8 U): 32 where they still give three quarters of the
// compute units one, else 16 (32 tokens of int8 through 2 x 6144 rows of 4096
// 12.1, 14.1 us); more of them read the activations less often and fewer put more
// waves on a unit: 2 x 16384 rows of 4096 from memory with U = 8 / 4: 2 tokens
// 13.7 / 12.7 us, 8 tokens 14.6 / 13.5, 12 tokens 15.6 / 15.6, 16 tokens 16.2 /
// 17.2, 32 tokens (twice as many workgroups) 28.9 / 26.8; int8, half the bytes, 16
// tokens 15.9 / 14.9.
template <bool I8>
hipError_t launch_few(const GatedArgs& a, int out_dtype, hipStream_t st) {
  const auto fill = [&](int64_t rows) { return 4 * ((a.N + rows - 1) / rows) >= 3 * cus(); };
  if constexpr (I8) {
    if (a.M > 16) return fill(32) ? launch_few<I8, 4, 2, 2>(a, out_dtype, st) : launch_few<I8, 2, 2, 2>(a, out_dtype, st);
  } else {
    if (a.M > 12 && a.M <= 16 && fill(64) && a.K <= kMostOf64) return launch_few<I8, 8, 1, 2>(a, out_dtype, st);
  }
  return fill(32) ? launch_few<I8, 4, 1, 4>(a, out_dtype, st) : launch_few<I8, 2, 1, 4>(a, out_dtype, st);
}

hipError_t launch_one(const GatedArgs& a, int out_dtype, hipStream_t st) {
  const dim3 grid((unsigned)gated_one_groups(a.N, a.K)), block(kGatedOneThreads);
  const int waves = gated_one_waves(a.K);
  if (waves == 1) hipLaunchKernelGGL(k_gated_one<1>, grid, block, 0, st, a, out_dtype);
  else if (waves == 2) hipLaunchKernelGGL(k_gated_one<2>, grid, block, 0, st, a, out_dtype);
  else hipLaunchKernelGGL(k_gated_one<4>, grid, block, 0, st, a, out_dtype);
  return hipGetLastError();
}

template <int WR, int NT, int KS>
hipError_t launch_many(const GatedArgs& a, int out_dtype, hipStream_t st) {
  const dim3 grid((unsigned)((a.N + 32 * WR - 1) / (32 * WR)), (unsigned)((a.M + 16 * NT - 1) / (16 * NT)));
  const dim3 block(64 * WR * KS);
  TQ2_GATED_OF(k_gated_many, WR, NT, KS);
  return hipGetLastError();
}

// Tokens go through the pieces' workspace in slabs of whole workgroups.
int64_t slab_tokens(int64_t K, int64_t M) {
  const int64_t per = kSlab / 16 * (K / 256) * kPieces, most = (M + kSlab - 1) / kSlab;
  const int64_t fit = kGatedWorkspace / per;
  return (fit < most ? fit : most) * kSlab;
}

hipError_t launch_many_i8(const GatedArgs& whole, int out_dtype, hipStream_t st) {
  const int64_t slab = slab_tokens(whole.K, whole.M), K = whole.K;
  for (int64_t m = 0; m < whole.M; m += slab) {
    GatedArgs a = whole;
    a.M = whole.M - m < slab ? whole.M - m : slab;
    a.x = (const int8_t*)whole.x + m * K;
    if (a.x_scales) a.x_scales += m;
    a.h = (uint8_t*)whole.h + m * whole.N * (out_dtype == kF32 ? 4 : 2);
    const int64_t groups = (a.M + kSlab - 1) / kSlab * (kSlab / 16), jobs = groups * (K / 256) * 128;
    hipLaunchKernelGGL(k_split_i8, dim3((unsigned)(jobs / 256)), dim3(256), 0, st, (const int8_t*)a.x, a.M, K, (uint8_t*)a.pieces);
    // 512 rows by 128 tokens, or, while they all run at once (two a CU), 256 by
    // 64: 2 x 16384 rows of 4096 from memory with 128 / 256 / 512 / 4096 tokens 62 /
    // 63 / 70 / 491 us and 35 / 52 / 91 / 641.
    if ((a.N + 127) / 128 * ((a.M + 63) / 64) <= 2 * cus()) {
      const dim3 grid((unsigned)((a.N + 127) / 128), (unsigned)((a.M + 63) / 64)), block(256);
      TQ2_GATED_OF(k_gated_many_i8, 4, 4);
    } else {
      const dim3 grid((unsigned)((a.N + 255) / 256), (unsigned)((a.M + 127) / 128)), block(512);
      TQ2_GATED_OF(k_gated_many_i8, 8, 8);
    }
  }
  return hipGetLastError();
}

constexpr int64_t kFewTokens8 = 32;

}  // namespace

size_t gated_workspace_bytes(int64_t K, int64_t M, bool int8) {
  return int8 && M > kFewTokens8 ? (size_t)(slab_tokens(K, M) / 16 * (K / 256) * kPieces) : 0;
}

// Which form takes a call, by its tokens and by its workgroups for each compute
// unit; times are of 2 x 16384 rows of 4096 unless stated, weights from memory.
hipError_t launch_gated(const GatedArgs& a, bool int8, int out_dtype, hipStream_t st) {
  if (int8) return a.M > kFewTokens8 ? launch_many_i8(a, out_dtype, st) : launch_few<true>(a, out_dtype, st);
  if (a.M == 1 && gated_one_fits(a.N, a.K)) return launch_one(a, out_dtype, st);
  // Groups of 16 tokens up to 32, and up to 64 while their grid has at most four
  // workgroups a CU (LDS has room for two at once, so that is two rounds of them):
  // 32 / 48 / 64 tokens 26.8 / 35.9 / 44.6 us, and 29.9 / 30.2 / 30.8 by the form
  // below; 64 tokens through 2 x 6144 rows 20.1 and 29.2, 32 through 2 x 8192 15.5
  // and 28.6.  (The grid would carry more tokens too: 77 through 2 x 5461 rows of
  // 2560 take 19.9 and 20.4, 128 through 2 x 4096 24.2 and 29.0.)
  if (a.M <= 32 || (a.M <= 64 && (a.N + 31) / 32 * ((a.M + 15) / 16) <= 4 * cus())) return launch_few<false>(a, out_dtype, st);
  // While they all run at once (one a CU), 64 rows by 64 or 128 tokens, whose
  // waves share K: 64 / 128 tokens 31 / 47 us, and 62 / 65 by the form below; 77
  // tokens through 2 x 5461 rows of 2560 20, 30 (by 128 tokens) and 43.  256
  // tokens: 69 us below, 91 as two rounds of these.
  const auto at_once = [&](int64_t tokens) { return (a.N + 63) / 64 * ((a.M + tokens - 1) / tokens) <= cus(); };
  if (at_once(64)) return launch_many<2, 4, 4>(a, out_dtype, st);
  if (at_once(128)) return launch_many<2, 8, 2>(a, out_dtype, st);
  return launch_many<4, 8, 1>(a, out_dtype, st);
}

}  // namespace tq2
