// gfx950 (MI355X, CDNA4) kernels of the attention half of a decode step:
// norms and rotation of the query and key heads, the 4-bit key/value cache,
// and the attention that reads it.  Layout and launch interface: tq2_kv4.h.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "tq2_kv4.h"

namespace tq2 {
namespace {

typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

template <int DT>
struct Elem;
template <>
struct Elem<kF16> {
  typedef _Float16 T;
};
template <>
struct Elem<kBF16> {
  typedef __bf16 T;
};
template <>
struct Elem<kF32> {
  typedef float T;
};

// Eight consecutive elements as floats; one rounding (nearest even) on the way out.
template <int DT>
__device__ __forceinline__ void load8(const void* p, int64_t at, float (&x)[8]) {
  typedef typename Elem<DT>::T T;
  typedef T v8 __attribute__((ext_vector_type(8)));
  typedef T v4 __attribute__((ext_vector_type(4)));
  const T* e = (const T*)p + at;
  if constexpr (DT == kF32) {
    const v4 a = *(const v4*)e, b = *(const v4*)(e + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = a[i], x[4 + i] = b[i];
  } else {
    const v8 a = *(const v8*)e;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)a[i];
  }
}
template <int DT>
__device__ __forceinline__ void store8(void* p, int64_t at, const float (&x)[8]) {
  typedef typename Elem<DT>::T T;
  typedef T v8 __attribute__((ext_vector_type(8)));
  typedef T v4 __attribute__((ext_vector_type(4)));
  T* e = (T*)p + at;
  if constexpr (DT == kF32) {
    v4 a, b;
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = x[i], b[i] = x[4 + i];
    *(v4*)e = a;
    *(v4*)(e + 4) = b;
  } else {
    v8 a;
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = (T)x[i];
    *(v8*)e = a;
  }
}

// ---- norms and rotation ----

// y = x * rsqrt(mean(x^2) + eps) * w per head, then the rotation of channel
// pairs by position * inv_freq, in fp32 with one rounding at the end.  The
// angle is an exact fp64 product reduced by whole turns in fp64 (at a
// position of 10^6 an fp32 angle is off by 0.06 rad).  A workgroup takes a
// few tokens: every angle is turned into (cos, sin) once, in LDS, and shared
// by all heads of the token; 8 channels per lane, a power of two of lanes per
// head.  A lane reads its partners' channels itself (a second load of a line
// that is there) because the partner distance rot/2 need not be a power of two.
template <int SRC, int DST>
__global__ __launch_bounds__(256) void k_qk_norm_rope(RopeArgs a, int tokens, int heads_per_wg, int lanes) {
  extern __shared__ float2 turn[];  // [tokens][rot/2] (cos, sin)
  const int64_t t0 = (int64_t)blockIdx.x * tokens;
  const int nt = (int)(a.T - t0 < tokens ? a.T - t0 : tokens);
  const int h0 = blockIdx.y * heads_per_wg, H = a.Hq + a.Hk;
  const int nh = H - h0 < heads_per_wg ? H - h0 : heads_per_wg;
  const int half = a.rot / 2;
  for (int i = threadIdx.x; i < nt * half; i += 256) {
    const int t = i / half, f = i - t * half;
    const double turns = (double)a.positions[t0 + t] * (double)a.inv_freq[f] * 0.15915494309189533577;
    const float frac = (float)(turns - rint(turns));
    float c, s;
    sincospif(2.0f * frac, &s, &c);
    turn[i] = make_float2(c, s);
  }
  __syncthreads();
  const int l = threadIdx.x % lanes, d = 8 * l;
  const bool on = d < a.D;
  for (int it = threadIdx.x / lanes; it < nt * nh; it += 256 / lanes) {
    const int t = it / nh, hh = h0 + it - t * nh;
    const bool isq = hh < a.Hq;
    const int h = isq ? hh : hh - a.Hq;
    const void* src = isq ? a.q : a.k;
    const int64_t at = isq ? (t0 + t) * a.q_ts + h * a.q_hs : (t0 + t) * a.k_ts + h * a.k_hs;
    const float* w = isq ? a.q_weight : a.k_weight;
    float x[8] = {}, p[8] = {};
    // which channels pair with this lane's
    const bool turned = d < a.rot;
    const bool upper = d >= half;
    const int pd = upper ? d - half : d + half;
    if (on) {
      load8<SRC>(src, at + d, x);
      if (turned && !a.interleaved) load8<SRC>(src, at + pd, p);
    }
    if (w) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
      for (int o = lanes / 2; o > 0; o >>= 1) ss += __shfl_xor(ss, o, 64);
      const float r = 1.0f / sqrtf(ss / (float)a.D + a.eps);
      if (on) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[d + i];
        if (turned && !a.interleaved) {
#pragma unroll
          for (int i = 0; i < 8; ++i) p[i] = p[i] * r * w[pd + i];
        }
      }
    }
    if (!on) continue;
    if (turned) {
      const float2* cs = turn + t * half;
      if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 z = cs[d / 2 + i];
          const float u = x[2 * i], v = x[2 * i + 1];
          x[2 * i] = u * z.x - v * z.y;
          x[2 * i + 1] = v * z.x + u * z.y;
        }
      } else {
        const int f = upper ? d - half : d;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 z = cs[f + i];
          x[i] = x[i] * z.x + (upper ? p[i] : -p[i]) * z.y;
        }
      }
    }
    const int64_t out = ((t0 + t) * (isq ? a.Hq : a.Hk) + h) * a.D + d;
    store8<DST>(isq ? a.q_out : a.k_out, out, x);
  }
}

// ---- the cache: write and read back ----

// Per (token, head): z = f16((max+min)/2), s = f16((max-min)/15), code =
// clamp(rint((x-z)/s + 7.5), 0, 15), every fp32 step an IEEE one, so that the
// codes are the definition's bit for bit.  8 channels (one 32-bit word of
// codes) per lane, D/8 lanes per head.
template <int DT>
__global__ __launch_bounds__(256) void k_kv4_store(Kv4StoreArgs a) {
  const int lanes = a.D / 8, l = threadIdx.x % lanes;
  const int64_t it = (int64_t)blockIdx.x * (256 / lanes) + threadIdx.x / lanes;
  if (it >= a.T * a.Hk * 2) return;  // whole heads leave together
  const int64_t t = it / (2 * a.Hk);
  const int r = (int)(it - t * 2 * a.Hk);
  const bool isv = r >= a.Hk;
  const int h = isv ? r - a.Hk : r;
  int at;
  const int64_t block = kv4_slot_block(a.slots[t], a.pages, a.Hk, a.P, a.D, h, &at);
  if (block < 0) return;
  float x[8];
  load8<DT>(isv ? a.v : a.k, (isv ? t * a.v_ts + h * a.v_hs : t * a.k_ts + h * a.k_hs) + 8 * l, x);
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) lo = fminf(lo, x[i]), hi = fmaxf(hi, x[i]);
  for (int o = lanes / 2; o > 0; o >>= 1) {
    lo = fminf(lo, __shfl_xor(lo, o, 64));
    hi = fmaxf(hi, __shfl_xor(hi, o, 64));
  }
  const _Float16 z = (_Float16)((hi + lo) * 0.5f), s = (_Float16)((hi - lo) / 15.0f);
  uint32_t w = 0;
  if (s != (_Float16)0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float c = rintf((x[i] - (float)z) / (float)s + 7.5f);
      w |= (uint32_t)fminf(fmaxf(c, 0.f), 15.f) << (4 * i);
    }
  }
  uint8_t* b = a.cache + block;
  if (!isv) {
    *(uint32_t*)(b + kv4_key_at(a.D, at) + 4 * l) = w;
  } else {
    *(uint16_t*)(b + kv4_value_unit_at(a.P, a.D, at, 2 * l)) = (uint16_t)w;
    *(uint16_t*)(b + kv4_value_unit_at(a.P, a.D, at, 2 * l + 1)) = (uint16_t)(w >> 16);
  }
  if (l == 0) {
    const uint32_t pair = __builtin_bit_cast(uint16_t, s) | (uint32_t)__builtin_bit_cast(uint16_t, z) << 16;
    *(uint32_t*)(b + (isv ? kv4_value_pair_at(a.P, a.D, at) : kv4_key_pair_at(a.P, a.D, at))) = pair;
  }
}

// value = z + s*(code - 7.5); s*(code - 7.5) is exact in fp32.
template <int DT>
__global__ __launch_bounds__(256) void k_kv4_load(Kv4LoadArgs a) {
  const int lanes = a.D / 8, l = threadIdx.x % lanes;
  const int64_t it = (int64_t)blockIdx.x * (256 / lanes) + threadIdx.x / lanes;
  if (it >= a.T * a.Hk * 2) return;
  const int64_t t = it / (2 * a.Hk);
  const int r = (int)(it - t * 2 * a.Hk);
  const bool isv = r >= a.Hk;
  const int h = isv ? r - a.Hk : r;
  void* dst = isv ? a.v : a.k;
  if (!dst) return;
  int at;
  const int64_t block = kv4_slot_block(a.slots[t], a.pages, a.Hk, a.P, a.D, h, &at);
  float x[8] = {};
  if (block >= 0) {
    const uint8_t* b = a.cache + block;
    uint32_t w, pair;
    if (!isv) {
      w = *(const uint32_t*)(b + kv4_key_at(a.D, at) + 4 * l);
      pair = *(const uint32_t*)(b + kv4_key_pair_at(a.P, a.D, at));
    } else {
      w = *(const uint16_t*)(b + kv4_value_unit_at(a.P, a.D, at, 2 * l));
      w |= (uint32_t) * (const uint16_t*)(b + kv4_value_unit_at(a.P, a.D, at, 2 * l + 1)) << 16;
      pair = *(const uint32_t*)(b + kv4_value_pair_at(a.P, a.D, at));
    }
    const v2h sz = __builtin_bit_cast(v2h, pair);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float c = (float)((w >> (4 * i)) & 15) - 7.5f;
      x[i] = sz[0] == (_Float16)0 ? (float)sz[1] : fmaf((float)sz[0], c, (float)sz[1]);
    }
  }
  store8<DT>(dst, (t * a.Hk + h) * a.D + 8 * l, x);
}

// ---- attention ----

constexpr int kWaves = 4;          // waves of a workgroup, which share its token range
constexpr float kLazy = 8.0f;      // a row's reference moves when a score passes it by 2^8
constexpr float kNegInf = -INFINITY;

__device__ __forceinline__ float max_g(float v) {  // over the four lanes of a row
  v = fmaxf(v, __shfl_xor(v, 16, 64));
  return fmaxf(v, __shfl_xor(v, 32, 64));
}
__device__ __forceinline__ float sum_g(float v) {
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}
__device__ __forceinline__ float half_lo(uint32_t w) { return (float)__builtin_bit_cast(v2h, w)[0]; }
__device__ __forceinline__ float half_hi(uint32_t w) { return (float)__builtin_bit_cast(v2h, w)[1]; }

// The largest finite value scale (low half of a pair) of a row's 32 tokens, as bits.
__device__ __forceinline__ int largest_scale(const uint32_t (&pair)[8]) {
  int top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int s = pair[i] & 0xffff;
    top = s < 0x7c00 && s > top ? s : top;
  }
  const int u = __shfl_xor(top, 16, 64);
  top = u > top ? u : top;
  const int v = __shfl_xor(top, 32, 64);
  return v > top ? v : top;
}

// Four codes of a 32-bit word, two 16-bit halves each, as binary16
// subnormals: nibble 0 and 2 as c * 2^-24, nibble 1 and 3 as c * 2^-20.
__device__ __forceinline__ uint32_t nib(uint32_t w, int j) {
  const uint32_t s = j >= 2 ? w >> 8 : w;
  return s & (j & 1 ? 0x00f000f0u : 0x000f000fu);
}

// out = softmax(scale q K^T) V over the 4-bit cache; see tq2.h.
//
// A workgroup takes 16*MT rows (new token x query head) of one key head and a
// run of 32-token tiles, dealt to its four waves.  Per tile a wave computes
// the transposed scores K Q^T (v_mfma_f32_16x16x32_f16), so that a lane holds
// eight tokens of one row, which is already the operand layout of V^T P^T:
// the probabilities never cross lanes.  Codes enter the matrix cores as
// masked binary16 subnormals; a token's scale and middle are applied to its
// score and to its probability instead:
//   score = s_k (q.c - 7.5 sum q) + z_k sum q,  out = sum P s_v c - 7.5 sum P s_v + sum P z_v.
// Softmax statistics and sums are fp32.  P s_v is rounded once to binary16
// for the product, kept in [0, 2^12) by the row's running reference and its
// largest s_v so far (2^E); the -7.5 term sums the rounded values, so rounding
// acts on the centred codes.
template <int D, int MT, bool BF>
__global__ __launch_bounds__(64 * kWaves) void k_kv4_attn(Kv4AttnArgs a) {
  constexpr int NW = D / 32;   // 32-bit code words of a lane and token (keys)
  constexpr int NJ = D / 16;   // channels of a lane (values)
  typedef typename Elem<BF ? kBF16 : kF16>::T T;
  extern __shared__ float lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, g = lane >> 4;

  int id = blockIdx.x;
  const int split = id % a.nsplit;
  id /= a.nsplit;
  const int head = id % a.Hk;
  id /= a.Hk;
  const int b = id % a.B;
  const int row0 = (a.tiles - 1 - id / a.B) * 16 * MT;  // the longest causal ranges first

  const int64_t s0 = a.q_start ? a.q_start[b] : (int64_t)b * a.max_q;
  const int64_t s1 = a.q_start ? a.q_start[b + 1] : s0 + a.max_q;
  const int64_t q0 = s0 < 0 ? 0 : s0 > a.T ? a.T : s0;
  const int n = kv4_clamp((s1 > a.T ? a.T : s1) - q0, 0, a.max_q);
  const int c = kv4_clamp(a.ctx[b], 0, (int64_t)a.width * a.P);
  const int rows = n * a.G;
  if (row0 >= rows) return;
  const Kv4Range range = kv4_range(n, c, a.G, row0, 16 * MT, a.window, a.nsplit, kWaves);
  if (split > 0 && split >= range.splits) return;
  const int tbeg = range.first + split * range.chunk;
  const int tend = range.last < tbeg + range.chunk ? range.last : tbeg + range.chunk;

  // this lane's rows, one per row tile
  int lim[MT], low[MT];
  int64_t out_row[MT];
  bool valid[MT];
  v8h qf[MT][NW];
  float fa[MT], fb[MT], cinit[MT];
  int limmin = c, lowmax = 0;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int r = row0 + m * 16 + col;
    valid[m] = r < rows;
    const int i = valid[m] ? r / a.G : 0, h = valid[m] ? r - i * a.G : 0;
    const int pos = c - n + i;
    lim[m] = valid[m] ? pos + 1 : c;
    low[m] = valid[m] && a.window > 0 && pos >= a.window ? pos + 1 - a.window : 0;
    out_row[m] = (q0 + i) * a.Hq + head * a.G + h;
    limmin = lim[m] < limmin ? lim[m] : limmin;
    lowmax = low[m] > lowmax ? low[m] : lowmax;
    // D/4 channels of the row: scaled by a power of two into binary16's middle
    float x[D / 4];
    const T* qp = (const T*)a.q + (q0 + i) * a.q_ts + (head * a.G + h) * a.q_hs + g * (D / 4);
    float big = 0.f, sum = 0.f;
#pragma unroll
    for (int k = 0; k < D / 4; k += 8) {
      float y[8];
      load8<BF ? kBF16 : kF16>(qp, k, y);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[k + e] = valid[m] ? y[e] : 0.f;
        big = fmaxf(big, fabsf(x[k + e]));
        sum += x[k + e];
      }
    }
    big = max_g(big);
    sum = sum_g(sum);
    int ex = 0;
    if (big > 0.f && big < INFINITY) {
      ex = 8 - ilogbf(big);
      ex = ex > 100 ? 100 : ex < -100 ? -100 : ex;
    }
    const float up = ldexpf(1.0f, ex);
    float used = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int nibble = (e & 1 ? 4 : 0) + (e >> 1);  // slots 0 4 1 5 2 6 3 7 of the word
        const bool odd = nibble & 1;
        const _Float16 y = (_Float16)(x[w * 8 + nibble] * up * (odd ? 0.0625f : 1.0f));
        qf[m][w][e] = y;
        used += (float)y * (odd ? 16.0f : 1.0f);
      }
    }
    used = sum_g(used);
    cinit[m] = -7.5f * 0x1p-24f * used;
    const float to2 = a.scale * 1.44269504088896340736f;
    fa[m] = ldexpf(to2, 24 - ex);
    fb[m] = sum * to2;
  }
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) {
    const int u = __shfl_xor(limmin, o, 64), v = __shfl_xor(lowmax, o, 64);
    limmin = u < limmin ? u : limmin;
    lowmax = v > lowmax ? v : lowmax;
  }

  v4f acc[MT][NJ];
  float mrun[MT], lsum[MT], zsum[MT], rsum[MT];
  int E[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    mrun[m] = kNegInf;
    E[m] = -27;
    lsum[m] = zsum[m] = rsum[m] = 0.f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[m][j] = v4f{0.f, 0.f, 0.f, 0.f};
  }

  const int pshift = 31 - __builtin_clz(a.P) - 5;  // tiles of a page, as a shift
  for (int tile = tbeg + wave; tile < tend; tile += kWaves) {
    const int32_t page = a.table[b * a.table_stride + (tile >> pshift)];
    const int64_t block = kv4_page_block(page, a.pages, a.Hk, a.P, D, head);
    const uint8_t* base = a.cache + (block < 0 ? 0 : block);
    const int t32 = (tile & ((1 << pshift) - 1)) * 32;
    uint32_t kc[2][NW], vc[NJ], kp[8], vp[8];
    {
      const int tok = t32 + (col >> 2) * 8 + (col & 3);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t* p = (const uint32_t*)(base + kv4_key_at(D, tok + 4 * u) + g * (D / 8));
#pragma unroll
        for (int w = 0; w < NW; ++w) kc[u][w] = p[w];
      }
      const uint32_t* p = (const uint32_t*)(base + kv4_value_unit_at(a.P, D, t32, 0) + lane * (D / 4));
#pragma unroll
      for (int w = 0; w < NJ; ++w) vc[w] = p[w];
      const uint32_t* pk = (const uint32_t*)(base + kv4_key_pair_at(a.P, D, t32 + g * 8));
      const uint32_t* pv = (const uint32_t*)(base + kv4_value_pair_at(a.P, D, t32 + g * 8));
#pragma unroll
      for (int i = 0; i < 8; ++i) kp[i] = pk[i], vp[i] = pv[i];
    }
    const int j0 = tile * 32 + g * 8;
    const bool partial = block < 0 || tile * 32 + 32 > limmin || tile * 32 < lowmax;
    if (partial) {  // tokens that are not there: their pairs may hold anything
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (block < 0 || j0 + i >= c) kp[i] = vp[i] = 0;
    }
    int top = partial ? 0 : largest_scale(vp);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      float x[8];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        v4f d = {cinit[m], cinit[m], cinit[m], cinit[m]};
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          const v4u f = {nib(kc[u][w], 0), nib(kc[u][w], 1), nib(kc[u][w], 2), nib(kc[u][w], 3)};
          d = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, f), qf[m][w], d, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t p = kp[4 * u + i];
          x[4 * u + i] = fmaf(half_lo(p), d[i] * fa[m], half_hi(p) * fb[m]);
        }
      }
      uint32_t vq[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) vq[i] = vp[i];
      if (partial) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (block < 0 || j0 + i >= lim[m] || j0 + i < low[m]) {
            x[i] = kNegInf;
            vq[i] = 0;
          }
        }
        top = largest_scale(vq);  // of the tokens that this row sees
      }
      // the row's E follows the largest value scale it has seen
      float grow = 1.0f;  // 2^(old E - new E)
      if (top) {
        const int e = ilogbf((float)__builtin_bit_cast(_Float16, (uint16_t)top)) - 3;
        grow = e > E[m] ? ldexpf(1.0f, E[m] - e) : 1.0f;
        E[m] = e > E[m] ? e : E[m];
      }
      float mx = x[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) mx = fmaxf(mx, x[i]);
      mx = max_g(mx);
      const bool moves = mx > mrun[m] + kLazy;
      if (__builtin_amdgcn_ballot_w64(moves || grow != 1.0f)) {
        const float to = moves ? mx : mrun[m];
        const float f = grow * (to == kNegInf ? 1.0f : exp2f(mrun[m] - to));
        mrun[m] = to;
        lsum[m] *= f;
        zsum[m] *= f;
        rsum[m] *= f;
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[m][j] *= f;
      }
      const float ref = (mrun[m] == kNegInf ? 0.f : mrun[m]) + (float)E[m];
      v8h pf;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float p = exp2f(x[i] - ref);
        lsum[m] += p;
        const float s = half_lo(vq[i]);
        zsum[m] = fmaf(p, half_hi(vq[i]), zsum[m]);
        pf[i] = (_Float16)(p * s);
      }
#pragma unroll
      for (int i = 0; i < 8; i += 2)
        rsum[m] = __builtin_amdgcn_fdot2(v2h{pf[i], pf[i + 1]}, v2h{(_Float16)1, (_Float16)1}, rsum[m], false);
#pragma unroll
      for (int h = 0; h < NJ / 4; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const v4u f = {nib(vc[4 * h], j), nib(vc[4 * h + 1], j), nib(vc[4 * h + 2], j), nib(vc[4 * h + 3], j)};
          acc[m][4 * h + j] =
              __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, f), pf, acc[m][4 * h + j], 0, 0, 0);
        }
    }
  }

  // the waves' parts meet in LDS: [wave][16*MT rows][D + 4] sums, then
  // [wave][16*MT][2] (reference, weight)
  constexpr int LD = D + 4;
  float* ml = lds + kWaves * 16 * MT * LD;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const float l = sum_g(lsum[m]);
    const float shift = sum_g(zsum[m]) - 7.5f * sum_g(rsum[m]);
    float* o = lds + (wave * 16 * MT + m * 16 + col) * LD;
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int h = 0; h < NJ / 4; ++h) {
        v4f y;
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = fmaf(acc[m][4 * h + j][r], j & 1 ? 0x1p20f : 0x1p24f, shift);
        *(v4f*)(o + (g * 4 + r) * NJ + 4 * h) = y;
      }
    if (g == 0) {
      float* p = ml + (wave * 16 * MT + m * 16 + col) * 2;
      p[0] = mrun[m] == kNegInf ? kNegInf : mrun[m] + (float)E[m];
      p[1] = l;
    }
  }
  __syncthreads();
  constexpr int kParts = D / 8;  // threads of a row, 8 channels each
  for (int it = threadIdx.x; it < 16 * MT * kParts; it += 64 * kWaves) {
    const int row = it / kParts, d = (it - row * kParts) * 8;
    const int r = row0 + row;
    if (r >= rows) continue;
    float ref = kNegInf;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) ref = fmaxf(ref, ml[(w * 16 * MT + row) * 2]);
    float o[8] = {}, l = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float rw = ml[(w * 16 * MT + row) * 2];
      const float f = rw == kNegInf ? 0.f : exp2f(rw - ref);
      const float* p = lds + (w * 16 * MT + row) * LD + d;
      l = fmaf(f, ml[(w * 16 * MT + row) * 2 + 1], l);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = rw == kNegInf ? o[i] : fmaf(f, p[i], o[i]);
    }
    const int i = r / a.G;
    const int64_t orow = (q0 + i) * a.Hq + head * a.G + (r - i * a.G);
    if (range.splits <= 1) {
      const float inv = ref == kNegInf ? 0.f : 1.0f / l;
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] *= inv;
      store8<BF ? kBF16 : kF16>(a.out, orow * D + d, o);
      if (a.lse && d == 0) a.lse[orow] = ref == kNegInf ? kNegInf : (ref + log2f(l)) * 0.69314718055994530942f;
    } else {
      store8<kF32>(a.part, (orow * a.nsplit + split) * D + d, o);
      if (d == 0) {
        float* p = a.part + a.T * a.Hq * a.nsplit * D + (orow * a.nsplit + split) * 2;
        p[0] = ref;
        p[1] = l;
      }
    }
  }
}

// Joins the splits of a row: one workgroup per row, D/4 lanes a split.
template <int D, bool BF>
__global__ __launch_bounds__(256) void k_kv4_join(Kv4AttnArgs a, int mt) {
  constexpr int LN = D / 4, NS = 256 / LN;
  __shared__ float part[NS][D + 2];
  int id = blockIdx.x;
  const int head = id % a.Hk;
  id /= a.Hk;
  const int r = id % (a.max_q * a.G), b = id / (a.max_q * a.G);
  const int64_t s0 = a.q_start ? a.q_start[b] : (int64_t)b * a.max_q;
  const int64_t s1 = a.q_start ? a.q_start[b + 1] : s0 + a.max_q;
  const int64_t q0 = s0 < 0 ? 0 : s0 > a.T ? a.T : s0;
  const int n = kv4_clamp((s1 > a.T ? a.T : s1) - q0, 0, a.max_q);
  const int c = kv4_clamp(a.ctx[b], 0, (int64_t)a.width * a.P);
  if (r >= n * a.G) return;
  const Kv4Range range = kv4_range(n, c, a.G, r / (16 * mt) * 16 * mt, 16 * mt, a.window, a.nsplit, kWaves);
  if (range.splits <= 1) return;
  const int i = r / a.G;
  const int64_t orow = (q0 + i) * a.Hq + head * a.G + (r - i * a.G);
  const float* ml = a.part + a.T * a.Hq * a.nsplit * D + orow * a.nsplit * 2;
  const float* src = a.part + orow * a.nsplit * D;
  const int l = threadIdx.x % LN, k = threadIdx.x / LN;
  float ref = kNegInf;
  for (int s = 0; s < range.splits; ++s) ref = fmaxf(ref, ml[2 * s]);
  v4f o = {0.f, 0.f, 0.f, 0.f};
  float sum = 0.f;
  for (int s = k; s < range.splits; s += NS) {
    const float rs = ml[2 * s];
    if (rs == kNegInf) continue;
    const float f = exp2f(rs - ref);
    o += f * *(const v4f*)(src + (int64_t)s * D + 4 * l);
    sum = fmaf(f, ml[2 * s + 1], sum);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) part[k][4 * l + e] = o[e];
  if (l == 0) part[k][D] = sum;
  __syncthreads();
  if (threadIdx.x >= D / 8) return;
  float y[8] = {};
  sum = 0.f;
  for (int s = 0; s < NS; ++s) {
    sum += part[s][D];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] += part[s][8 * threadIdx.x + e];
  }
  const float inv = ref == kNegInf ? 0.f : 1.0f / sum;
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] *= inv;
  store8<BF ? kBF16 : kF16>(a.out, orow * D + 8 * threadIdx.x, y);
  if (a.lse && threadIdx.x == 0)
    a.lse[orow] = ref == kNegInf ? kNegInf : (ref + log2f(sum)) * 0.69314718055994530942f;
}

template <int D, int MT, bool BF>
hipError_t attn_go(const Kv4AttnArgs& a, hipStream_t s) {
  const size_t lds = (size_t)kWaves * 16 * MT * (D + 4 + 2) * 4;
  const int64_t wgs = (int64_t)a.B * a.Hk * a.tiles * a.nsplit;
  hipLaunchKernelGGL((k_kv4_attn<D, MT, BF>), dim3((uint32_t)wgs), dim3(64 * kWaves), lds, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.nsplit == 1) return e;
  const int64_t rows = (int64_t)a.B * a.max_q * a.Hq;
  hipLaunchKernelGGL((k_kv4_join<D, BF>), dim3((uint32_t)rows), dim3(256), 0, s, a, MT);
  return hipGetLastError();
}
template <int D, bool BF>
hipError_t attn_mt(const Kv4AttnArgs& a, int mt, hipStream_t s) {
  return mt == 1 ? attn_go<D, 1, BF>(a, s) : attn_go<D, 2, BF>(a, s);
}
template <bool BF>
hipError_t attn_d(const Kv4AttnArgs& a, int mt, hipStream_t s) {
  return a.D == 64 ? attn_mt<64, BF>(a, mt, s) : a.D == 128 ? attn_mt<128, BF>(a, mt, s) : attn_mt<256, BF>(a, mt, s);
}

template <int SRC>
hipError_t rope_dst(const RopeArgs& a, int dst, dim3 grid, size_t lds, hipStream_t s, int tokens, int hpw, int lanes) {
  if (dst == kF16)
    hipLaunchKernelGGL((k_qk_norm_rope<SRC, kF16>), grid, dim3(256), lds, s, a, tokens, hpw, lanes);
  else if (dst == kBF16)
    hipLaunchKernelGGL((k_qk_norm_rope<SRC, kBF16>), grid, dim3(256), lds, s, a, tokens, hpw, lanes);
  else
    hipLaunchKernelGGL((k_qk_norm_rope<SRC, kF32>), grid, dim3(256), lds, s, a, tokens, hpw, lanes);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_qk_norm_rope(const RopeArgs& a, int in_dtype, int out_dtype, hipStream_t s) {
  int lanes = 2;
  while (8 * lanes < a.D) lanes *= 2;
  const int H = a.Hq + a.Hk, slots = 256 / lanes;
  // few tokens: one pass of heads per workgroup; many: four tokens with all
  // their heads, so that a workgroup's last pass is seldom empty
  const bool few = a.T * ((H + slots - 1) / slots) <= 1024;
  const int tokens = few ? 1 : 4, hpw = few ? slots : H;
  const dim3 grid((uint32_t)((a.T + tokens - 1) / tokens), (H + hpw - 1) / hpw);
  const size_t lds = (size_t)tokens * (a.rot / 2) * 8;
  return in_dtype == kF16    ? rope_dst<kF16>(a, out_dtype, grid, lds, s, tokens, hpw, lanes)
         : in_dtype == kBF16 ? rope_dst<kBF16>(a, out_dtype, grid, lds, s, tokens, hpw, lanes)
                             : rope_dst<kF32>(a, out_dtype, grid, lds, s, tokens, hpw, lanes);
}

hipError_t launch_kv4_store(const Kv4StoreArgs& a, int dtype, hipStream_t s) {
  const int64_t per = 256 / (a.D / 8);
  const dim3 grid((uint32_t)((a.T * a.Hk * 2 + per - 1) / per));
  if (dtype == kF16)
    hipLaunchKernelGGL(k_kv4_store<kF16>, grid, dim3(256), 0, s, a);
  else if (dtype == kBF16)
    hipLaunchKernelGGL(k_kv4_store<kBF16>, grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL(k_kv4_store<kF32>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_kv4_load(const Kv4LoadArgs& a, int dtype, hipStream_t s) {
  const int64_t per = 256 / (a.D / 8);
  const dim3 grid((uint32_t)((a.T * a.Hk * 2 + per - 1) / per));
  if (dtype == kF16)
    hipLaunchKernelGGL(k_kv4_load<kF16>, grid, dim3(256), 0, s, a);
  else if (dtype == kBF16)
    hipLaunchKernelGGL(k_kv4_load<kBF16>, grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL(k_kv4_load<kF32>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

Kv4AttnPlan plan_kv4_attn(int64_t T, int Hq, int Hk, int D, int P, int width, int B, int max_q) {
  Kv4AttnPlan p;
  const int64_t G = Hq / Hk, rows = (int64_t)max_q * G;
  p.mt = rows > 16 ? 2 : 1;
  p.tiles = (int)((rows + 16 * p.mt - 1) / (16 * p.mt));
  // enough workgroups for two on each of the 256 CUs, but at least one
  // 32-token tile for each wave of a split
  const int64_t wgs = (int64_t)B * Hk * p.tiles;
  const int64_t most = ((int64_t)width * P / kKvTile + kWaves - 1) / kWaves;
  int64_t ns = (512 + wgs - 1) / wgs;
  if (ns > most) ns = most;
  if (ns < 1) ns = 1;
  p.nsplit = (int)ns;
  p.ws_bytes = ns > 1 ? (size_t)(T * Hq * ns * (D + 2) * 4) : 0;
  return p;
}

hipError_t launch_kv4_attn(Kv4AttnArgs a, const Kv4AttnPlan& p, int dtype, hipStream_t s) {
  a.tiles = p.tiles;
  a.nsplit = p.nsplit;
  return dtype == kBF16 ? attn_d<true>(a, p.mt, s) : attn_d<false>(a, p.mt, s);
}

}  // namespace tq2
