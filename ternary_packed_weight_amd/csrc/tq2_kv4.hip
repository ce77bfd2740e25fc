// gfx950 (MI355X, CDNA4) kernels of the attention half of a decode step:
// norms and rotation of the query and key heads, the 4-bit key/value cache,
// and the attention that reads it.  Layout and launch interface: tq2_kv4.h.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "tq2_elem.h"
#include "tq2_kv4.h"

namespace tq2 {
namespace {

typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef uint16_t v2us __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

using elem::Elem;
using elem::load8;
using elem::store8;

// ---- norms and rotation ----

// y = x * rsqrt(mean(x^2) + eps) * w per head, then the rotation of channel
// pairs by position * inv_freq, in fp32 with one rounding at the end.  The
// angle is the exact product, an fp64 number and its remainder, reduced by
// whole turns (at a position of 10^6 an fp32 angle is off by 0.06 rad).  A workgroup takes a
// few tokens: every angle is turned into (cos, sin) once, in LDS, and shared
// by all heads of the token.  A lane takes two runs of 8 channels that pair
// with each other (runs i and i + rot/16 of halves, neighbours of adjacent
// pairs, any two of what is not rotated), so that every element is read once;
// a power of two of lanes per head, and the next head's runs are on their way
// while one is computed.  What bounds it for many tokens is the bytes: 4096
// tokens of 34 heads of 128 in bf16 take 14.2 us, 5.0 TB/s, what a large copy
// reaches (21.2 us with partners read a second time and nothing on the way).
constexpr double kTurn = 0x1.45f306dc9c883p-3, kTurnLeft = -0x1.6b01ec5417056p-57;  // 1/(2 pi), and what it is more
template <int SRC, int DST>
__global__ __launch_bounds__(256) void k_qk_norm_rope(RopeArgs a, int tokens, int heads_per_wg, int lanes) {
  extern __shared__ float2 turn[];  // [tokens][rot/2] (cos, sin)
  const int64_t t0 = (int64_t)blockIdx.x * tokens;
  const int nt = (int)(a.T - t0 < tokens ? a.T - t0 : tokens);
  const int h0 = blockIdx.y * heads_per_wg, H = a.Hq + a.Hk;
  const int nh = H - h0 < heads_per_wg ? H - h0 : heads_per_wg;
  const int half = a.rot / 2;
  const int l = threadIdx.x % lanes;
  const bool on = 16 * l < a.D, turned = 16 * l < a.rot;
  // the lane's channels
  const bool far = turned && !a.interleaved;
  const int d0 = !on ? 0 : far ? 8 * l : 16 * l, d1 = !on ? 0 : far ? 8 * l + half : 16 * l + 8;
  const int items = nt * nh, step = 256 / lanes;
  struct Item {
    bool isq;
    int t, h;
  };
  const auto item = [&](int it) {
    const int t = it / nh, hh = h0 + it - t * nh;
    return Item{hh < a.Hq, t, hh < a.Hq ? hh : hh - a.Hq};
  };
  float x[2][8], next[2][8];
  const auto fetch = [&](int it) {
    const Item i = item(it < items ? it : items - 1);
    const void* src = i.isq ? a.q : a.k;
    const int64_t at = i.isq ? (t0 + i.t) * a.q_ts + i.h * a.q_hs : (t0 + i.t) * a.k_ts + i.h * a.k_hs;
    load8<SRC>(src, at + d0, next[0]);
    load8<SRC>(src, at + d1, next[1]);
  };
  int it = threadIdx.x / lanes;
  fetch(it);
  for (int i = threadIdx.x; i < nt * half; i += 256) {
    const int t = i / half, f = i - t * half;
    // what each step's rounding leaves is kept: at a position of 2^31 it is some fp32 roundings of a turn
    const double pos = a.positions[t0 + t], freq = a.inv_freq[f], angle = pos * freq, left = fma(pos, freq, -angle);
    const double frac = fma(left, kTurn, fma(angle, kTurnLeft, fma(angle, kTurn, -rint(angle * kTurn))));
    // what rounding the angle to fp32 leaves (2^-26 turns at most) is turned by afterwards
    const float near = (float)frac, rest = (float)(frac - near) * 6.2831853f;
    float c, s;
    sincospif(2.0f * near, &s, &c);
    turn[i] = make_float2(fmaf(-s, rest, c), fmaf(c, rest, s));
  }
  __syncthreads();
  for (; it < items; it += step) {
    const Item i = item(it);
#pragma unroll
    for (int c = 0; c < 8; ++c) x[0][c] = on ? next[0][c] : 0.f, x[1][c] = on ? next[1][c] : 0.f;
    fetch(it + step);
    const float* w = i.isq ? a.q_weight : a.k_weight;
    if (w) {
      float ss = 0.f;
#pragma unroll
      for (int c = 0; c < 8; ++c) ss = fmaf(x[0][c], x[0][c], fmaf(x[1][c], x[1][c], ss));
      for (int o = lanes / 2; o > 0; o >>= 1) ss += __shfl_xor(ss, o, 64);
      const float r = 1.0f / sqrtf(ss / (float)a.D + a.eps);
#pragma unroll
      for (int c = 0; c < 8; ++c) x[0][c] = x[0][c] * r * w[d0 + c], x[1][c] = x[1][c] * r * w[d1 + c];
    }
    if (!on) continue;
    if (turned) {
      const float2* cs = turn + i.t * half + 8 * l;  // of pairs 8l ..
      if (a.interleaved) {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float2 z = cs[c];
          float &u = x[c / 4][c % 4 * 2], &v = x[c / 4][c % 4 * 2 + 1];
          const float y = u * z.x - v * z.y;
          v = v * z.x + u * z.y;
          u = y;
        }
      } else {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float2 z = cs[c];
          const float y = x[0][c] * z.x - x[1][c] * z.y;
          x[1][c] = x[1][c] * z.x + x[0][c] * z.y;
          x[0][c] = y;
        }
      }
    }
    void* dst = i.isq ? a.q_out : a.k_out;
    const int64_t out = ((t0 + i.t) * (i.isq ? a.Hq : a.Hk) + i.h) * a.D;
    store8<DST>(dst, out + d0, x[0]);
    store8<DST>(dst, out + d1, x[1]);
  }
}

// ---- the cache: write and read back ----
//
// A workgroup takes TOK tokens of one head, keys and values, 8 channels (one
// 32-bit word of codes) per lane and D/8 lanes per row.  Groups of TOK tokens
// start where the first token's slot makes slots of a run (a prompt) multiples
// of TOK: a group that is such a run owns whole cache lines.  Both kernels are
// bound by the bytes of the heads, and by the latency of a workgroup's three
// steps (first slot, heads, codes): 16383 tokens of 8 heads of 128 in bf16 are
// stored in 26.2 us (3.3 TB/s) and read back in 19.7 us (4.3 TB/s).  With one
// token per workgroup a value tile's lines were written a few bytes at a time
// through several L2s, and full divisions cost more than the bytes: 40 and 28 us.

// Tokens of a workgroup, [t0, t0 + TOK) of the call's T; some may lie outside.
template <int TOK>
__device__ __forceinline__ int64_t group_start(const int64_t* slots, uint32_t group) {
  const int64_t first = slots[0];
  return (int64_t)group * TOK - (first < 0 ? 0 : first % TOK);
}
// The slots of the group in LDS; whether they are a run from a multiple of TOK in a page that is there.
template <int TOK>
__device__ __forceinline__ bool group_slots(const int64_t* slots, int64_t t0, int64_t T, int64_t most, int64_t (&s)[TOK]) {
  bool run = true;
  const int i = threadIdx.x;
  if (i < TOK) {
    const int64_t t = t0 + i;
    s[i] = t >= 0 && t < T ? slots[t] : -1;
    const int64_t first = t0 >= 0 && t0 < T ? slots[t0] : -1;
    run = first >= 0 && first % TOK == 0 && s[i] == first + i && s[i] < most;
  }
  return __syncthreads_and(run);
}
// Over the D/8 lanes of a row: every lane gets the result.
template <int LANES, class F>
__device__ __forceinline__ float over_row(float v, F f) {
  const auto dpp = [&](auto ctrl) {
    const int x = __builtin_bit_cast(int, v);
    v = f(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(x, x, decltype(ctrl)::value, 0xf, 0xf, false)));
  };
  dpp(std::integral_constant<int, 0xb1>());   // lane ^ 1
  dpp(std::integral_constant<int, 0x4e>());   // lane ^ 2
  dpp(std::integral_constant<int, 0x141>());  // mirrored in 8 lanes
  if constexpr (LANES >= 16) dpp(std::integral_constant<int, 0x140>());  // in 16
  if constexpr (LANES >= 32) {
    const uint32_t x = __builtin_bit_cast(uint32_t, v);
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    v = f(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
  }
  return v;
}

// a / b rounded as a division, for b of at most 12 significant bits (a
// binary16 value, 15) and r = 1/b within 1 ulp.  q = a*r is off by less than
// 3 ulp, a - q*b is exact in one fma, and the sum before its rounding is off by
// less than 3 * 2^-23 ulp; the quotient of a 24-bit by a 12-bit significand is
// no nearer than 2^-13 ulp to a border between two floats.
__device__ __forceinline__ float quotient(float a, float b, float r) {
  const float q = a * r;
  return fmaf(fmaf(-q, b, a), r, q);
}

// Per (token, head): z = f16((max+min)/2), s = f16((max-min)/15), code =
// clamp(rint((x-z)/s + 7.5), 0, 15), so that the codes are the definition's
// bit for bit (the clamp before the rounding gives the same: its ends are whole).
template <int DT, int D, int TOK>
__global__ __launch_bounds__(256) void k_kv4_store(Kv4StoreArgs a) {
  constexpr int LANES = D / 8, PER = 256 / LANES, N = 2 * TOK / PER;  // rows of a pass, passes
  static_assert(TOK % PER == 0 || PER == 2 * TOK, "a pass is of whole rows");
  __shared__ int64_t slot[TOK];
  __shared__ __align__(16) uint16_t units[TOK * D / 4];
  const uint32_t group = blockIdx.x / a.Hk;
  const int h = blockIdx.x - group * a.Hk, l = threadIdx.x % LANES;  // the heads of a token side by side in time
  const int64_t t0 = group_start<TOK>(a.slots, group);
  float x[N][8];
#pragma unroll
  for (int p = 0; p < N; ++p) {
    const int row = p * PER + threadIdx.x / LANES, i = row % TOK;
    const int64_t t = t0 + i < 0 ? 0 : t0 + i < a.T ? t0 + i : a.T - 1;
    load8<DT>(row >= TOK ? a.v : a.k, (row >= TOK ? t * a.v_ts + h * a.v_hs : t * a.k_ts + h * a.k_hs) + 8 * l, x[p]);
  }
  const bool run = group_slots<TOK>(a.slots, t0, a.T, a.pages * a.P, slot);
#pragma unroll
  for (int p = 0; p < N; ++p) {
    const int row = p * PER + threadIdx.x / LANES, i = row % TOK;
    const bool isv = row >= TOK;
    float lo = x[p][0], hi = x[p][0];
#pragma unroll
    for (int c = 1; c < 8; ++c) lo = fminf(lo, x[p][c]), hi = fmaxf(hi, x[p][c]);
    lo = over_row<LANES>(lo, [](float u, float v) { return fminf(u, v); });
    hi = over_row<LANES>(hi, [](float u, float v) { return fmaxf(u, v); });
    float range = quotient(hi - lo, 15.0f, 1.0f / 15.0f);
    asm("" : "+v"(range));  // its own rounding: the compiler would make one of the last step's and the next line's
    const _Float16 z = (_Float16)((hi + lo) * 0.5f), s = (_Float16)range;
    const float sf = (float)s, zf = (float)z, r = __builtin_amdgcn_rcpf(sf);
    // a code in a float's last bits: 1.5 * 2^23 + code, the bits above it taken off the sum of all eight
    constexpr uint32_t kMagic = 0x4b400000u;
    uint32_t w = 0u - 0x11111111u * kMagic;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float code = __builtin_amdgcn_fmed3f(quotient(x[p][c] - zf, sf, r) + 7.5f, 0.f, 15.f);
      w += __builtin_bit_cast(uint32_t, code + 12582912.0f) << (4 * c);
    }
    w = sf == 0.f ? 0 : w;
    int at;
    const int64_t block = kv4_slot_block(slot[i], a.pages, a.Hk, a.P, D, h, &at);
    if (block < 0) continue;
    uint8_t* b = a.cache + block;
    if (!isv) {
      *(uint32_t*)(b + kv4_key_at(D, at) + 4 * l) = w;
    } else if (run) {
      uint16_t* u = units + ((i / 8) * (D / 4) + 2 * l) * 8 + i % 8;
      u[0] = (uint16_t)w;
      u[8] = (uint16_t)(w >> 16);
    } else {
      *(uint16_t*)(b + kv4_value_unit_at(a.P, D, at, 2 * l)) = (uint16_t)w;
      *(uint16_t*)(b + kv4_value_unit_at(a.P, D, at, 2 * l + 1)) = (uint16_t)(w >> 16);
    }
    if (l == 0) {
      const uint32_t pair = __builtin_bit_cast(uint16_t, s) | (uint32_t)__builtin_bit_cast(uint16_t, z) << 16;
      *(uint32_t*)(b + (isv ? kv4_value_pair_at(a.P, D, at) : kv4_key_pair_at(a.P, D, at))) = pair;
    }
  }
  if (!run) return;  // all threads or none
  __syncthreads();
  int at;
  uint8_t* b = a.cache + kv4_slot_block(slot[0], a.pages, a.Hk, a.P, D, h, &at);
  uint64_t* to = (uint64_t*)(b + kv4_value_unit_at(a.P, D, at, 0));
  for (int i = threadIdx.x; i < TOK * D / 16; i += 256) to[i] = ((const uint64_t*)units)[i];
}

// value = z + s*(code - 7.5); s*(code - 7.5) is exact in fp32.
template <int DT, int D, int TOK>
__global__ __launch_bounds__(256) void k_kv4_load(Kv4LoadArgs a) {
  constexpr int LANES = D / 8, PER = 256 / LANES, N = 2 * TOK / PER;
  __shared__ int64_t slot[TOK];
  __shared__ __align__(16) uint16_t units[TOK * D / 4];
  const uint32_t group = blockIdx.x / a.Hk;
  const int h = blockIdx.x - group * a.Hk, l = threadIdx.x % LANES;  // the heads of a token side by side in time
  const int64_t t0 = group_start<TOK>(a.slots, group);
  const bool run = group_slots<TOK>(a.slots, t0, a.T, a.pages * a.P, slot) && a.v;
  if (run) {
    int at;
    const uint8_t* b = a.cache + kv4_slot_block(slot[0], a.pages, a.Hk, a.P, D, h, &at);
    const uint64_t* from = (const uint64_t*)(b + kv4_value_unit_at(a.P, D, at, 0));
    for (int i = threadIdx.x; i < TOK * D / 16; i += 256) ((uint64_t*)units)[i] = from[i];
  }
  uint32_t w[N], pair[N];
#pragma unroll
  for (int p = 0; p < N; ++p) {
    const int row = p * PER + threadIdx.x / LANES, i = row % TOK;
    const bool isv = row >= TOK;
    int at;
    const int64_t block = kv4_slot_block(slot[i], a.pages, a.Hk, a.P, D, h, &at);
    w[p] = pair[p] = 0;
    if (block < 0) continue;
    const uint8_t* b = a.cache + block;
    if (!isv) {
      w[p] = *(const uint32_t*)(b + kv4_key_at(D, at) + 4 * l);
    } else if (!run) {
      w[p] = *(const uint16_t*)(b + kv4_value_unit_at(a.P, D, at, 2 * l));
      w[p] |= (uint32_t) * (const uint16_t*)(b + kv4_value_unit_at(a.P, D, at, 2 * l + 1)) << 16;
    }
    pair[p] = *(const uint32_t*)(b + (isv ? kv4_value_pair_at(a.P, D, at) : kv4_key_pair_at(a.P, D, at)));
  }
  if (run) __syncthreads();
#pragma unroll
  for (int p = 0; p < N; ++p) {
    const int row = p * PER + threadIdx.x / LANES, i = row % TOK;
    const bool isv = row >= TOK;
    const int64_t t = t0 + i;
    void* dst = isv ? a.v : a.k;
    if (t < 0 || t >= a.T || !dst) continue;
    if (isv && run) {
      const uint16_t* u = units + ((i / 8) * (D / 4) + 2 * l) * 8 + i % 8;
      w[p] = u[0] | (uint32_t)u[8] << 16;
    }
    const v2h sz = __builtin_bit_cast(v2h, pair[p]);
    float x[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) x[c] = fmaf((float)sz[0], (float)((w[p] >> (4 * c)) & 15) - 7.5f, (float)sz[1]);
    store8<DT>(dst, (t * a.Hk + h) * D + 8 * l, x);
  }
}

// ---- attention ----

// A row's reference (see Rows) moves when a product p s may pass 2^kMost, and
// is then such that the largest so far is 2^kSet, and p at most 2^kSetP.
constexpr float kMost = 12.0f, kSet = 4.0f, kSetP = 30.0f;
constexpr float kNone = -3.4028234663852886e38f;  // the reference of a row that has seen nothing
constexpr float kNegInf = -INFINITY;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

// Over the four lanes (16 and 32 apart) of a row: every lane gets the result.
__device__ __forceinline__ float max_g(float v) {
  const uint32_t x = __builtin_bit_cast(uint32_t, v);
  auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  v = fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
  const uint32_t y = __builtin_bit_cast(uint32_t, v);
  r = __builtin_amdgcn_permlane16_swap(y, y, false, false);
  return fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
}
__device__ __forceinline__ float sum_g(float v) {
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}
// log(sum exp) of a row's sum in units of 2^ref: -inf where it saw nothing (a
// reference of -inf and a sum of zero), NaN where all that it saw was.
__device__ __forceinline__ float log_sum(float ref, float sum) {
  return ref == kNegInf ? kNegInf + sum : (ref + log2f(sum)) * kLn2;
}
__device__ __forceinline__ float half_lo(uint32_t w) { return (float)__builtin_bit_cast(v2h, w)[0]; }
__device__ __forceinline__ float half_hi(uint32_t w) { return (float)__builtin_bit_cast(v2h, w)[1]; }

// A power of two above the value scales (low halves of pairs, without their
// signs) of a lane's tokens, by its exponent; without any, one that lets p grow to 2^38.
template <int N>
__device__ __forceinline__ float above_scales(const uint32_t (&pair)[N][8]) {
  v2us top = {0, 0};
#pragma unroll
  for (int i = 0; i < 8 * N; i += 2) {
    const uint32_t two = __builtin_amdgcn_perm(pair[i / 8][i % 8 + 1], pair[i / 8][i % 8], 0x05040100) & 0x7fff7fffu;
    top = __builtin_elementwise_max(top, __builtin_bit_cast(v2us, two));
  }
  const int t = top[0] > top[1] ? top[0] : top[1];
  return t ? (float)((t >> 10) - 14) : kMost - kSetP - 8.0f;
}

// Codes enter the matrix cores as masked binary16 subnormals, code j of each
// 16-bit half as c * 2^-SUB.  The products do not normalize them: what a
// subnormal has of leading zeros is cut off the other end, towards zero.  Codes
// in the lowest bits (2^-24) left an output of 131000 tokens off by 2^-9, in
// four bits more (2^-20, a shift for three of four) by 2^-13, in the highest
// ones (2^-18, a shift each) by 2^-15.
template <int SUB>
__device__ __forceinline__ uint32_t nib(uint32_t w, int j) {
  constexpr int at = 24 - SUB;  // bit of the code
  static_assert(at >= 0 && at <= 6, "four bits of the mantissa");
  const int up = at - 4 * j;
  return (up > 0 ? w << up : w >> -up) & (0x000f000fu << at);
}
template <int SUB>
__device__ __forceinline__ v4u key_frag(uint32_t w) {
  return v4u{nib<SUB>(w, 0), nib<SUB>(w, 1), nib<SUB>(w, 2), nib<SUB>(w, 3)};
}
template <int SUB>
__device__ __forceinline__ v4u value_frag(const uint32_t* w, int j) {
  return v4u{nib<SUB>(w[0], j), nib<SUB>(w[1], j), nib<SUB>(w[2], j), nib<SUB>(w[3], j)};
}
constexpr int kSubFew = 18, kSubMany = 20;

// Page tables are read by scalar loads.
typedef const int32_t __attribute__((address_space(4))) * PageTable;

// The tiles first, first + step, .. below last of one key head's cache, as a
// wave reads them: the codes and pairs of one tile, its keys and its values
// each replaced by the next tile's as soon as they are used.
template <int D>
struct Tiles {
  static constexpr int NW = D / 32;  // 32-bit code words of a lane and token (keys)
  static constexpr int NJ = D / 16;  // and of a lane (values)
  uint32_t kc[2][NW], kp[8], vc[NJ], vp[1][8];
  PageTable table;
  const uint8_t* cache;  // the key head's part of page 0
  const uint8_t* base;   // of the page of the tile whose keys are held
  bool there;            // whether there is such a page
  int tile, last, step, pshift;  // tiles of a page, as a shift
  uint32_t pages, page_units, kat, vat, kpat, vpat;
  int32_t ahead;  // page of the tile behind it

  __device__ __forceinline__ void open(const Kv4AttnArgs& a, const int32_t* table_, int head, int first, int last_,
                                       int step_, int lane) {
    table = (PageTable)table_, tile = first, last = last_, step = step_;
    pshift = 31 - __builtin_clz(a.P) - 5;
    cache = a.cache + head * kv4_block_bytes(a.P, D);
    pages = kv4_page_limit(a.pages);
    page_units = (uint32_t)(a.Hk * kv4_block_bytes(a.P, D) / 16);
    const int col = lane & 15, g = lane >> 4;
    kat = ((col >> 2) * 8 + (col & 3)) * (D / 2) + g * (D / 8), vat = a.P * (D / 2) + lane * (D / 4);
    kpat = a.P * D + g * 32, vpat = kpat + a.P * 4;
    // a wave without a tile looks at the first entry, and reads nothing for it
    ahead = table[(tile < last ? tile : 0) >> pshift];
  }
  __device__ __forceinline__ int place() const { return tile & ((1 << pshift) - 1); }
  __device__ __forceinline__ void keys() {  // of `tile`; its page is `ahead`
    const uint32_t page = ahead;
    there = kv4_page_there(ahead, pages);
    base = cache + (uint64_t)(there ? page : 0) * page_units * 16;
    const uint8_t* k = base + (uint32_t)place() * (16 * D);
#pragma unroll
    for (int u = 0; u < 2; ++u) __builtin_memcpy(kc[u], __builtin_assume_aligned(k + kat + u * 2 * D, 8), D / 8);
    __builtin_memcpy(kp, __builtin_assume_aligned(base + (uint32_t)place() * 128 + kpat, 16), 32);
    ahead = table[(tile + step < last ? tile + step : tile) >> pshift];
  }
  __device__ __forceinline__ void vals() {
    __builtin_memcpy(vc, __builtin_assume_aligned(base + (uint32_t)place() * (16 * D) + vat, 16), D / 4);
    __builtin_memcpy(vp[0], __builtin_assume_aligned(base + (uint32_t)place() * 128 + vpat, 16), 32);
  }
};

// TPS tiles unpacked once for the four waves of a workgroup, in LDS, for two
// steps in turn.  Of a tile: operand fragments of the keys [2][NW], then of the
// values [NJ], 64 lanes of 16 bytes each; behind the tiles their key and value
// pairs.  A wave unpacks a quarter of every tile, the keys of one u or half of
// the value fragments, and copies 32 pairs.  Codes are requested two steps
// ahead and pages three, so that a step waits for neither.
template <int D, int TPS>
struct Staged {
  static constexpr int NW = D / 32, NJ = D / 16;
  static constexpr int kFrags = 4 * NW * 64 * TPS;  // 16-byte units
  static constexpr int kStep = kFrags + 16 * TPS;   // and those of the pairs
  v4u* buf;
  uint32_t codes[TPS][NW < 4 ? 4 : NW], pair;  // of the step to unpack next
  PageTable table;
  const uint8_t *cache, *next[TPS];  // the key head's part of page 0; of the pages of the step behind the one at hand
  uint32_t there, there_next;        // a bit for each of a step's tiles whose page there is
  uint32_t pages, page_units, at, pat;
  int tile, last, pshift, wave, odd;
  int32_t ahead[TPS];  // pages of the step behind `next`

  // Behind the last tile: the last one's again.
  __device__ __forceinline__ int held(int t) const { return t < last ? t : last - 1; }
  __device__ __forceinline__ void find(const int32_t (&page)[TPS]) {
    there_next = 0;
#pragma unroll
    for (int i = 0; i < TPS; ++i) {
      const uint32_t p = page[i];
      const bool is = kv4_page_there(page[i], pages);
      there_next |= (uint32_t)is << i;
      next[i] = cache + (uint64_t)(is ? p : 0) * page_units * 16;
    }
  }
  __device__ __forceinline__ void look(int t) {
#pragma unroll
    for (int i = 0; i < TPS; ++i) ahead[i] = table[held(t + i) >> pshift];
  }
  __device__ __forceinline__ void load(int t) {  // of tiles t .. in the pages `next`
    const int mask = (1 << pshift) - 1;
#pragma unroll
    for (int i = 0; i < TPS; ++i) {
      const uint8_t* p = next[i] + (uint32_t)(held(t + i) & mask) * (16 * D);
      if (D == 64 && wave >= 2)
        __builtin_memcpy(codes[i], __builtin_assume_aligned(p + at, 16), 16);
      else
        __builtin_memcpy(codes[i], __builtin_assume_aligned(p + at, 8), 4 * NW);
    }
    const int i = TPS == 2 ? wave >> 1 : 0;
    const uint8_t* p = TPS == 2 && i ? next[TPS - 1] : next[0];
    pair = *(const uint32_t*)(p + (uint32_t)(held(t + i) & mask) * 128 + pat);
  }
  __device__ __forceinline__ void unpack() {
    v4u* b = buf + odd * kStep;
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < TPS; ++i) {
      v4u* o = b + (i * 4 + wave) * NW * 64 + lane;
      if (wave < 2) {
#pragma unroll
        for (int w = 0; w < NW; ++w) o[w * 64] = key_frag<kSubMany>(codes[i][w]);
      } else if (D == 64) {  // nibbles 0 and 1, or 2 and 3
#pragma unroll
        for (int j = 0; j < NW; ++j)
          o[j * 64] = wave == 3 ? value_frag<kSubMany>(codes[i], 2 + j) : value_frag<kSubMany>(codes[i], j);
      } else {
#pragma unroll
        for (int f = 0; f < NW; ++f) o[f * 64] = value_frag<kSubMany>(codes[i] + f / 4 * 4, f % 4);
      }
    }
    if (wave < 2 * TPS && lane < 32) ((uint32_t*)(b + kFrags))[wave * 32 + lane] = pair;
  }
  // Pairs of tokens 8g .. of plane 2*tile (keys) or 2*tile + 1 (values) of a step.
  __device__ __forceinline__ void pairs(const v4u* f, int plane, int g, uint32_t (&to)[8]) const {
    const v4u* p = f + kFrags + plane * 8 + g * 2;
    const v4u lo = p[0], hi = p[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) to[i] = lo[i], to[4 + i] = hi[i];
  }
  __device__ __forceinline__ void open(const Kv4AttnArgs& a, v4u* buf_, const int32_t* table_, int head, int first,
                                       int last_, int lane, int wave_) {
    buf = buf_, table = (PageTable)table_, tile = first, last = last_, wave = wave_, odd = 0;
    pshift = 31 - __builtin_clz(a.P) - 5;
    cache = a.cache + head * kv4_block_bytes(a.P, D);
    pages = kv4_page_limit(a.pages);
    page_units = (uint32_t)(a.Hk * kv4_block_bytes(a.P, D) / 16);
    const int col = lane & 15, g = lane >> 4;
    // a lane's place in a tile's codes and pairs, from the tile's place in the page's key codes
    at = wave < 2 ? ((col >> 2) * 8 + (col & 3) + 4 * wave) * (D / 2) + g * (D / 8)
                  : a.P * (D / 2) + lane * (D / 4) + (D == 64 ? 0 : (wave - 2) * (D / 8));
    pat = a.P * D + (wave & 1) * a.P * 4 + (lane & 31) * 4;
    look(tile);
    find(ahead);
    there = there_next;
    load(tile);
    look(tile + TPS);
    unpack();
    find(ahead);
    load(tile + TPS);
    look(tile + 2 * TPS);
  }
  // The fragments of the step at hand; the next step's go to LDS, the codes of
  // the one behind it are requested, and the next becomes the step at hand.
  __device__ __forceinline__ const v4u* stage() {
    const v4u* f = buf + odd * kStep;
    odd ^= 1;
    tile += TPS;
    unpack();
    there = there_next;
    find(ahead);
    load(tile + TPS);
    look(tile + 2 * TPS);
    return f;
  }
};

// 16*MT rows (new token x query head of one key head) in a wave, and what
// they have seen so far.
//
// Per tile of 32 tokens the wave computes the transposed scores K Q^T
// (v_mfma_f32_16x16x32_f16), so that a lane holds eight tokens of one row,
// which is already the operand layout of V^T P^T: the probabilities never
// cross lanes.  Codes go in as they are; a token's scale and middle are applied to its score and its probability:
//   score = s_k (q.c - 7.5 sum q) + z_k sum q,  out = sum P s_v c - 7.5 sum P s_v + sum P z_v.
// Scores stay in the units of the scaled query (fa turns them into powers of
// two inside the exponential's argument).  Softmax statistics and sums are
// fp32.  P s_v goes to the matrix cores in binary16, so a row's reference is
// the largest P s_v it has seen, not the largest P: held between 2^4 and 2^12,
// it leaves every other product a least step of 2^-28 of itself (by the largest
// s_v alone, one token of no weight but a large scale took the bits of all the
// others).  It moves seldom: a tile's largest score and scale bound its
// products, and only where they pass 2^12 are the products looked at.  The
// -7.5 term sums the rounded values, so rounding acts on the centred codes.
// FINE adds the rounding's remainder in a second product, which leaves an error
// of 2^-22: many thousand tokens can average out to an output far smaller than
// its terms, where one rounding to binary16 would show.
template <int D, int MT, bool BF, bool FINE>
struct Rows {
  static constexpr int NW = D / 32;  // 32-bit code words of a lane and token (keys)
  static constexpr int NJ = D / 16;  // channels of a lane (values)
  static constexpr int SUB = FINE ? kSubFew : kSubMany;
  typedef typename Elem<BF ? kBF16 : kF16>::T T;

  typedef T v8 __attribute__((ext_vector_type(8)));

  v8 raw[MT][NW];
  int place[MT];  // the row's new token, or -1
  v8h qf[MT][NW];
  float fa[MT], qs[MT], cinit[MT];
  int lim[MT], low[MT], limmin, lowmax;
  v4f acc[MT][NJ], racc[MT];
  float ref[MT], lsum[MT], zsum[MT];  // the reference as a power of two

  // The queries of rows row0 + col + 16 m of `rows`, as they are.
  __device__ __forceinline__ void fetch(const Kv4AttnArgs& a, const Kv4Seq& s, int head, int row0, int rows, int col,
                                        int g) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int r = row0 + m * 16 + col;
      const int i = r < rows ? r / a.G : 0, h = r < rows ? r - i * a.G : 0;
      const T* p = (const T*)a.q + (s.q0 + i) * a.q_ts + (head * a.G + h) * a.q_hs + g * (D / 4);
#pragma unroll
      for (int w = 0; w < NW; ++w) raw[m][w] = *(const v8*)(p + 8 * w);
      place[m] = r < rows ? i : -1;
    }
  }
  __device__ __forceinline__ void load(const Kv4AttnArgs& a, const Kv4Seq& s) {
    limmin = s.c;
    lowmax = 0;
    const float sign = a.scale < 0.f ? -1.f : 1.f;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const bool valid = place[m] >= 0;
      const int pos = s.c - s.n + place[m];
      lim[m] = valid ? pos + 1 : s.c;
      low[m] = valid && a.window > 0 && pos >= a.window ? pos + 1 - a.window : 0;
      limmin = lim[m] < limmin ? lim[m] : limmin;
      lowmax = low[m] > lowmax ? low[m] : lowmax;
      // D/4 channels of the row: scaled by a power of two into binary16's middle
      float x[D / 4];
      float big = 0.f, sum = 0.f;
#pragma unroll
      for (int k = 0; k < D / 4; ++k) {
        x[k] = valid ? sign * (float)raw[m][k / 8][k % 8] : 0.f;
        big = fmaxf(big, fabsf(x[k]));
        sum += x[k];
      }
      big = max_g(big);
      sum = sum_g(sum);
      int ex = 0;
      if (big > 0.f && big < INFINITY) {
        ex = 9 - __builtin_amdgcn_frexp_expf(big);
        ex = ex > 100 ? 100 : ex < -100 ? -100 : ex;
      }
      float up = ldexpf(1.0f, ex), f = ldexpf(fabsf(a.scale) * kLog2e, SUB - ex);
      if (f == 0.f) up = sum = 0.f, f = 1.0f;  // every score is zero
      float used = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int nibble = (e & 1 ? 4 : 0) + (e >> 1);  // slots 0 4 1 5 2 6 3 7 of the word
          const _Float16 y = (_Float16)(x[w * 8 + nibble] * up);
          qf[m][w][e] = y;
          used += (float)y;
        }
      }
      used = sum_g(used);
      cinit[m] = -7.5f * ldexpf(used, -SUB);
      fa[m] = f;
      qs[m] = ldexpf(sum * up, -SUB);
      ref[m] = kNone;
      lsum[m] = zsum[m] = 0.f;
      racc[m] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[m][j] = v4f{0.f, 0.f, 0.f, 0.f};
    }
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) {
      const int u = __shfl_xor(limmin, o, 64), v = __shfl_xor(lowmax, o, 64);
      limmin = u < limmin ? u : limmin;
      lowmax = v > lowmax ? v : lowmax;
    }
    limmin = __builtin_amdgcn_readfirstlane(limmin);
    lowmax = __builtin_amdgcn_readfirstlane(lowmax);
  }

  // Of one tile: operand fragments frag(u, w) of the tokens (col/4)*8 + col%4
  // + 4u; kp: pairs of tokens 8g ..
  template <class F>
  __device__ __forceinline__ void scores(const F& frag, const uint32_t (&kp)[8], float (&x)[MT][8]) {
    v4f d[MT][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int m = 0; m < MT; ++m) d[m][u] = v4f{cinit[m], cinit[m], cinit[m], cinit[m]};
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const v8h f = __builtin_bit_cast(v8h, frag(u, w));
#pragma unroll
        for (int m = 0; m < MT; ++m)
          d[m][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f, qf[m][w], d[m][u], 0, 0, 0);
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 8; ++i) x[m][i] = fmaf(half_lo(kp[i]), d[m][i / 4][i % 4], fmaf(half_hi(kp[i]), qs[m], 0.f));
  }

  // Of TPS tiles together: x: scores of tokens j0 + 32 t .. + 7; frag(t, h, j):
  // fragments of the values; vp: their pairs.  c: cached tokens that are there.
  template <int TPS, class F>
  __device__ __forceinline__ void values(float (&x)[TPS][MT][8], const F& frag, const uint32_t (&vp)[TPS][8], int j0,
                                         const int (&c)[TPS], bool partial) {
    v8h hi[TPS][MT], lo[TPS][MT];
    float above = partial ? 0.f : above_scales(vp);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      uint32_t vq[TPS][8];
#pragma unroll
      for (int t = 0; t < TPS; ++t)
#pragma unroll
        for (int i = 0; i < 8; ++i) vq[t][i] = vp[t][i];
      if (partial) {  // tokens that are not there, or not for this row: their pairs may hold anything
#pragma unroll
        for (int t = 0; t < TPS; ++t) {
          const int end = c[t] < lim[m] ? c[t] : lim[m];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int j = j0 + 32 * t + i;
            if (j >= end || j < low[m]) {
              x[t][m][i] = kNegInf;
              vq[t][i] = 0;
            }
          }
        }
        above = above_scales(vq);
      }
      float mx = x[0][m][0];
#pragma unroll
      for (int t = 0; t < TPS; ++t)
#pragma unroll
        for (int i = 0; i < 8; ++i) mx = fmaxf(mx, x[t][m][i]);
      const float bound = fmaf(mx, fa[m], above - kMost);
      if (__builtin_amdgcn_ballot_w64(bound > ref[m])) {
        float v = kNegInf;  // log2 of the largest product
#pragma unroll
        for (int t = 0; t < TPS; ++t)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            // as it was read (a masked token's x is -inf): the logarithm is
            // for here alone, shared by all m it would take the registers
            uint32_t pair = vp[t][i];
            asm volatile("" : "+v"(pair));
            v = fmaxf(v, fmaf(x[t][m][i], fa[m], fminf(__builtin_amdgcn_logf(fabsf(half_lo(pair))), 16.0f)));
          }
        // of the whole row; the others of the wave stay as they are
        v = fmaxf(max_g(v) - kSet, fmaf(max_g(mx), fa[m], -kSetP));
        const float to = max_g(bound) > ref[m] ? fmaxf(v, ref[m]) : ref[m];
        const float f = __builtin_amdgcn_exp2f(ref[m] - to);
        ref[m] = to;
        lsum[m] *= f;
        zsum[m] *= f;
        racc[m] *= f;
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[m][j] *= f;
      }
#pragma unroll
      for (int t = 0; t < TPS; ++t) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float p = __builtin_amdgcn_exp2f(fmaf(x[t][m][i], fa[m], -ref[m]));
          lsum[m] += p;
          const float s = half_lo(vq[t][i]);
          zsum[m] = fmaf(p, half_hi(vq[t][i]), zsum[m]);
          hi[t][m][i] = (_Float16)fmaf(p, s, 0.f);
          if constexpr (FINE) lo[t][m][i] = (_Float16)fmaf(p, s, -(float)hi[t][m][i]);
        }
        const v8h one = {1, 1, 1, 1, 1, 1, 1, 1};
        racc[m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(one, hi[t][m], racc[m], 0, 0, 0);
        if constexpr (FINE) racc[m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(one, lo[t][m], racc[m], 0, 0, 0);
      }
    }
#pragma unroll
    for (int t = 0; t < TPS; ++t)
#pragma unroll
      for (int h = 0; h < NJ / 4; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const v8h f = __builtin_bit_cast(v8h, frag(t, h, j));
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            v4f& o = acc[m][4 * h + j];
            o = __builtin_amdgcn_mfma_f32_16x16x32_f16(f, hi[t][m], o, 0, 0, 0);
            if constexpr (FINE) o = __builtin_amdgcn_mfma_f32_16x16x32_f16(f, lo[t][m], o, 0, 0, 0);
          }
        }
  }

  // Channels (g*4 + r)*NJ + 4h .. + 3 of the row's sum, and its weight.
  __device__ __forceinline__ v4f sums(int m, int r, int h, float shift) const {
    v4f y;
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = fmaf(acc[m][4 * h + j][r], (float)(1 << SUB), shift);
    return y;
  }
  __device__ __forceinline__ float shift(int m) const { return sum_g(zsum[m]) - 7.5f * racc[m][0]; }

  // All tiles of t, whose first is on its way.
  __device__ __forceinline__ void run(Tiles<D>& t, int c, int g) {
    if (t.tile >= t.last) return;
    for (bool more = true; more;) {
      float x[1][MT][8];
      scores([&](int u, int w) { return key_frag<SUB>(t.kc[u][w]); }, t.kp, x[0]);
      const bool there = t.there;
      const int j = t.tile * 32;
      // the last tile loads itself again: a load on a condition would be
      // copied, and waited for, where the paths meet
      more = t.tile + t.step < t.last;
      t.tile = more ? t.tile + t.step : t.tile;
      t.keys();
      const bool partial = !there || j > limmin - 32 || j < lowmax;
      const int seen[1] = {there ? c : 0};
      values<1>(x, [&](int, int h, int i) { return value_frag<SUB>(t.vc + 4 * h, i); }, t.vp, j + g * 8, seen, partial);
      t.vals();
    }
  }
  // The same where the waves of a workgroup unpack a part of the tiles each, TPS tiles a step.
  template <int TPS>
  __device__ __forceinline__ void run(Staged<D, TPS>& t, int c, int g) {
    for (bool more = true; more;) {
      __syncthreads();
      const int j = t.tile * 32;
      int seen[TPS];
#pragma unroll
      for (int i = 0; i < TPS; ++i) seen[i] = t.there >> i & 1 ? c : 0;
      // (a step's end may pass 2^31, where the last tile stands twice)
      const bool partial = t.there != (1u << TPS) - 1 || j > limmin - 32 * TPS || j < lowmax;
      const v4u* f = t.stage();
      more = t.tile < t.last;
      float x[TPS][MT][8];
#pragma unroll
      for (int i = 0; i < TPS; ++i) {
        uint32_t kp[8];
        t.pairs(f, 2 * i, g, kp);
        scores([&](int u, int w) { return f[(i * 4 * NW + u * NW + w) * 64 + (threadIdx.x & 63)]; }, kp, x[i]);
      }
      uint32_t vp[TPS][8];
#pragma unroll
      for (int i = 0; i < TPS; ++i) t.pairs(f, 2 * i + 1, g, vp[i]);
      values<TPS>(x, [&](int i, int h, int n) { return f[(i * 4 * NW + 2 * NW + 4 * h + n) * 64 + (threadIdx.x & 63)]; },
                  vp, j + g * 8, seen, partial);
    }
  }
};

__device__ __forceinline__ Kv4Seq sequence(const Kv4AttnArgs& a, int b) {
  const int64_t s0 = a.q_start ? a.q_start[b] : (int64_t)b * a.max_q;
  const int64_t s1 = a.q_start ? a.q_start[b + 1] : s0 + a.max_q;
  return kv4_seq(s0, s1, a.ctx[b], a.T, a.max_q, (int64_t)a.width * a.P);
}
template <bool BF>
__device__ __forceinline__ void store4(void* p, int64_t at, v4f y) {
  typedef typename Elem<BF ? kBF16 : kF16>::T T;
  typedef T v4 __attribute__((ext_vector_type(4)));
  v4 t;
#pragma unroll
  for (int j = 0; j < 4; ++j) t[j] = (T)y[j];
  *(v4*)((T*)p + at) = t;
}
__device__ __forceinline__ float* part_stats(const Kv4AttnArgs& a, int D) {
  return a.part + (int64_t)a.slots * a.rows * D;
}
__device__ __forceinline__ Kv4Group* part_groups(const Kv4AttnArgs& a, int D) {
  return (Kv4Group*)(a.part + (int64_t)a.slots * a.rows * (D + 2));
}

__device__ __forceinline__ Kv4Work* work_list(const Kv4AttnArgs& a, int D) {
  return (Kv4Work*)(part_groups(a, D) + a.groups);
}
__device__ __forceinline__ uint32_t* work_count(const Kv4AttnArgs& a, int D) {
  return (uint32_t*)(part_groups(a, D) + a.groups - 1) + 7;  // the last group's spare word
}

// Sum of the lanes up to and with this one.
__device__ __forceinline__ uint32_t scan(uint32_t v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);   // row_shr 1, 2, 4, 8: in rows of 16 lanes
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // a row's last lane to the next row
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // lane 31 to the upper half
  return v;
}

__device__ __forceinline__ uint32_t lane_of(uint32_t v, int l) { return __builtin_amdgcn_readlane(v, l); }

// What a workgroup does: part `part` of `parts` of an (entry, head), its slot,
// and its group where the parts are joined.  Entries are row tiles of R rows,
// the first ones of all sequences first.
template <int R>
__device__ __forceinline__ int entry_tiles(const Kv4AttnArgs& a, int e, Kv4Seq* s, int* row0, int* first) {
  const int rt = e / a.B;
  *s = sequence(a, e - rt * a.B);
  *row0 = rt * R;
  return kv4_tiles(*s, a.G, *row0, R, a.window, first);
}
// The work and what it is of: its sequence, first row, first tile and tiles (0: nothing to do).
struct Kv4Found {
  Kv4Work w;
  Kv4Seq s;
  int row0, first, tiles;
};
template <int R>
__device__ __forceinline__ Kv4Found found_entry(const Kv4AttnArgs& a, const Kv4Work& w) {
  Kv4Found f;
  f.w = w;
  f.tiles = __builtin_amdgcn_readfirstlane(entry_tiles<R>(a, w.e, &f.s, &f.row0, &f.first));
  f.first = __builtin_amdgcn_readfirstlane(f.first);
  f.s.q0 = __builtin_amdgcn_readfirstlane((int)f.s.q0);
  f.s.n = __builtin_amdgcn_readfirstlane(f.s.n);
  f.s.c = __builtin_amdgcn_readfirstlane(f.s.c);
  return f;
}
// One long sequence among short ones would leave most CUs idle, so every
// (entry, head) gets workgroups by its length: each wave sums the lengths by
// itself, without a barrier, an entry or two a lane (more are in a list).
// The last entries come first.
template <int R>
__device__ __forceinline__ Kv4Found find_work(const Kv4AttnArgs& a, int D, int lane) {
  const int entries = a.B * a.tiles;
  if (!a.budget) {
    const int id = gridDim.x - 1 - blockIdx.x, e = id / a.Hk;
    return found_entry<R>(a, {e, id - e * a.Hk, 1, 0, 0, 0, 0, 0});
  }
  Kv4Found f;
  f.tiles = 0;
  const auto units = [&](int i) { return kv4_units(entry_tiles<R>(a, i, &f.s, &f.row0, &f.first), a.grain); };
  int per = (entries + 63) / 64, lo = 0, hi = entries;
  const bool one = per == 1;
  const uint32_t own = one && lane < entries ? units(lane) : 0;
  uint32_t all = own;
  for (int i = lane * per; !one && i < lane * per + per && i < entries; ++i) all += units(i);
  uint32_t share = kv4_share(lane_of(scan(all), 63), a.Hk, a.budget, a.least);
  // remainders make more workgroups than that: a share that lets all of them
  // be resident at once (64 unequal sequences: 43.6 us, with a few left over 47.5)
  for (int i = 0; i < 8; ++i) {
    uint32_t wgs = one ? kv4_take(own, a.Hk, share).wgs : 0;
    for (int k = lane * per; !one && k < lane * per + per && k < entries; ++k) wgs += kv4_take(units(k), a.Hk, share).wgs;
    if (lane_of(scan(wgs), 63) <= (uint32_t)a.budget) break;
    share += (share + 7) / 8;
  }
  uint32_t w = blockIdx.x, slot = 0, group = 0;  // counted from the entry's first
  for (bool outer = true;; outer = false) {
    Kv4Take t = {0, 0, 0};
    const int i0 = lo + lane * per;
    if (one) t = kv4_take(own, a.Hk, share);
    for (int i = i0; !one && i < i0 + per && i < hi; ++i) {
      const Kv4Take n = kv4_take(units(i), a.Hk, share);
      t.wgs += n.wgs, t.slots += n.slots, t.splits += n.splits;
    }
    const uint32_t wgs = scan(t.wgs), slots = scan(t.slots), splits = scan(t.splits);
    if (outer) {
      if (blockIdx.x == 0 && threadIdx.x == 0) part_groups(a, D)->groups = lane_of(splits, 63);
      const uint32_t total = lane_of(wgs, 63);
      if (w >= total) return f;  // more workgroups than needed
      w = total - 1 - w;
    }
    // a lane, whatever the lengths do meanwhile
    const int l = __builtin_ctzll(__builtin_amdgcn_ballot_w64(wgs > w) | (uint64_t)1 << 63);
    w -= lane_of(wgs - t.wgs, l);
    slot += lane_of(slots - t.slots, l);
    group += lane_of(splits - t.splits, l);
    lo += l * per;
    hi = lo + per < hi ? lo + per : hi;
    if (per == 1) {
      const int parts = lane_of(t.wgs, l) / a.Hk, head = w / parts;
      const Kv4Work k = {lo, head, parts, (int)w - head * parts, (int)(slot + w), (int)group + head, 0, 0};
      if (!one) return found_entry<R>(a, k);
      f.w = k;
      f.s.q0 = lane_of((int)f.s.q0, l), f.s.n = lane_of(f.s.n, l), f.s.c = lane_of(f.s.c, l);
      f.row0 = lane_of(f.row0, l), f.first = lane_of(f.first, l);
      const Kv4Range r = kv4_range(f.s.n, f.s.c, a.G, f.row0, R, a.window, 1, 1);
      f.tiles = r.last > r.first ? r.last - r.first : 1;
      return f;
    }
    per = (hi - lo + 63) / 64;
  }
}

// The same from a list, where the lengths are too many to sum in every wave.
template <int R>
__device__ __forceinline__ Kv4Found listed_work(const Kv4AttnArgs& a, int D) {
  if (blockIdx.x < *work_count(a, D)) return found_entry<R>(a, work_list(a, D)[blockIdx.x]);
  Kv4Found f;
  f.tiles = 0;
  return f;
}

// The list, written by one workgroup in 7 us (a wave that sums 564 lengths
// takes 14, in every round of workgroups); the longest parts first.
constexpr int kDeal = 1024;
template <int R>
__global__ __launch_bounds__(kDeal) void k_kv4_deal(Kv4AttnArgs a, int D) {
  Kv4Work* list = work_list(a, D);
  __shared__ uint32_t sums[3][kDeal / 64], place[8];
  const int entries = a.B * a.tiles, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int per = (entries + kDeal - 1) / kDeal, e0 = threadIdx.x * per, e1 = e0 + per < entries ? e0 + per : entries;
  const auto units = [&](int e) {
    Kv4Seq q;
    int row0, f;
    return kv4_units(entry_tiles<R>(a, e, &q, &row0, &f), a.grain);
  };
  // the sum before this thread and in all
  const auto over = [&](uint32_t v, int which, uint32_t* all) {
    const uint32_t in = scan(v);
    if (lane == 63) sums[which][wave] = in;
    __syncthreads();
    uint32_t before = 0;
    *all = 0;
    for (int w = 0; w < kDeal / 64; ++w) {
      before += w < wave ? sums[which][w] : 0;
      *all += sums[which][w];
    }
    return before + in - v;
  };
  uint32_t mine = 0, all;
  for (int e = e0; e < e1; ++e) mine += units(e);
  over(mine, 0, &all);
  const uint32_t share = kv4_share(all, a.Hk, a.budget, a.least);
  // the longest parts first: a part's class is by eighths of a share
  const auto kind = [&](uint32_t u, uint32_t parts) {
    const uint32_t k = (uint64_t)((u + parts - 1) / parts) * 8 / share;
    return k < 7 ? 7 - k : 0;
  };
  if (threadIdx.x < 8) place[threadIdx.x] = 0;
  __syncthreads();
  Kv4Take t = {0, 0, 0};
  for (int e = e0; e < e1; ++e) {
    const uint32_t u = units(e);
    const Kv4Take n = kv4_take(u, a.Hk, share);
    t.wgs += n.wgs, t.slots += n.slots, t.splits += n.splits;
    if (n.wgs) atomicAdd(&place[kind(u, n.wgs / a.Hk)], n.wgs);
  }
  uint32_t total, slots, splits;
  over(t.wgs, 0, &total);
  uint32_t slot = over(t.slots, 1, &slots), group = over(t.splits, 2, &splits);
  if (threadIdx.x == 0) {
    uint32_t sum = 0;
    for (int k = 0; k < 8; ++k) {
      const uint32_t n = place[k];
      place[k] = sum;
      sum += n;
    }
    *work_count(a, D) = total, part_groups(a, D)->groups = splits;
  }
  __syncthreads();
  for (int e = e0; e < e1; ++e) {
    const uint32_t u = units(e);
    const Kv4Take n = kv4_take(u, a.Hk, share);
    if (!n.wgs) continue;
    const int parts = n.wgs / a.Hk;
    // in a class the order is as it comes: it decides when a workgroup runs, not what it does
    const uint32_t at = atomicAdd(&place[kind(u, parts)], n.wgs);
    for (uint32_t i = 0; i < n.wgs; ++i) {
      const int head = i / parts;
      list[at + i] = Kv4Work{e, head, parts, (int)i - head * parts, (int)(slot + i), (int)group + head, 0, 0};
    }
    slot += n.slots, group += n.splits;
  }
}

// Written by the workgroup of the first part.
__device__ __forceinline__ void set_group(const Kv4AttnArgs& a, int D, const Kv4Work& w, const Kv4Seq& s, int row0) {
  Kv4Group* p = part_groups(a, D) + w.group;
  p->q0 = (int32_t)s.q0, p->row0 = row0, p->rows = s.n * a.G, p->head = w.head, p->slot = w.slot, p->count = w.parts;
}

// Few rows a key head (a decode step): out = softmax(scale q K^T) V over the
// 4-bit cache; see tq2.h.  The waves of a workgroup share 16*MT rows and take
// every fourth tile each; their parts meet in LDS.  What bounds it is the cache
// read once: 64 unequal sequences of up to 32768 tokens (2 key heads of 128)
// take 36 us, 4.3 TB/s, and a join of 5; one of 131000 takes 16 us, 8 of them a
// workgroup's start and end.  Four waves: eight were 63 us and 20, two 57 and
// 24, as a workgroup's last tiles leave waves idle, or its parts are too many.
// A second tile in flight for each wave gained nothing (46 us): what it waits
// for then is its own instructions.
template <int D, int MT, bool BF>
__global__ __launch_bounds__(64 * kWaves, few_resident(D, MT)) void k_kv4_attn_few(Kv4AttnArgs a) {
  constexpr int R = 16 * MT, LD = D + 4, W = kWaves;
  extern __shared__ float lds[];  // [W][R][LD] sums, then [W][R][2] (reference, weight)
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, g = lane >> 4;
  float* ml = lds + W * R * LD;

  const Kv4Found found = a.list ? listed_work<R>(a, D) : find_work<R>(a, D, lane);
  const auto same = [](int v) { return __builtin_amdgcn_readfirstlane(v); };  // in scalar registers
  const int n = same(found.tiles), row0 = same(found.row0), tile0 = same(found.first);
  if (!n) return;
  const Kv4Work wk = {same(found.w.e),    same(found.w.head), same(found.w.parts), same(found.w.part),
                      same(found.w.slot), same(found.w.group), 0,                  0};
  const Kv4Seq s = {same((int)found.s.q0), same(found.s.n), same(found.s.c)};
  const int rows = s.n * a.G, b = wk.e % a.B, head = wk.head, parts = wk.parts, slot = wk.slot;
  const Kv4Part part = kv4_part(n, parts, wk.part, 1);
  const int first = tile0 + part.first, last = tile0 + part.last;

  {
    Rows<D, MT, BF, true> r;
    Tiles<D> t;
    t.open(a, a.table + b * a.table_stride, head, first + wave, last, W, lane);
    r.fetch(a, s, head, row0, rows, col, g);
    if (t.tile < t.last) t.keys(), t.vals();
    r.load(a, s);
    r.run(t, s.c, g);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const float l = sum_g(r.lsum[m]), shift = r.shift(m);
      float* o = lds + (wave * R + m * 16 + col) * LD;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int h = 0; h < D / 64; ++h) *(v4f*)(o + (g * 4 + i) * (D / 16) + 4 * h) = r.sums(m, i, h, shift);
      if (g == 0) {
        float* p = ml + (wave * R + m * 16 + col) * 2;
        p[0] = r.ref[m] == kNone ? kNegInf : r.ref[m];
        p[1] = l;
      }
    }
  }
  __syncthreads();
  constexpr int kParts = D / 4;  // threads of a row, 4 channels each
#pragma unroll 1
  for (int it = threadIdx.x; it < R * kParts; it += 64 * W) {
    const int row = it / kParts, d = (it - row * kParts) * 4;
    if (row0 + row >= rows) continue;
    float ref = kNegInf;
#pragma unroll
    for (int v = 0; v < W; ++v) ref = fmaxf(ref, ml[(v * R + row) * 2]);
    v4f o = {0.f, 0.f, 0.f, 0.f};
    float l = 0.f;
#pragma unroll
    for (int v = 0; v < W; ++v) {
      const float rw = ml[(v * R + row) * 2];
      const float f = rw == kNegInf ? 0.f : __builtin_amdgcn_exp2f(rw - ref);  // a wave without tiles holds zeros
      l = fmaf(f, ml[(v * R + row) * 2 + 1], l);
      o += f * *(const v4f*)(lds + (v * R + row) * LD + d);
    }
    if (parts == 1) {
      const int i = (row0 + row) / a.G;
      const int64_t orow = (s.q0 + i) * a.Hq + head * a.G + (row0 + row - i * a.G);
      store4<BF>(a.out, orow * D + d, o * (ref == kNegInf ? 0.f : 1.0f / l));
      if (a.lse && d == 0) a.lse[orow] = log_sum(ref, l);
    } else {
      *(v4f*)(a.part + ((int64_t)slot * R + row) * D + d) = o;
      if (d == 0) *(float2*)(part_stats(a, D) + ((int64_t)slot * R + row) * 2) = make_float2(ref, l);
    }
  }
  if (parts > 1 && wk.part == 0 && threadIdx.x == 0) set_group(a, D, wk, s, row0);
}

// Many rows a key head (a prompt): 4 waves of 16*MT rows each, every wave over
// all tokens that the workgroup's rows see, straight from its registers to the
// output.  What bounds it is instructions: per 32 rows and 32 tokens 34 matrix
// products of 20 cycles and 200 vector instructions, which two waves a SIMD
// overlap little (a loop of both takes the sum of the two).  So keys and values
// are unpacked once for four waves, two tiles a barrier: 705 TFLOP/s where all
// CUs are busy, 61 % of a large library product (730, 664 with a wave unpacking
// for itself and 623 with 16 rows a wave and twice the waves, all while the
// reference went by scores).  Three prompt chunks of up to 1500 tokens (32 query
// heads) behind up to 3500 take 206 us, list and join with them; without parts
// of even length the longest row tiles run alone at the end (262 us).  A
// probability times its scale is rounded once to binary16: with the remainder
// the chunks take 257 us, 4096 tokens of a prompt 289 instead of 218, for an
// error of 2.1e-4 instead of 2.8e-4.
template <int D, int MT, bool BF>
__global__ __launch_bounds__(256, 2) void k_kv4_attn_many(Kv4AttnArgs a) {
  constexpr int R = 64 * MT;
  constexpr int TPS = D <= 128 ? 2 : 1;
  __shared__ v4u staged[2 * Staged<D, TPS>::kStep];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, g = lane >> 4;
  Kv4Found found;
  if (a.list) {
    found = listed_work<R>(a, D);
  } else {
    const int id = gridDim.x - 1 - blockIdx.x, e = id / a.Hk;  // the longest causal ranges first
    found = found_entry<R>(a, {e, id - e * a.Hk, 1, 0, 0, 0, 0, 0});
  }
  const Kv4Work& wk = found.w;
  if (!found.tiles) return;
  const Kv4Seq& s = found.s;
  const int n = found.tiles, row0 = found.row0, first = found.first;
  const int rows = s.n * a.G, b = wk.e % a.B, head = wk.head, wrow = row0 + wave * 16 * MT;
  const bool split = wk.parts > 1;
  const Kv4Part range = kv4_part(n, wk.parts, wk.part, TPS);
  const int tbeg = first + range.first, tend = first + range.last;
  if (split && wk.part == 0 && threadIdx.x == 0) set_group(a, D, wk, s, row0);

  Rows<D, MT, BF, false> r;
  Staged<D, TPS> t;
  r.fetch(a, s, head, wrow, rows, col, g);
  if (tbeg < tend) t.open(a, staged, a.table + b * a.table_stride, head, tbeg, tend, lane, wave);
  r.load(a, s);
  if (tbeg < tend) r.run(t, s.c, g);
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int row = wrow + m * 16 + col;
    const float l = sum_g(r.lsum[m]), shift = r.shift(m);
    if (row >= rows) continue;
    const bool none = r.ref[m] == kNone;
    const int i = row / a.G;
    const int64_t orow = (s.q0 + i) * a.Hq + head * a.G + (row - i * a.G);
    const int64_t part = (int64_t)wk.slot * R + row - row0;
    const float inv = split ? 1.0f : none ? 0.f : 1.0f / l;
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        const int d = (g * 4 + e) * (D / 16) + 4 * h;
        const v4f y = r.sums(m, e, h, shift) * inv;
        if (split) {
          *(v4f*)(a.part + part * D + d) = y;
        } else {
          store4<BF>(a.out, orow * D + d, y);
        }
      }
    if (g == 0) {
      if (split) {
        float* p = part_stats(a, D) + part * 2;
        p[0] = none ? kNegInf : r.ref[m];
        p[1] = l;
      } else if (a.lse) {
        a.lse[orow] = log_sum(none ? kNegInf : r.ref[m], l);
      }
    }
  }
}

// Joins the parts of a row in their order: one workgroup per row, D/4 lanes a
// part.  A part that saw nothing holds zeros.  Latency: four dependent loads
// and two barriers, 5 us; more threads where few rows have hundreds of parts.
constexpr int kMostParts = 1024;
template <int D, bool BF, int kJoin>
__global__ __launch_bounds__(kJoin) void k_kv4_join(Kv4AttnArgs a) {
  constexpr int LN = D / 4, NS = kJoin / LN;
  __shared__ float weight[kMostParts], red[2][kJoin / 64], part[NS][D];
  const Kv4Group* groups = part_groups(a, D);
  const Kv4Group grp = groups[blockIdx.y];
  const int row = blockIdx.x;
  if ((int)blockIdx.y >= groups->groups || grp.count < 2 || grp.row0 + row >= grp.rows) return;
  const float2* ml = (const float2*)part_stats(a, D) + (int64_t)grp.slot * a.rows + row;
  const float* sums = a.part + ((int64_t)grp.slot * a.rows + row) * D;
  // weights of the parts: 2^(reference - largest)
  float top = kNegInf, sum = 0.f;
  for (int k = threadIdx.x; k < grp.count; k += kJoin) top = fmaxf(top, ml[(int64_t)k * a.rows].x);
  for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
  if ((threadIdx.x & 63) == 0) red[0][threadIdx.x >> 6] = top;
  __syncthreads();
  float ref = red[0][0];
#pragma unroll
  for (int v = 1; v < kJoin / 64; ++v) ref = fmaxf(ref, red[0][v]);
  for (int k = threadIdx.x; k < grp.count; k += kJoin) {
    const float2 m = ml[(int64_t)k * a.rows];
    const float f = m.x == kNegInf ? 0.f : __builtin_amdgcn_exp2f(m.x - ref);
    weight[k] = f;
    sum = fmaf(f, m.y, sum);
  }
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
  if ((threadIdx.x & 63) == 0) red[1][threadIdx.x >> 6] = sum;
  __syncthreads();
  const int l = threadIdx.x % LN, k0 = threadIdx.x / LN;
  v4f o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int k = k0; k < grp.count; k += NS) o += weight[k] * *(const v4f*)(sums + (int64_t)k * a.rows * D + 4 * l);
  *(v4f*)&part[k0][4 * l] = o;
  __syncthreads();
  if (threadIdx.x >= LN) return;
  for (int k = 1; k < NS; ++k) o += *(const v4f*)&part[k][4 * l];
  float all = 0.f;
#pragma unroll
  for (int v = 0; v < kJoin / 64; ++v) all += red[1][v];
  const int r = grp.row0 + row, i = r / a.G;
  const int64_t orow = ((int64_t)grp.q0 + i) * a.Hq + grp.head * a.G + (r - i * a.G);
  store4<BF>(a.out, orow * D + 4 * l, o * (ref == kNegInf ? 0.f : 1.0f / all));
  if (a.lse && l == 0) a.lse[orow] = log_sum(ref, all);
}

// The same for many rows of few parts each: D/4 lanes a row.
template <int D, bool BF>
__global__ __launch_bounds__(256) void k_kv4_join_rows(Kv4AttnArgs a) {
  constexpr int LN = D / 4;
  const Kv4Group* groups = part_groups(a, D);
  const Kv4Group grp = groups[blockIdx.y];
  const int row = blockIdx.x * (256 / LN) + threadIdx.x / LN, l = threadIdx.x % LN;
  if ((int)blockIdx.y >= groups->groups || grp.count < 2 || grp.row0 + row >= grp.rows) return;
  const float2* ml = (const float2*)part_stats(a, D) + (int64_t)grp.slot * a.rows + row;
  const float* sums = a.part + ((int64_t)grp.slot * a.rows + row) * D + 4 * l;
  float ref = kNegInf, all = 0.f;
  for (int k = 0; k < grp.count; ++k) ref = fmaxf(ref, ml[(int64_t)k * a.rows].x);
  v4f o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int k = 0; k < grp.count; ++k) {
    const float2 m = ml[(int64_t)k * a.rows];
    const float f = m.x == kNegInf ? 0.f : __builtin_amdgcn_exp2f(m.x - ref);
    all = fmaf(f, m.y, all);
    o += f * *(const v4f*)(sums + (int64_t)k * a.rows * D);
  }
  const int r = grp.row0 + row, i = r / a.G;
  const int64_t orow = ((int64_t)grp.q0 + i) * a.Hq + grp.head * a.G + (r - i * a.G);
  store4<BF>(a.out, orow * D + 4 * l, o * (ref == kNegInf ? 0.f : 1.0f / all));
  if (a.lse && l == 0) a.lse[orow] = log_sum(ref, all);
}

template <int D, bool BF>
hipError_t attn_join(const Kv4AttnArgs& a, const Kv4AttnPlan& p, hipStream_t s) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !p.groups) return e;
  const int64_t rows = (int64_t)a.max_q * a.G;
  const dim3 few((uint32_t)(rows < p.rows ? rows : p.rows), p.groups);
  // few rows to join: more parts of each at once (2 groups 21.3 -> 20.8 us the
  // two kernels, 8 19.5 -> 18.8; but 64 15.7 -> 16.5, 128 40.9 -> 41.7)
  if (p.few && p.groups < 64)
    hipLaunchKernelGGL((k_kv4_join<D, BF, 512>), few, dim3(512), 0, s, a);
  else if (p.few)
    hipLaunchKernelGGL((k_kv4_join<D, BF, 256>), few, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((k_kv4_join_rows<D, BF>), dim3(p.rows / (1024 / D), p.groups), dim3(256), 0, s, a);
  return hipGetLastError();
}
template <int D, int MT, bool BF>
hipError_t attn_few(const Kv4AttnArgs& a, const Kv4AttnPlan& p, hipStream_t s) {
  constexpr int W = kWaves;
  if (p.list) hipLaunchKernelGGL((k_kv4_deal<16 * MT>), dim3(1), dim3(kDeal), 0, s, a, D);
  hipLaunchKernelGGL((k_kv4_attn_few<D, MT, BF>), dim3((uint32_t)p.grid), dim3(64 * W), W * 16 * MT * (D + 6) * 4, s, a);
  return attn_join<D, BF>(a, p, s);
}
template <int D, int MT, bool BF>
hipError_t attn_many(const Kv4AttnArgs& a, const Kv4AttnPlan& p, hipStream_t s) {
  if (p.list) hipLaunchKernelGGL((k_kv4_deal<64 * MT>), dim3(1), dim3(kDeal), 0, s, a, D);
  hipLaunchKernelGGL((k_kv4_attn_many<D, MT, BF>), dim3((uint32_t)p.grid), dim3(256), 0, s, a);
  return attn_join<D, BF>(a, p, s);
}
template <int D, bool BF>
hipError_t attn_d(const Kv4AttnArgs& a, const Kv4AttnPlan& p, hipStream_t s) {
  if (p.few) return p.mt == 1 ? attn_few<D, 1, BF>(a, p, s) : attn_few<D, 2, BF>(a, p, s);
  if constexpr (D < 256) {
    if (p.mt == 2) return attn_many<D, 2, BF>(a, p, s);
  }
  return attn_many<D, 1, BF>(a, p, s);
}
template <bool BF>
hipError_t attn_go(const Kv4AttnArgs& a, const Kv4AttnPlan& p, hipStream_t s) {
  return a.D == 64 ? attn_d<64, BF>(a, p, s) : a.D == 128 ? attn_d<128, BF>(a, p, s) : attn_d<256, BF>(a, p, s);
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

// Tokens of a workgroup: 32, the cache's value tile; where that leaves less
// than two workgroups a CU, as few as a workgroup's rows hold.
constexpr int kFewTokens[] = {16, 8, 8};  // of heads of 64, 128, 256
template <template <int, int, int> class K, class A>
hipError_t cache_go(const A& a, int dtype, hipStream_t s) {
  const auto at = [&](auto dt, auto d) {
    constexpr int DT = decltype(dt)::value, D = decltype(d)::value, FEW = kFewTokens[D / 128];
    const bool few = a.T * a.Hk < 2 * 256 * 32;
    const int tok = few ? FEW : 32;
    const dim3 grid((uint32_t)((a.T + 2 * (tok - 1)) / tok * a.Hk));
    if (few)
      K<DT, D, FEW>::go(a, grid, s);
    else
      K<DT, D, 32>::go(a, grid, s);
  };
  const auto of = [&](auto dt) {
    if (a.D == 64)
      at(dt, std::integral_constant<int, 64>());
    else if (a.D == 128)
      at(dt, std::integral_constant<int, 128>());
    else
      at(dt, std::integral_constant<int, 256>());
  };
  if (dtype == kF16)
    of(std::integral_constant<int, kF16>());
  else if (dtype == kBF16)
    of(std::integral_constant<int, kBF16>());
  else
    of(std::integral_constant<int, kF32>());
  return hipGetLastError();
}
template <int DT, int D, int TOK>
struct Store {
  static void go(const Kv4StoreArgs& a, dim3 grid, hipStream_t s) {
    hipLaunchKernelGGL((k_kv4_store<DT, D, TOK>), grid, dim3(256), 0, s, a);
  }
};
template <int DT, int D, int TOK>
struct Load {
  static void go(const Kv4LoadArgs& a, dim3 grid, hipStream_t s) {
    hipLaunchKernelGGL((k_kv4_load<DT, D, TOK>), grid, dim3(256), 0, s, a);
  }
};

}  // namespace

hipError_t launch_kv4_store(const Kv4StoreArgs& a, int dtype, hipStream_t s) { return cache_go<Store>(a, dtype, s); }
hipError_t launch_kv4_load(const Kv4LoadArgs& a, int dtype, hipStream_t s) { return cache_go<Load>(a, dtype, s); }

hipError_t launch_qk_norm_rope(const RopeArgs& a, int in_dtype, int out_dtype, hipStream_t s) {
  int lanes = 1;
  while (16 * lanes < a.D) lanes *= 2;
  const int H = a.Hq + a.Hk, slots = 256 / lanes;
  // few tokens: one pass of heads per workgroup; many: four tokens with all
  // their heads, so that a workgroup's last pass is seldom empty
  const bool few = a.T * ((H + slots - 1) / slots) <= 1024;
  // (eight where four would ask for 2^32 threads, which no grid holds)
  const int tokens = few ? 1 : a.T <= (1 << 25) ? 4 : 8, hpw = few ? slots : H;
  const dim3 grid((uint32_t)((a.T + tokens - 1) / tokens), (H + hpw - 1) / hpw);
  const size_t lds = (size_t)tokens * (a.rot / 2) * 8;
  return in_dtype == kF16    ? rope_dst<kF16>(a, out_dtype, grid, lds, s, tokens, hpw, lanes)
         : in_dtype == kBF16 ? rope_dst<kBF16>(a, out_dtype, grid, lds, s, tokens, hpw, lanes)
                             : rope_dst<kF32>(a, out_dtype, grid, lds, s, tokens, hpw, lanes);
}

hipError_t launch_kv4_attn(Kv4AttnArgs a, const Kv4AttnPlan& p, int dtype, hipStream_t s) {
  a.tiles = p.tiles;
  a.budget = p.budget;
  a.least = p.least;
  a.grain = p.grain;
  a.list = p.list;
  a.slots = p.slots;
  a.rows = p.rows;
  a.groups = p.groups;
  return dtype == kBF16 ? attn_go<true>(a, p, s) : attn_go<false>(a, p, s);
}

}  // namespace tq2
