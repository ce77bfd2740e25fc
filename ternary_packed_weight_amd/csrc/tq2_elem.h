// Element types of the calls that take binary16, bfloat16 or fp32 tensors, in
// device code: eight consecutive elements as floats, and back with one
// rounding (nearest even); and values of other lanes of a wave.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tq2 {
namespace elem {

constexpr int kF16 = 0, kBF16 = 1, kF32 = 2;  // tq2_dtype

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

template <int DT, int N>
using Vec = typename Elem<DT>::T __attribute__((ext_vector_type(N)));

template <int DT>
__device__ __forceinline__ void load8(const void* p, int64_t at, float (&x)[8]) {
  const typename Elem<DT>::T* e = (const typename Elem<DT>::T*)p + at;
  if constexpr (DT == kF32) {
    const Vec<DT, 4> a = *(const Vec<DT, 4>*)e, b = *(const Vec<DT, 4>*)(e + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = a[i], x[4 + i] = b[i];
  } else {
    const Vec<DT, 8> a = *(const Vec<DT, 8>*)e;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)a[i];
  }
}
template <int DT>
__device__ __forceinline__ void store8(void* p, int64_t at, const float (&x)[8]) {
  typename Elem<DT>::T* e = (typename Elem<DT>::T*)p + at;
  if constexpr (DT == kF32) {
    Vec<DT, 4> a, b;
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = x[i], b[i] = x[4 + i];
    *(Vec<DT, 4>*)e = a;
    *(Vec<DT, 4>*)(e + 4) = b;
  } else {
    Vec<DT, 8> a;
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = (typename Elem<DT>::T)x[i];
    *(Vec<DT, 8>*)e = a;
  }
}
// x rounded to the type and back
template <int DT>
__device__ __forceinline__ float rounded(float x) {
  return (float)(typename Elem<DT>::T)x;
}

// ---- lanes ----

// The value of lane ^ O.  Lanes of a row of 16 exchange through the vector
// unit's own moves, rows through its swaps: a step of the networks below takes
// some 20 cycles, through LDS it took more than 100.
template <int CTRL>
__device__ __forceinline__ uint32_t moved_by(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
template <int O>
__device__ __forceinline__ uint32_t across(uint32_t v, int lane) {
  if constexpr (O == 1) return moved_by<0xB1>(v);                    // quad_perm 1 0 3 2
  else if constexpr (O == 2) return moved_by<0x4E>(v);               // quad_perm 2 3 0 1
  else if constexpr (O == 4) return moved_by<0x1B>(moved_by<0x141>(v));  // half a row mirrored (^ 7), quads too (^ 3)
  else if constexpr (O == 8) return moved_by<0x128>(v);              // row rotated by 8
  else if constexpr (O == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);  // odd rows of one, even rows of the other
    return lane & 16 ? r[0] : r[1];
  } else {
    static_assert(O == 32, "a power of two below the wave");
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return lane & 32 ? r[0] : r[1];
  }
}
template <int O>
__device__ __forceinline__ uint64_t across(uint64_t v, int lane) {
  return ((uint64_t)across<O>((uint32_t)(v >> 32), lane) << 32) | across<O>((uint32_t)v, lane);
}
template <int O>
__device__ __forceinline__ float across(float v, int lane) {
  return __builtin_bit_cast(float, across<O>(__builtin_bit_cast(uint32_t, v), lane));
}
template <int O>
__device__ __forceinline__ double across(double v, int lane) {
  return __builtin_bit_cast(double, across<O>(__builtin_bit_cast(uint64_t, v), lane));
}

}  // namespace elem
}  // namespace tq2
