// Element types of the calls that take binary16, bfloat16 or fp32 tensors, in
// device code: eight consecutive elements as floats, and back with one
// rounding (nearest even).
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

}  // namespace elem
}  // namespace tq2
