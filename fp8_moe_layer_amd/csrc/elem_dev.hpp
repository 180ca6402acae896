// elem_dev.hpp -- element types of activations and outputs, stores of runs of
// them, and the sigmoid, for the dense operators, the norms and the 4-bit
// products.
#pragma once

#include "common.hpp"
#include "expert_dev.hpp"  // exp_neg

namespace fp8moe {

// ---------------------------------------------------------------- elements
template <class T>
struct Elem;
// 16 and 8 bytes at an address that is aligned for a 32-bit or a 16-bit value.
struct Align4 {
  typedef int Quad __attribute__((ext_vector_type(4), aligned(4)));
  typedef int Pair __attribute__((ext_vector_type(2), aligned(4)));
};
struct Align2 {
  typedef int Quad __attribute__((ext_vector_type(4), aligned(2)));
  typedef int Pair __attribute__((ext_vector_type(2), aligned(2)));
};
template <>
struct Elem<float> : Align4 {
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
};
template <>
struct Elem<__bf16> : Align2 {
  static __device__ __forceinline__ float get(__bf16 v) { return (float)v; }
  static __device__ __forceinline__ __bf16 put(float v) { return (__bf16)v; }
};
template <>
struct Elem<_Float16> : Align2 {
  static __device__ __forceinline__ float get(_Float16 v) { return (float)v; }
  static __device__ __forceinline__ _Float16 put(float v) { return (_Float16)v; }
};

// CNT consecutive values to dst, rounded once to T (nearest, ties to even);
// the first `valid` of them exist.  The wide stores ask for no more than T's
// alignment, which global memory takes at any address: rows of an odd length
// start anywhere (fp32, 333 x 1408 x 2051 int8: 8.6 us with single stores,
// 6.4 us so; 4099 x 2048 x 1409 51 and 27 us).
template <class T, int CNT>
__device__ __forceinline__ void store_run(T *dst, const float (&v)[CNT], int valid) {
  typedef typename Elem<T>::Quad Quad;
  typedef typename Elem<T>::Pair Pair;
  T tmp[CNT];
#pragma unroll
  for (int i = 0; i < CNT; ++i) tmp[i] = Elem<T>::put(v[i]);
  if (valid >= CNT) {
    constexpr int kBytes = CNT * (int)sizeof(T);
    if constexpr (kBytes >= 16) {
#pragma unroll
      for (int b = 0; b < kBytes / 16; ++b) {
        Quad w;
        __builtin_memcpy(&w, reinterpret_cast<const char *>(tmp) + b * 16, 16);
        reinterpret_cast<Quad *>(dst)[b] = w;
      }
    } else {
      Pair w;
      __builtin_memcpy(&w, tmp, 8);
      *reinterpret_cast<Pair *>(dst) = w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < CNT; ++i)
      if (i < valid) dst[i] = tmp[i];
  }
}

// 1 / (1 + e^-g) with the reciprocal instruction (1 ulp) for the divide.  g is
// held within +-130, where e^-g is 0 or infinite already: past 2.36e38 the
// exponent g * log2(e) would overflow, and the exponential's compensation make a
// NaN of it.
__device__ __forceinline__ float sigmoid(float g) {
  return __builtin_amdgcn_rcpf(1.0f + exp_neg(__builtin_amdgcn_fmed3f(g, -130.0f, 130.0f)));
}

// SiLU(g) * u.
__device__ __forceinline__ float silu_mul(float g, float u) { return g * sigmoid(g) * u; }

}  // namespace fp8moe
