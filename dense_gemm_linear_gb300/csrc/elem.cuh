// Elements of a row in units of up to 16 bytes (or two such): loads, conversions to and from
// fp32, stores.  For the kernels that are bound by memory (norm.cu, embed.cu,
// adamw.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace dgl {

template <int BYTES>
struct UnitOf;
template <>
struct UnitOf<2> {
  using type = uint16_t;
};
template <>
struct UnitOf<4> {
  using type = uint32_t;
};
template <>
struct UnitOf<8> {
  using type = uint2;
};
template <>
struct UnitOf<16> {
  using type = uint4;
};
struct alignas(16) TwoUnits {  // accessed as two units of 16 bytes
  uint4 lo, hi;
};
template <>
struct UnitOf<32> {
  using type = TwoUnits;
};

// N elements of T as one access of N sizeof(T) bytes.
template <class T, int N>
using Unit = typename UnitOf<static_cast<int>(sizeof(T)) * N>::type;

template <class T, int N>
__device__ __forceinline__ Unit<T, N> load_unit(const T* p) {
  return *reinterpret_cast<const Unit<T, N>*>(p);
}

// A load of what this kernel reads once: it leaves no line in L1.
template <class T, int N>
__device__ __forceinline__ Unit<T, N> load_unit_once(const T* p) {
  return __ldcg(reinterpret_cast<const Unit<T, N>*>(p));
}

template <class T, int N>
__device__ __forceinline__ void unpack(const Unit<T, N>& u, float (&f)[N]) {
  if constexpr (sizeof(T) == 2 && N >= 2) {
    const uint32_t* two = reinterpret_cast<const uint32_t*>(&u);
#pragma unroll
    for (int i = 0; i < N; i += 2) {  // a bf16 is the upper half of an fp32
      f[i] = __uint_as_float(two[i / 2] << 16);
      f[i + 1] = __uint_as_float(two[i / 2] & 0xffff0000u);
    }
  } else {
    const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (sizeof(T) == 2) f[i] = __bfloat162float(e[i]);
      else f[i] = e[i];
    }
  }
}

// Rounds to nearest even where T is bf16.
template <class T, int N>
__device__ __forceinline__ void store_unit(T* p, const float (&f)[N]) {
  Unit<T, N> u;
  if constexpr (sizeof(T) == 2 && N >= 2) {
    __nv_bfloat162* two = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
    for (int i = 0; i < N; i += 2) two[i / 2] = __floats2bfloat162_rn(f[i], f[i + 1]);
  } else {
    T* e = reinterpret_cast<T*>(&u);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (sizeof(T) == 2) e[i] = __float2bfloat16_rn(f[i]);
      else e[i] = f[i];
    }
  }
  *reinterpret_cast<Unit<T, N>*>(p) = u;
}

template <class T>
__device__ __forceinline__ float to_float(T v) {
  if constexpr (sizeof(T) == 2) return __bfloat162float(v);
  else return v;
}

template <class T>
__device__ __forceinline__ T from_float(float v) {
  if constexpr (sizeof(T) == 2) return __float2bfloat16_rn(v);
  else return v;
}

}  // namespace dgl
