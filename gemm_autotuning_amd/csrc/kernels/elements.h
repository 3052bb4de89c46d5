// elements.h -- element types of the operators around the product: loads and
// stores of one element or of a 16-byte piece, converted from and to fp32.
#pragma once

#include "common.h"

namespace gtk {

using gt::DT_BF16;
using gt::DT_E4M3;
using gt::DT_F16;
using gt::DT_F32;

template <int DT>
struct Elem;
template <>
struct Elem<DT_F32> {
  typedef float T;
  static __device__ __forceinline__ float get(T v) { return v; }
  static __device__ __forceinline__ T put(float f) { return f; }
};
template <>
struct Elem<DT_F16> {
  typedef uint16_t T;
  static __device__ __forceinline__ float get(T v) { return f16_bits_to_f32(v); }
  static __device__ __forceinline__ T put(float f) { return f32_to_f16_bits(f); }
};
template <>
struct Elem<DT_BF16> {
  typedef uint16_t T;
  static __device__ __forceinline__ float get(T v) { return bf16_bits_to_f32(v); }
  static __device__ __forceinline__ T put(float f) { return f32_to_bf16_bits(f); }
};
// e4m3 is an output only: to nearest even, saturating at +-448, NaN kept (a
// comparison with NaN is false, so NaN passes both selections).
template <>
struct Elem<DT_E4M3> {
  typedef uint8_t T;
  static __device__ __forceinline__ float clip(float f) { return f > 448.f ? 448.f : (f < -448.f ? -448.f : f); }
  static __device__ __forceinline__ T put(float f) {
    const float c = clip(f);
    return (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, c, 0, false);
  }
};

// An element of a type known only at run time (weights and scales, which are
// few beside the rows).
__device__ __forceinline__ float load_any(const void* p, int64_t i, int dtype) {
  if (dtype == DT_F32) return reinterpret_cast<const float*>(p)[i];
  const uint16_t b = reinterpret_cast<const uint16_t*>(p)[i];
  return dtype == DT_BF16 ? bf16_bits_to_f32(b) : f16_bits_to_f32(b);
}

}  // namespace gtk
