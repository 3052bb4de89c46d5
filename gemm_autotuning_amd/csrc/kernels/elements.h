// elements.h -- element types of the operators around the product: loads and
// stores of one element or of a piece of a row, converted from and to fp32,
// and joins over a wave.
#pragma once

#include "common.h"

namespace gtk {

using gt::DT_BF16;
using gt::DT_E4M3;
using gt::DT_F16;
using gt::DT_F32;

typedef __attribute__((ext_vector_type(2))) float f32x2v;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2v;
typedef __attribute__((ext_vector_type(2))) _Float16 f16x2v;

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

// E consecutive elements of a row as stored.  Rows may start at any element,
// so the wide accesses are unaligned ones (the device takes them; an aligned
// row costs no more).
template <int DT, int E>
struct Piece {
  typedef typename Elem<DT>::T T;
  static constexpr int kWords = E * (int)sizeof(T) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  __device__ __forceinline__ void load(const T* p) { __builtin_memcpy(w, p, sizeof(w)); }
  __device__ __forceinline__ void set(int e, T v) {  // of a cleared piece
    if constexpr (DT == DT_F32)
      w[e] = __float_as_uint(v);
    else
      w[e / 2] |= (uint32_t)v << (16 * (e & 1));
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (DT == DT_F32) return __uint_as_float(w[e]);
    if constexpr (DT == DT_BF16) return __uint_as_float((e & 1) ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
    return f16_bits_to_f32((uint16_t)(w[e / 2] >> (16 * (e & 1))));
  }
};

// E floats rounded to DT and stored; past the caches where the call writes
// more than they hold for its reader (kPastCaches).
template <int DT, int E>
__device__ __forceinline__ void store_piece(typename Elem<DT>::T* p, const float* v, bool past_caches = false) {
  constexpr int kWords = E * (int)sizeof(*p) / 4;
  uint32_t w[kWords];
  if constexpr (DT == DT_F32) {
#pragma unroll
    for (int e = 0; e < E; ++e) w[e] = __float_as_uint(v[e]);
  } else if constexpr (DT == DT_E4M3) {
#pragma unroll
    for (int e = 0; e < E; e += 4) {
      const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(Elem<DT>::clip(v[e]), Elem<DT>::clip(v[e + 1]), 0, false);
      w[e / 4] = __builtin_amdgcn_cvt_pk_fp8_f32(Elem<DT>::clip(v[e + 2]), Elem<DT>::clip(v[e + 3]), lo, true);
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const f32x2v f = {v[e], v[e + 1]};
      if constexpr (DT == DT_BF16) {
        const bf16x2v h = __builtin_convertvector(f, bf16x2v);
        __builtin_memcpy(&w[e / 2], &h, 4);
      } else {
        const f16x2v h = __builtin_convertvector(f, f16x2v);
        __builtin_memcpy(&w[e / 2], &h, 4);
      }
    }
  }
  if (past_caches) {
    typedef __attribute__((ext_vector_type(kWords))) uint32_t words;
    typedef words words_any __attribute__((aligned(1)));
    words t;
    __builtin_memcpy(&t, w, sizeof(w));
    __builtin_nontemporal_store(t, reinterpret_cast<words_any*>(p));
  } else {
    __builtin_memcpy(p, w, sizeof(w));
  }
}

// Bytes that a call reads and writes from which on its results are stored
// past the caches.  The last-level cache holds 256 MB: below, a reader that
// follows finds them there (11000 x 8192 expanded to bf16, then a product of
// 512 rows: 126 us, 137 past the caches); above, they only drive each other
// out (12000 x 8192: 154 and 145, 14000 x 8192: 187 and 161).
constexpr double kPastCaches = 240e6;

// E weights from n on, of a type known at run time.
template <int E>
__device__ __forceinline__ void load_weights(const void* p, unsigned n, int dtype, float* out) {
  if (dtype == DT_F32) {
    __builtin_memcpy(out, reinterpret_cast<const float*>(p) + n, 4 * E);
  } else {
    Piece<DT_BF16, E> b;
    b.load(reinterpret_cast<const uint16_t*>(p) + n);
    if (dtype == DT_BF16) {
#pragma unroll
      for (int e = 0; e < E; ++e) out[e] = b.get(e);
    } else {
      Piece<DT_F16, E> h;
      __builtin_memcpy(&h, &b, sizeof(h));
#pragma unroll
      for (int e = 0; e < E; ++e) out[e] = h.get(e);
    }
  }
}

// A value of every lane joined over the wave, the same bits in every lane:
// four exchanges inside a row of 16 lanes by data-parallel moves, then one
// between the rows of each half and one between the halves.  No LDS trip.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
// The lower or upper 16-bit element of a dword.
template <int XT>
__device__ __forceinline__ float half_to_f32(uint32_t u, int upper) {
  if constexpr (XT == DT_BF16) return __uint_as_float(upper ? u & 0xffff0000u : u << 16);
  return f16_bits_to_f32((uint16_t)(upper ? u >> 16 : u));
}
template <class F>
__device__ __forceinline__ uint32_t wave_join(uint32_t v, F f) {
  v = f(v, dpp<0xB1>(v));   // lanes 1 0 3 2
  v = f(v, dpp<0x4E>(v));   // lanes 2 3 0 1
  v = f(v, dpp<0x141>(v));  // the other four of eight, mirrored
  v = f(v, dpp<0x140>(v));  // the other eight of sixteen, mirrored
  const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = f(r[0], r[1]);
  const auto h = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return f(h[0], h[1]);
}
__device__ __forceinline__ float wave_sum(float v) {
  return __uint_as_float(wave_join(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

}  // namespace gtk
