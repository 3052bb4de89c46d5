// route.hip -- the experts of each row by its logits.
//
// A row is held by LANES lanes, PER logits each, as unsigned keys in the
// order of the floats (a NaN above all of them, -0 as +0); topk times the
// largest key is joined over the lanes and taken out.  Equal logits go to the
// lowest index: 16-bit ones' keys hold the index below the logit, so that one
// join has both; fp32 ones' take a second join.  A few rows take one launch and a
// row's chain of choices (128 f32, 8 of them: 4.1 us); 8192 rows of 256 bf16, 8 of
// them, 6.4 us (7.6 with two joins) for 4.7 MB: 950 vector instructions a wave,
// most of them to find the largest of a lane's keys and to take it out, for every
// choice anew; a join is 8 of some 90 a choice.
#include "elements.h"
#include "launchers.h"

namespace gtk {

// A logit as a key, its value, and the largest key of -infinity; 0 is below every key.
template <int DT>
struct Keys {
  static constexpr bool kWhole = false;  // no index in it
  static constexpr uint32_t kMasked = 0x007fffffu;
  static __device__ __forceinline__ uint32_t key(const char* p, int e) {
    const float f = reinterpret_cast<const float*>(p)[e];
    const uint32_t u = __float_as_uint(f + 0.f);  // -0 becomes +0
    if (f != f) return 0xffffffffu;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
  }
  static __device__ __forceinline__ float value(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }
};
template <int DT>
struct HalfKeys {
  static constexpr bool kWhole = true;
  static constexpr uint32_t kInfinity = DT == DT_BF16 ? 0x7f80u : 0x7c00u;
  static constexpr uint32_t kMasked = (0x7fffu - kInfinity) << 16 | 0xffffu;
  static __device__ __forceinline__ uint32_t key(const char* p, int e) {
    uint32_t u = reinterpret_cast<const uint16_t*>(p)[e];
    u = u == 0x8000u ? 0u : u;
    uint32_t k = u & 0x8000u ? 0xffffu - u : u | 0x8000u;
    k = (u & 0x7fffu) > kInfinity ? 0xffffu : k;
    return k << 16 | (0xffffu - (uint32_t)e);
  }
  static __device__ __forceinline__ float value(uint32_t k) {
    const uint32_t u = k & 0x80000000u ? k >> 16 & 0x7fffu : 0xffffu - (k >> 16);
    return half_to_f32<DT>(u, 0);
  }
  static __device__ __forceinline__ int index(uint32_t k) { return (int)(0xffffu - (k & 0xffffu)); }
};
template <>
struct Keys<DT_F16> : HalfKeys<DT_F16> {};
template <>
struct Keys<DT_BF16> : HalfKeys<DT_BF16> {};

// A value joined over LANES neighbouring lanes, the same in all of them.
template <int LANES, class F>
__device__ __forceinline__ uint32_t lanes_join(uint32_t v, F f) {
  if constexpr (LANES == 64) return wave_join(v, f);
  v = f(v, dpp<0xB1>(v));
  v = f(v, dpp<0x4E>(v));
  v = f(v, dpp<0x141>(v));
  return f(v, dpp<0x140>(v));
}
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
  return __uint_as_float(lanes_join<LANES>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

template <int DT, int LANES, int PER>
__global__ __launch_bounds__(256) void route_kernel(gt::RouteArgs a) {
  typedef Keys<DT> Key;
  constexpr int kRows = 256 / LANES;
  constexpr uint32_t kMasked = Key::kMasked;
  const int lane = threadIdx.x % LANES;
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / LANES;
  const int64_t m = row < a.M ? row : a.M - 1;  // every lane takes part in the joins
  const char* p = static_cast<const char*>(a.logits) + m * a.ldl * (DT == DT_F32 ? 4 : 2);
  uint32_t key[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = j * LANES + lane;
    key[j] = e < a.E ? Key::key(p, e) : 0u;
  }
  auto largest = [](uint32_t x, uint32_t y) { return x > y ? x : y; };
  uint32_t mine = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) mine = largest(mine, key[j]);
  const uint32_t top = lanes_join<LANES>(mine, largest);
  const float most = top > kMasked ? Key::value(top) : 0.f;  // nothing left: no sum is used
  float all = 0.f;
  if (!a.sigmoid && !a.normalise) {
    // fast exponentials: one of an argument d is off by |d| of fp32's half steps, and with what it
    // carries of the sum all of 1024 by 4.5 at most, less than the sum's own 22 roundings may be.
    // Whole ones cost 8192 x 256 8.4 us for 7.5.
#pragma unroll
    for (int j = 0; j < PER; ++j) all += key[j] > kMasked ? __expf(Key::value(key[j]) - most) : 0.f;
    all = lanes_sum<LANES>(all);
  }
  int chosen = -1;          // of slot `lane`
  float logit = 0.f;
  uint32_t best = top;
  for (int s = 0; s < a.topk; ++s) {
    if (s > 0) {
      mine = 0;
#pragma unroll
      for (int j = 0; j < PER; ++j) mine = largest(mine, key[j]);
      best = lanes_join<LANES>(mine, largest);
    }
    if (best <= kMasked) best = 0u;  // nothing is left: no key is taken out
    int at;
    if constexpr (Key::kWhole) {
      at = Key::index(best);
#pragma unroll
      for (int j = 0; j < PER; ++j) key[j] = key[j] == best ? 0u : key[j];
    } else {
      at = 0x7fffffff;
#pragma unroll
      for (int j = PER - 1; j >= 0; --j) at = best && key[j] == best ? j * LANES + lane : at;
      at = (int)lanes_join<LANES>((uint32_t)at, [](uint32_t x, uint32_t y) { return x < y ? x : y; });
#pragma unroll
      for (int j = 0; j < PER; ++j) key[j] = at == j * LANES + lane ? 0u : key[j];
    }
    if (lane == s) {
      chosen = best ? at : -1;
      logit = Key::value(best);
    }
  }
  // With m = min(largest, 0) a sigmoid is exp(m) times what is here, so that
  // the quotient by the sum stands where all of them are below fp32's range.
  float w = 0.f;
  if (chosen >= 0) {
    if (a.sigmoid) {
      const float low = a.normalise && most < 0.f ? most : 0.f;
      w = logit >= 0.f ? 1.f / (1.f + expf(-logit)) : expf(logit - low) / (1.f + expf(logit));
    } else {
      w = expf(logit - most);
    }
  }
  if (a.normalise) all = lanes_sum<LANES>(w);
  if (a.normalise || !a.sigmoid) w = w / all;
  if (row < a.M && lane < a.topk) {
    a.index[row * a.ldi + lane] = chosen;
    a.weight[row * a.ldw + lane] = chosen >= 0 ? w * a.scale : 0.f;
  }
}

}  // namespace gtk

namespace gt {

// (launches of 2^22 workgroups: a grid has fewer than 2^32 threads)
template <int DT>
int route(const RouteArgs& all) {
  const bool few = all.topk > 16 || all.E > 256;
  const int64_t rows = few ? 4 : 16, most = rows << 22;
  for (int64_t m = 0; m < all.M; m += most) {
    RouteArgs a = all;
    a.M = all.M - m < most ? all.M - m : most;
    a.logits = static_cast<const char*>(all.logits) + m * all.ldl * elem_bytes(DT);
    a.index = all.index + m * all.ldi;
    a.weight = all.weight + m * all.ldw;
    const dim3 grid((unsigned)((a.M + rows - 1) / rows)), block(256);
#define GT_ROUTE(LANES, PER) \
  if (a.E <= LANES * PER) { hipLaunchKernelGGL((gtk::route_kernel<DT, LANES, PER>), grid, block, 0, a.stream, a); }
    if (few) {
      GT_ROUTE(64, 4) else GT_ROUTE(64, 8) else GT_ROUTE(64, 16)
    } else {
      GT_ROUTE(16, 4) else GT_ROUTE(16, 8) else GT_ROUTE(16, 16)
    }
#undef GT_ROUTE
  }
  return hipGetLastError() == hipSuccess ? LS_OK : LS_HIP_ERROR;
}

int launch_route(const RouteArgs& a) {
  if (a.dtype == DT_F32) return route<DT_F32>(a);
  return a.dtype == DT_F16 ? route<DT_F16>(a) : route<DT_BF16>(a);
}

}  // namespace gt
