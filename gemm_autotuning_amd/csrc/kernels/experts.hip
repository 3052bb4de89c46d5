// experts.hip -- a layer of gated experts for a few tokens.
#include "elements.h"
#include "launchers.h"

namespace gtk {

constexpr int kInt4 = 0, kE2m1 = 1;

__device__ __forceinline__ float wave_sum(float v) {
  return __uint_as_float(wave_join(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

// Weight (e, n, k) as a float.
__device__ __forceinline__ float expert_weight(const gt::ExpertWeights& w, int64_t e, int64_t n, int64_t k, int dtype, int format,
                                               int scale_dtype, int group_lg) {
  const char* row = w.p + e * w.stride + n * w.ld;
  if (format < 0) return load_any(row, k, dtype);
  const uint32_t c = (uint8_t)row[k >> 1] >> (4 * (k & 1)) & 15u;
  float v;
  if (format == kInt4) {
    v = (float)((int)(c << 28) >> 28);
  } else {
    const uint32_t m = c & 7u;
    v = m < 2 ? 0.5f * m : __uint_as_float(((m >> 1) + 126u) << 23 | (m & 1u) << 22);
    v = c & 8u ? -v : v;
  }
  return v * load_any(w.scales, e * w.s_lde + n * w.s_ldn + (k >> group_lg) * w.s_ldg, scale_dtype);
}

__device__ __forceinline__ float activated(float g, float u, int activation) {
  // GELU's tanh form is g / (1 + exp(-2 z)), z = sqrt(2 / pi) (g + 0.044715 g^3)
  const float z = activation == 0 ? g : 1.5957691216057308f * (g + 0.044715f * g * g * g);
  return g / (1.f + expf(-z)) * u;
}

__global__ __launch_bounds__(256) void moe_up_kernel(gt::MoeArgs a, float* act) {
  const int lane = threadIdx.x & 63;
  const int64_t h = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t pair = blockIdx.y, t = pair / a.topk;
  const int e = a.index[t * a.ldi + pair % a.topk];
  if (h >= a.H || e < 0 || e >= a.E) return;
  float g = 0.f, u = 0.f;
  for (int64_t k = lane; k < a.K; k += 64) {
    const float x = load_any(a.x, t * a.ldx + k, a.x_dtype);
    g += x * expert_weight(a.gate_up, e, h, k, a.x_dtype, a.format, a.scale_dtype, a.group_lg);
    u += x * expert_weight(a.gate_up, e, a.H + h, k, a.x_dtype, a.format, a.scale_dtype, a.group_lg);
  }
  g = wave_sum(g);
  u = wave_sum(u);
  if (lane == 0) act[pair * a.H + h] = activated(g, u, a.activation);
}

__global__ __launch_bounds__(256) void moe_down_kernel(gt::MoeArgs a, const float* act) {
  const int lane = threadIdx.x & 63;
  const int64_t n = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6), t = blockIdx.y;
  if (n >= a.K) return;
  float y = a.base ? load_any(a.base, t * a.ldb + n, a.out_dtype) : 0.f;
  for (int j = 0; j < a.topk; ++j) {
    const int e = a.index[t * a.ldi + j];
    if (e < 0 || e >= a.E) continue;
    float v = 0.f;
    for (int64_t k = lane; k < a.H; k += 64)
      v += act[(t * a.topk + j) * a.H + k] * expert_weight(a.down, e, n, k, a.x_dtype, a.format, a.scale_dtype, a.group_lg);
    y += a.weight[t * a.ldw + j] * wave_sum(v);
  }
  if (lane == 0) store_out(a.y, t * a.ldy + n, y, a.out_dtype);
}

}  // namespace gtk

namespace gt {

int64_t moe_range(const MoeArgs& a) {
  const int64_t pairs = ((int64_t)64 << 20) / (4 * a.H);
  const int64_t t = (pairs < 2048 ? pairs : 2048) / a.topk;
  return t > 0 ? t : 1;
}
size_t moe_workspace_bytes(const MoeArgs& a, int64_t tokens) { return (size_t)(tokens * a.topk * a.H * 4); }

int launch_moe(const MoeArgs& a) {
  float* act = reinterpret_cast<float*>(a.ws);
  hipLaunchKernelGGL(gtk::moe_up_kernel, dim3((unsigned)((a.H + 3) / 4), (unsigned)(a.M * a.topk)), dim3(256), 0, a.stream, a, act);
  hipLaunchKernelGGL(gtk::moe_down_kernel, dim3((unsigned)((a.K + 3) / 4), (unsigned)a.M), dim3(256), 0, a.stream, a, act);
  return hipGetLastError() == hipSuccess ? LS_OK : LS_HIP_ERROR;
}

}  // namespace gt
