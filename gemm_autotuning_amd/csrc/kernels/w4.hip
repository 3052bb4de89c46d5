// w4.hip -- rows times 4-bit weights with group scales, and the expansion of
// such weights.
#include "elements.h"
#include "launchers.h"

namespace gtk {

constexpr int kWaves = 4;

__device__ __forceinline__ float nibble_value(uint32_t c, int format) {
  if (format == 0) return (float)((int)(c << 28) >> 28);
  const uint32_t m = c & 7u;
  const float v = m < 2 ? 0.5f * m : __uint_as_float(((m >> 1) + 126u) << 23 | (m & 1u) << 22);
  return c & 8u ? -v : v;
}

__device__ __forceinline__ float x_value(const void* x, int64_t i, int dtype) {
  return dtype == DT_E4M3 ? e4m3_bits_to_f32(reinterpret_cast<const uint8_t*>(x)[i]) : load_any(x, i, dtype);
}

// one wave per output: group sums in fp32, then the scale
__global__ __launch_bounds__(64 * kWaves) void w4_matmul_kernel(gt::W4Args a) {
  const int lane = threadIdx.x & 63;
  const int64_t n = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  if (n >= a.w.N) return;
  const uint8_t* q = a.w.q + n * a.w.ldq;
  for (int64_t m = blockIdx.y; m < a.M; m += gridDim.y) {
    float acc = 0;
    for (int64_t k0 = 0; k0 < a.w.K; k0 += a.w.group) {
      const int64_t k = k0 + 2 * lane;
      float t = 0;
      if (2 * lane < a.w.group && k < a.w.K) {
        const uint32_t b = q[k >> 1];
        t = x_value(a.x, m * a.ldx + k, a.x_dtype) * nibble_value(b & 15u, a.w.format);
        if (k + 1 < a.w.K) t += x_value(a.x, m * a.ldx + k + 1, a.x_dtype) * nibble_value(b >> 4, a.w.format);
      }
      for (int o = 32; o; o >>= 1) t += __shfl_xor(t, o);
      acc += load_any(a.w.scales, n * a.w.lds_n + (k0 / a.w.group) * a.w.lds_g, a.w.scale_dtype) * t;
    }
    if (lane == 0) {
      const float rs = a.row_scale ? a.row_scale[m] : 1.f;
      store_out(a.y, m * a.ldy + n, acc * a.x_scale * rs, a.out_dtype);
    }
  }
}

__global__ __launch_bounds__(256) void w4_expand_kernel(gt::W4ExpandArgs a) {
  for (int64_t n = blockIdx.y; n < a.w.N; n += gridDim.y)
    for (int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x; k < a.w.K; k += (int64_t)gridDim.x * 256) {
      const uint32_t b = a.w.q[n * a.w.ldq + (k >> 1)];
      const float s = load_any(a.w.scales, n * a.w.lds_n + (k / a.w.group) * a.w.lds_g, a.w.scale_dtype);
      store_out(a.y, n * a.ldy + k, s * nibble_value(k & 1 ? b >> 4 : b & 15u, a.w.format), a.out_dtype);
    }
}

}  // namespace gtk

namespace gt {

int launch_w4_matmul(const W4Args& a) {
  const int64_t bx = (a.w.N + gtk::kWaves - 1) / gtk::kWaves;
  if (bx > 0x7fffffff) return LS_UNSUPPORTED;
  const dim3 g((unsigned)bx, (unsigned)(a.M < 65535 ? a.M : 65535));
  hipLaunchKernelGGL(gtk::w4_matmul_kernel, g, dim3(64 * gtk::kWaves), 0, a.stream, a);
  return hipGetLastError() == hipSuccess ? LS_OK : LS_HIP_ERROR;
}

int launch_w4_expand(const W4ExpandArgs& a) {
  const int64_t bx = (a.w.K + 255) / 256;
  const dim3 g((unsigned)(bx < 1024 ? bx : 1024), (unsigned)(a.w.N < 65535 ? a.w.N : 65535));
  hipLaunchKernelGGL(gtk::w4_expand_kernel, g, dim3(256), 0, a.stream, a);
  return hipGetLastError() == hipSuccess ? LS_OK : LS_HIP_ERROR;
}

}  // namespace gt
