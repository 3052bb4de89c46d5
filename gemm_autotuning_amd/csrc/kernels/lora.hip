// lora.hip -- adapters of many requests beside a shared projection.
#include "elements.h"
#include "launchers.h"

namespace gtk {

__device__ __forceinline__ float wave_sum(float v) {
  return __uint_as_float(wave_join(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

__global__ __launch_bounds__(256) void lora_shrink_kernel(gt::LoraArgs a, float* mid) {
  const int lane = threadIdx.x & 63, r = blockIdx.y * 4 + (threadIdx.x >> 6);
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    const int e = a.index[m];
    if (r >= a.rank || e < 0 || e >= a.adapters) continue;
    const char* row = a.a.p + e * a.a.stride + r * a.a.ld;
    float v = 0.f;
    for (int64_t k = lane; k < a.K; k += 64) v += load_any(a.x, m * a.ldx + k, a.x_dtype) * load_any(row, k, a.x_dtype);
    v = wave_sum(v);
    if (lane == 0) mid[m * a.rank + r] = v;
  }
}

__global__ __launch_bounds__(256) void lora_expand_kernel(gt::LoraArgs a, const float* mid) {
  for (int64_t m = blockIdx.y; m < a.M; m += gridDim.y) {
    const int e = a.index[m];
    const bool some = e >= 0 && e < a.adapters;
    if (!some && a.base == a.y) continue;
    for (int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x; n < a.N; n += (int64_t)gridDim.x * 256) {
      float v = 0.f;
      if (some) {
        const char* row = a.b.p + e * a.b.stride + n * a.b.ld;
        for (int r = 0; r < a.rank; ++r) v += mid[m * a.rank + r] * load_any(row, r, a.x_dtype);
        v *= a.scale ? a.scale[e] : 1.f;
      }
      if (a.base) v += load_any(a.base, m * a.ldb + n, a.out_dtype);
      store_out(a.y, m * a.ldy + n, v, a.out_dtype);
    }
  }
}

__global__ __launch_bounds__(256) void copy_rows_kernel(const void* base, void* y, int64_t M, int64_t N, int64_t ldb, int64_t ldy,
                                                        int dtype) {
  for (int64_t m = blockIdx.y; m < M; m += gridDim.y)
    for (int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x; n < N; n += (int64_t)gridDim.x * 256)
      store_out(y, m * ldy + n, base ? load_any(base, m * ldb + n, dtype) : 0.f, dtype);
}

}  // namespace gtk

namespace gt {

int64_t lora_range(const LoraArgs& a) {
  const int64_t rows = ((int64_t)64 << 20) / (4 * a.rank);
  return rows;
}
size_t lora_workspace_bytes(const LoraArgs& a, int64_t rows) { return (size_t)(rows * a.rank * 4); }

static unsigned at_most(int64_t n, int64_t most) { return (unsigned)(n < most ? n : most); }

int launch_lora(const LoraArgs& a) {
  float* mid = reinterpret_cast<float*>(a.ws);
  hipLaunchKernelGGL(gtk::lora_shrink_kernel, dim3(at_most(a.M, 65536), (a.rank + 3) / 4), dim3(256), 0, a.stream, a, mid);
  hipLaunchKernelGGL(gtk::lora_expand_kernel, dim3(at_most((a.N + 255) / 256, 1024), at_most(a.M, 32768)), dim3(256), 0, a.stream, a,
                     mid);
  return hipGetLastError() == hipSuccess ? LS_OK : LS_HIP_ERROR;
}

int launch_copy_rows(const void* base, void* y, int64_t M, int64_t N, int64_t ldb, int64_t ldy, int dtype, hipStream_t stream) {
  if (base == y) return LS_OK;
  hipLaunchKernelGGL(gtk::copy_rows_kernel, dim3(at_most((N + 255) / 256, 1024), at_most(M, 32768)), dim3(256), 0, stream, base, y, M,
                     N, ldb, ldy, dtype);
  return hipGetLastError() == hipSuccess ? LS_OK : LS_HIP_ERROR;
}

}  // namespace gt
