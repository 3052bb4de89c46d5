// rmsnorm.hip -- the RMS norm with the residual's addition, and its backward
// pass.
#include "elements.h"
#include "launchers.h"

namespace gtk {

constexpr int kNT = 256;

__device__ __forceinline__ float block_sum(float v, float* part) {
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0;
  for (int i = 0; i < kNT / 64; ++i) v += part[i];
  return v;
}
// largest |v| by the bits below the sign: NaN above infinity above the finite
__device__ __forceinline__ float block_amax(float v, float* part) {
  uint32_t b = __float_as_uint(v) & 0x7fffffffu;
  for (int o = 32; o; o >>= 1) b = max(b, (uint32_t)__shfl_xor((int)b, o));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = __uint_as_float(b);
  __syncthreads();
  b = 0;
  for (int i = 0; i < kNT / 64; ++i) b = max(b, __float_as_uint(part[i]));
  return __uint_as_float(b);
}

template <int IN, int OUT>
__global__ __launch_bounds__(kNT) void rmsnorm_kernel(gt::NormArgs a) {
  __shared__ float part[kNT / 64];
  extern __shared__ float row[];
  typedef typename Elem<IN>::T TI;
  typedef typename Elem<OUT>::T TO;
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    const TI* x = reinterpret_cast<const TI*>(a.x) + m * a.ldx;
    const TI* r = a.r ? reinterpret_cast<const TI*>(a.r) + m * a.ldr : nullptr;
    TI* s = a.sum ? reinterpret_cast<TI*>(a.sum) + m * a.lds : nullptr;
    TO* y = reinterpret_cast<TO*>(a.y) + m * a.ldy;
    auto h_of = [&](int64_t n) { return Elem<IN>::get(x[n]) + (r ? Elem<IN>::get(r[n]) : 0.f); };
    auto w_of = [&](int64_t n) { return a.w ? load_any(a.w, n, a.w_dtype) + a.offset : 1.f; };
    float q = 0;
    for (int64_t n = threadIdx.x; n < a.N; n += kNT) {
      const float h = h_of(n);
      q += h * h;
    }
    const float rstd = 1.0f / sqrtf(block_sum(q, part) / (float)a.N + a.eps);
    float inv = 1.0f / a.scale;
    if (a.row_scale) {
      float big = 0;
      for (int64_t n = threadIdx.x; n < a.N; n += kNT) {
        const float v = h_of(n) * rstd * w_of(n);
        const uint32_t u = max(__float_as_uint(big), __float_as_uint(v) & 0x7fffffffu);
        big = __uint_as_float(u);
      }
      big = block_amax(big, part);
      const float scale = (big < 0x1p-100f ? 0x1p-100f : big) / 448.f;
      if (threadIdx.x == 0) a.row_scale[m] = scale;
      inv = 1.0f / scale;
    }
    if (threadIdx.x == 0 && a.rstd) a.rstd[m] = rstd;
    for (int64_t n = threadIdx.x; n < a.N; n += kNT) {
      const float h = h_of(n);
      float v = h * rstd * w_of(n);
      if (OUT == DT_E4M3) v *= inv;
      if (s) s[n] = Elem<IN>::put(h);
      y[n] = Elem<OUT>::put(v);
    }
  }
}

template <int IN, int DY>
__global__ __launch_bounds__(kNT) void rmsnorm_dx_kernel(gt::NormBwdArgs a) {
  __shared__ float part[kNT / 64];
  typedef typename Elem<IN>::T TI;
  typedef typename Elem<DY>::T TD;
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    const TD* dy = reinterpret_cast<const TD*>(a.dy) + m * a.lddy;
    const TI* h = reinterpret_cast<const TI*>(a.h) + m * a.ldh;
    const TI* ds = a.dsum ? reinterpret_cast<const TI*>(a.dsum) + m * a.ldds : nullptr;
    TI* dx = reinterpret_cast<TI*>(a.dx) + m * a.lddx;
    const float rstd = a.rstd[m];
    auto g_of = [&](int64_t n) {
      return Elem<DY>::get(dy[n]) * (a.w ? load_any(a.w, n, a.w_dtype) + a.offset : 1.f);
    };
    float q = 0;
    for (int64_t n = threadIdx.x; n < a.N; n += kNT) q += g_of(n) * (Elem<IN>::get(h[n]) * rstd);
    const float mean = block_sum(q, part) / (float)a.N;
    for (int64_t n = threadIdx.x; n < a.N; n += kNT) {
      const float v = rstd * (g_of(n) - Elem<IN>::get(h[n]) * rstd * mean);
      dx[n] = Elem<IN>::put(v + (ds ? Elem<IN>::get(ds[n]) : 0.f));
    }
  }
}

template <int IN, int DY>
__global__ __launch_bounds__(kNT) void rmsnorm_dw_kernel(gt::NormBwdArgs a) {
  typedef typename Elem<IN>::T TI;
  typedef typename Elem<DY>::T TD;
  const int64_t n = (int64_t)blockIdx.x * kNT + threadIdx.x;
  if (n >= a.N) return;
  float s = 0;
  for (int64_t m = 0; m < a.M; ++m)
    s += Elem<DY>::get(reinterpret_cast<const TD*>(a.dy)[m * a.lddy + n]) *
         (Elem<IN>::get(reinterpret_cast<const TI*>(a.h)[m * a.ldh + n]) * a.rstd[m]);
  store_out(a.dw, n, s, a.dw_dtype);
}

}  // namespace gtk

namespace gt {

namespace {
int rows_grid(int64_t M) { return (int)(M < 65536 ? M : 65536); }
int status() { return hipGetLastError() == hipSuccess ? LS_OK : LS_HIP_ERROR; }

template <int IN>
int norm_in(const NormArgs& a) {
  const dim3 g(rows_grid(a.M)), b(gtk::kNT);
  switch (a.out_dtype) {
    case DT_F32: hipLaunchKernelGGL((gtk::rmsnorm_kernel<IN, DT_F32>), g, b, 0, a.stream, a); break;
    case DT_F16: hipLaunchKernelGGL((gtk::rmsnorm_kernel<IN, DT_F16>), g, b, 0, a.stream, a); break;
    case DT_BF16: hipLaunchKernelGGL((gtk::rmsnorm_kernel<IN, DT_BF16>), g, b, 0, a.stream, a); break;
    default: hipLaunchKernelGGL((gtk::rmsnorm_kernel<IN, DT_E4M3>), g, b, 0, a.stream, a); break;
  }
  return status();
}

template <int IN, int DY>
int bwd_types(const NormBwdArgs& a) {
  if (a.dw) {
    const dim3 g((unsigned)((a.N + gtk::kNT - 1) / gtk::kNT));
    hipLaunchKernelGGL((gtk::rmsnorm_dw_kernel<IN, DY>), g, dim3(gtk::kNT), 0, a.stream, a);
    const int rc = status();
    if (rc != LS_OK) return rc;
  }
  if (!a.dx) return LS_OK;
  hipLaunchKernelGGL((gtk::rmsnorm_dx_kernel<IN, DY>), dim3(rows_grid(a.M)), dim3(gtk::kNT), 0, a.stream, a);
  return status();
}
}  // namespace

int launch_rmsnorm(const NormArgs& a) {
  switch (a.in_dtype) {
    case DT_F32: return norm_in<DT_F32>(a);
    case DT_F16: return norm_in<DT_F16>(a);
    default: return norm_in<DT_BF16>(a);
  }
}

size_t rmsnorm_bwd_workspace_bytes(const NormBwdArgs&) { return 0; }

int launch_rmsnorm_bwd(const NormBwdArgs& a) {
  const bool wide = a.dy_dtype == DT_F32;
  switch (a.in_dtype) {
    case DT_F32: return bwd_types<DT_F32, DT_F32>(a);
    case DT_F16: return wide ? bwd_types<DT_F16, DT_F32>(a) : bwd_types<DT_F16, DT_F16>(a);
    default: return wide ? bwd_types<DT_BF16, DT_F32>(a) : bwd_types<DT_BF16, DT_BF16>(a);
  }
}

}  // namespace gt
