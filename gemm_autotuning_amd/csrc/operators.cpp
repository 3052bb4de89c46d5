// operators.cpp -- the entry points of the operators around the product
// (include/gemm_tune.h): argument checks, workspaces and launches of the RMS
// norm, its backward pass, and the product and expansion of 4-bit weights.
#include <math.h>

#include <new>
#include <string>

#include "context.h"

namespace gt {
namespace {

// One failed check: the message for gt_last_error and the status to return.
gt_status refuse(gt_status st, const std::string& msg) {
  set_error(msg);
  return st;
}
gt_status invalid(const std::string& msg) { return refuse(GT_ERR_INVALID_ARG, msg); }

// A type of the 16- or 32-bit floating ones; `dflt` replaces a negative code.
gt_status float_type(int code, int dflt, const char* what, int* out) {
  const int t = code < 0 ? dflt : code;
  if (t < 0 || t > DT_E4M3) return invalid(std::string("unknown type of ") + what);
  if (t == DT_E4M3) return refuse(GT_ERR_UNSUPPORTED, std::string("e4m3 is not provided for ") + what);
  *out = t;
  return GT_OK;
}

gt_status leading(int64_t ld, int64_t row, const char* what, int64_t* out) {
  *out = ld > 0 ? ld : row;
  if (*out < row) return invalid(std::string(what) + ": leading dimension smaller than the row");
  return GT_OK;
}

// A matrix of `rows` rows must be addressable in 64-bit byte offsets, and
// its base aligned to its element.
gt_status operand(const void* p, bool required, int64_t rows, int64_t ld, int bytes, const char* what) {
  if (!p) return required ? invalid(std::string(what) + " is NULL") : GT_OK;
  if ((uintptr_t)p % bytes) return invalid(std::string(what) + " is not aligned to its element");
  if (rows > 0 && ld > INT64_MAX / 8 / rows) return invalid(std::string(what) + " spans more than 64-bit offsets");
  return GT_OK;
}

#define GT_CHECK(expr)                 \
  do {                                 \
    const gt_status _s = (expr);       \
    if (_s != GT_OK) return _s;        \
  } while (0)

hipStream_t stream_of(void* s) { return (hipStream_t)(s ? s : ctx().default_stream.load()); }

gt_status launched(int rc, const char* what) {
  if (rc == LS_OK) return GT_OK;
  if (rc == LS_UNSUPPORTED) return refuse(GT_ERR_UNSUPPORTED, std::string(what) + ": problem too large for the grid");
  return refuse(GT_ERR_HIP, std::string(what) + ": kernel launch failed");
}

// The stream's workspace for an operator.  Growing it allocates and clears
// memory, which a captured graph must not hold, so that is refused.
gt_status operator_workspace(DeviceState& d, hipStream_t stream, size_t bytes, void** ws, std::mutex** mu) {
  size_t have = 0;
  if (!d.fake) {
    if (find_workspace(d, (void*)stream, bytes, ws, &have, mu)) return GT_OK;
    hipStreamCaptureStatus cs = hipStreamCaptureStatusNone;
    const bool asked = hipStreamIsCapturing(stream, &cs) == hipSuccess;
    if (!asked) hipGetLastError();  // the status says it; no later check should find it
    if ((!asked || cs != hipStreamCaptureStatusNone) && !workspace_ready(d, (void*)stream, bytes))
      return invalid("the workspace would have to grow under stream capture: make this call once before capturing");
  }
  return get_workspace(d, (void*)stream, bytes, ws, &have, mu);
}

constexpr int64_t kNormMaxN = 65536;

gt_status rmsnorm(const gt_rmsnorm_desc* d) {
  if (!d) return invalid("desc is NULL");
  NormArgs a;
  if (d->M < 0 || d->N < 0) return invalid("negative dimension");
  if (d->quant < GT_QUANT_NONE || d->quant > GT_QUANT_ROW) return invalid("unknown gt_quant");
  GT_CHECK(float_type(d->in_dtype, -1, "x", &a.in_dtype));
  GT_CHECK(float_type(d->weight_dtype, a.in_dtype, "weight", &a.w_dtype));
  const bool quant = d->quant != GT_QUANT_NONE;
  a.out_dtype = d->out_dtype < 0 ? (quant ? (int)DT_E4M3 : a.in_dtype) : d->out_dtype;
  if (a.out_dtype > DT_E4M3) return invalid("unknown type of y");
  if (quant != (a.out_dtype == DT_E4M3)) return invalid("e4m3 output and a gt_quant go together");
  if (!(d->eps >= 0) || !isfinite(d->eps)) return invalid("eps must be finite and not negative");
  if (!isfinite(d->weight_offset)) return invalid("weight_offset must be finite");
  if (d->quant == GT_QUANT_TENSOR && !(d->scale > 0 && isfinite(d->scale)))
    return invalid("scale must be finite and positive");
  if (d->N > kNormMaxN) return refuse(GT_ERR_UNSUPPORTED, "gt_rmsnorm takes rows of at most 65536 elements");
  GT_CHECK(leading(d->ldx, d->N, "x", &a.ldx));
  GT_CHECK(leading(d->ldr, d->N, "residual", &a.ldr));
  GT_CHECK(leading(d->lds, d->N, "sum_out", &a.lds));
  GT_CHECK(leading(d->ldy, d->N, "y", &a.ldy));
  if (d->M == 0 || d->N == 0) return GT_OK;
  const int e = elem_bytes(a.in_dtype);
  GT_CHECK(operand(d->x, true, d->M, a.ldx, e, "x"));
  GT_CHECK(operand(d->residual, false, d->M, a.ldr, e, "residual"));
  GT_CHECK(operand(d->weight, false, 1, d->N, elem_bytes(a.w_dtype), "weight"));
  GT_CHECK(operand(d->sum_out, false, d->M, a.lds, e, "sum_out"));
  GT_CHECK(operand(d->y, true, d->M, a.ldy, elem_bytes(a.out_dtype), "y"));
  GT_CHECK(operand(d->rstd, false, d->M, 1, 4, "rstd"));
  GT_CHECK(operand(d->row_scale, d->quant == GT_QUANT_ROW, d->M, 1, 4, "row_scale"));
  a.x = d->x;
  a.r = d->residual;
  a.w = d->weight;
  a.sum = d->sum_out;
  a.y = d->y;
  a.rstd = d->rstd;
  a.row_scale = d->quant == GT_QUANT_ROW ? d->row_scale : nullptr;
  a.M = d->M;
  a.N = d->N;
  a.eps = d->eps;
  a.offset = d->weight_offset;
  a.scale = d->scale;
  a.stream = stream_of(d->stream);
  DeviceState* dev = nullptr;
  GT_CHECK(current_device(&dev));
  a.cus = dev->cus;
  if (dev->fake) return GT_OK;
  return launched(launch_rmsnorm(a), "gt_rmsnorm");
}

gt_status rmsnorm_backward(const gt_rmsnorm_bwd_desc* d) {
  if (!d) return invalid("desc is NULL");
  NormBwdArgs a;
  if (d->M < 0 || d->N < 0) return invalid("negative dimension");
  GT_CHECK(float_type(d->in_dtype, -1, "h", &a.in_dtype));
  GT_CHECK(float_type(d->dy_dtype, a.in_dtype, "dy", &a.dy_dtype));
  if (a.dy_dtype != a.in_dtype && a.dy_dtype != DT_F32)
    return refuse(GT_ERR_UNSUPPORTED, "dy is of h's type or f32");
  GT_CHECK(float_type(d->weight_dtype, a.in_dtype, "weight", &a.w_dtype));
  GT_CHECK(float_type(d->dweight_dtype, DT_F32, "dweight", &a.dw_dtype));
  if (!isfinite(d->weight_offset)) return invalid("weight_offset must be finite");
  if (d->N > kNormMaxN) return refuse(GT_ERR_UNSUPPORTED, "gt_rmsnorm_backward takes rows of at most 65536 elements");
  GT_CHECK(leading(d->lddy, d->N, "dy", &a.lddy));
  GT_CHECK(leading(d->ldh, d->N, "h", &a.ldh));
  GT_CHECK(leading(d->ldds, d->N, "dsum", &a.ldds));
  GT_CHECK(leading(d->lddx, d->N, "dx", &a.lddx));
  if (!d->dx && !d->dweight) return invalid("neither dx nor dweight is wanted");
  if (d->N == 0) return GT_OK;
  const int e = elem_bytes(a.in_dtype);
  const bool rows = d->M > 0;
  GT_CHECK(operand(d->dy, rows, d->M, a.lddy, elem_bytes(a.dy_dtype), "dy"));
  GT_CHECK(operand(d->h, rows, d->M, a.ldh, e, "h"));
  GT_CHECK(operand(d->weight, false, 1, d->N, elem_bytes(a.w_dtype), "weight"));
  GT_CHECK(operand(d->rstd, rows, d->M, 1, 4, "rstd"));
  GT_CHECK(operand(d->dsum, false, d->M, a.ldds, e, "dsum"));
  GT_CHECK(operand(d->dx, false, d->M, a.lddx, e, "dx"));
  GT_CHECK(operand(d->dweight, false, 1, d->N, elem_bytes(a.dw_dtype), "dweight"));
  a.dy = d->dy;
  a.h = d->h;
  a.w = d->weight;
  a.rstd = d->rstd;
  a.dsum = d->dsum;
  a.dx = d->dx;
  a.dw = d->dweight;
  a.M = d->M;
  a.N = d->N;
  a.offset = d->weight_offset;
  a.ws = nullptr;
  a.stream = stream_of(d->stream);
  DeviceState* dev = nullptr;
  GT_CHECK(current_device(&dev));
  a.cus = dev->cus;
  if (dev->fake) return GT_OK;
  if (!rows) {
    if (!a.dw) return GT_OK;
    return launched(launch_zero(a.dw, 1, a.N, a.N, a.dw_dtype, a.stream), "gt_rmsnorm_backward");
  }
  const size_t need = rmsnorm_bwd_workspace_bytes(a);
  if (need == 0) return launched(launch_rmsnorm_bwd(a), "gt_rmsnorm_backward");
  void* ws = nullptr;
  std::mutex* mu = nullptr;
  GT_CHECK(operator_workspace(*dev, a.stream, kCounterRegion + need, &ws, &mu));
  a.ws = reinterpret_cast<float*>(static_cast<char*>(ws) + kCounterRegion);
  std::lock_guard<std::mutex> g(*mu);
  return launched(launch_rmsnorm_bwd(a), "gt_rmsnorm_backward");
}

// The 4-bit weights of a descriptor (D: gt_w4_desc or gt_w4_expand_desc).
template <class D>
gt_status weights(const D* d, W4Weights* w) {
  if (d->N < 0 || d->K < 0) return invalid("negative dimension");
  if (d->format != GT_W4_INT4 && d->format != GT_W4_E2M1) return invalid("unknown gt_w4_format");
  if (d->group != 32 && d->group != 64 && d->group != 128) return invalid("group must be 32, 64 or 128");
  GT_CHECK(float_type(d->scale_dtype, -1, "scales", &w->scale_dtype));
  const int64_t groups = d->K / d->group + (d->K % d->group != 0);
  GT_CHECK(leading(d->ldq, d->K / 2 + d->K % 2, "qweight", &w->ldq));
  w->lds_n = d->scale_ldn > 0 ? d->scale_ldn : (groups > 0 ? groups : 1);
  w->lds_g = d->scale_ldg > 0 ? d->scale_ldg : 1;
  w->q = static_cast<const uint8_t*>(d->qweight);
  w->scales = d->scales;
  w->N = d->N;
  w->K = d->K;
  w->format = d->format;
  w->group = d->group;
  if (d->N == 0 || d->K == 0) return GT_OK;
  GT_CHECK(operand(d->qweight, true, d->N, w->ldq, 1, "qweight"));
  GT_CHECK(operand(d->scales, true, d->N, w->lds_n, elem_bytes(w->scale_dtype), "scales"));
  return operand(d->scales, true, groups, w->lds_g, 1, "scales");
}

gt_status w4_matmul(const gt_w4_desc* d) {
  if (!d) return invalid("desc is NULL");
  W4Args a;
  if (d->M < 0) return invalid("negative dimension");
  if (d->x_dtype < 0 || d->x_dtype > DT_E4M3) return invalid("unknown type of x");
  if (d->x_dtype == DT_F32) return refuse(GT_ERR_UNSUPPORTED, "rows of gt_w4_matmul are f16, bf16 or e4m3");
  a.x_dtype = d->x_dtype;
  GT_CHECK(float_type(d->out_dtype, a.x_dtype == DT_E4M3 ? (int)DT_F32 : a.x_dtype, "y", &a.out_dtype));
  GT_CHECK(weights(d, &a.w));
  if (!isfinite(d->x_scale)) return invalid("x_scale must be finite");
  GT_CHECK(leading(d->ldx, d->K, "x", &a.ldx));
  GT_CHECK(leading(d->ldy, d->N, "y", &a.ldy));
  if (d->M == 0 || d->N == 0) return GT_OK;
  GT_CHECK(operand(d->y, true, d->M, a.ldy, elem_bytes(a.out_dtype), "y"));
  GT_CHECK(operand(d->x, d->K > 0, d->M, a.ldx, elem_bytes(a.x_dtype), "x"));
  GT_CHECK(operand(d->row_scale, false, d->M, 1, 4, "row_scale"));
  a.x = d->x;
  a.row_scale = d->row_scale;
  a.y = d->y;
  a.M = d->M;
  a.x_scale = d->x_scale;
  a.stream = stream_of(d->stream);
  DeviceState* dev = nullptr;
  GT_CHECK(current_device(&dev));
  if (dev->fake) return GT_OK;
  if (d->K == 0) return launched(launch_zero(a.y, a.M, a.w.N, a.ldy, a.out_dtype, a.stream), "gt_w4_matmul");
  const size_t need = w4_workspace_bytes(a, dev->cus);
  if (need == 0) return launched(launch_w4_matmul(a, nullptr, dev->cus), "gt_w4_matmul");
  void* ws = nullptr;
  std::mutex* mu = nullptr;
  GT_CHECK(operator_workspace(*dev, a.stream, need, &ws, &mu));
  std::lock_guard<std::mutex> g(*mu);
  return launched(launch_w4_matmul(a, ws, dev->cus), "gt_w4_matmul");
}

gt_status w4_expand(const gt_w4_expand_desc* d) {
  if (!d) return invalid("desc is NULL");
  W4ExpandArgs a;
  GT_CHECK(float_type(d->out_dtype, -1, "out", &a.out_dtype));
  GT_CHECK(weights(d, &a.w));
  GT_CHECK(leading(d->ldo, d->K, "out", &a.ldy));
  if (d->N == 0 || d->K == 0) return GT_OK;
  GT_CHECK(operand(d->out, true, d->N, a.ldy, elem_bytes(a.out_dtype), "out"));
  a.y = d->out;
  a.stream = stream_of(d->stream);
  DeviceState* dev = nullptr;
  GT_CHECK(current_device(&dev));
  if (dev->fake) return GT_OK;
  return launched(launch_w4_expand(a, dev->cus), "gt_w4_expand");
}

// Nothing throws across the C boundary: an allocation that fails while a
// message or a workspace entry is made becomes a status.
template <class F, class D>
gt_status guarded(F f, const D* d) {
  try {
    return f(d);
  } catch (const std::bad_alloc&) {
    return GT_ERR_OOM;
  } catch (...) {
    return GT_ERR_HIP;
  }
}

}  // namespace
}  // namespace gt

using namespace gt;

extern "C" {

gt_status gt_rmsnorm(const gt_rmsnorm_desc* d) { return guarded(rmsnorm, d); }
gt_status gt_rmsnorm_backward(const gt_rmsnorm_bwd_desc* d) { return guarded(rmsnorm_backward, d); }
gt_status gt_w4_matmul(const gt_w4_desc* d) { return guarded(w4_matmul, d); }
gt_status gt_w4_expand(const gt_w4_expand_desc* d) { return guarded(w4_expand, d); }

}  // extern "C"
