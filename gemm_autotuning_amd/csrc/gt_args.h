// gt_args.h -- the problem as handed from the host library to a kernel launcher.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gt {

enum DType { DT_F32 = 0, DT_F16 = 1, DT_BF16 = 2, DT_E4M3 = 3 };

inline int elem_bytes(int d) { return d == DT_F32 ? 4 : (d == DT_E4M3 ? 1 : 2); }

// A normalised problem: C (M x N, ldc) = op(A) * op(B).  ta: A is stored
// K x M (else M x K); tb: B is stored N x K (else K x N).  Leading dimensions
// are resolved (never <= 0).  sa * sb scale fp8 products (1 otherwise).
struct Problem {
  const void* A;
  const void* B;
  void* C;
  int64_t M, N, K, lda, ldb, ldc;
  int layout;  // gt_layout: bit 1 = lhs transposed, bit 0 = rhs transposed
  bool ta, tb;
  int in_dtype, out_dtype;
  float sa, sb;
  hipStream_t stream;
};

// What a launcher gets: the problem, the split count chosen for split-K
// candidates, and the workspace (device memory of at least ws_bytes).
struct LaunchArgs {
  Problem p;
  int splitk;
  void* ws;
  size_t ws_bytes;
};

// RMS norm of M rows of N elements (rmsnorm.hip): h = x + r, rstd =
// 1/sqrt(mean h^2 + eps), y = h * rstd * (w + offset).  r, w, sum, rstd and
// row_scale may be null.
struct NormArgs {
  const void* x;
  const void* r;
  const void* w;
  void* sum;
  void* y;
  float* rstd;
  float* row_scale;
  int64_t M, N, ldx, ldr, lds, ldy;
  int in_dtype, w_dtype, out_dtype;
  float eps, offset, scale;
  float near;  // set by the launcher: the power of two that brings scale nearer to 1
  int cus;
  bool past_caches;  // set by the launcher: more than the last-level cache passes by
  hipStream_t stream;
};

// Its backward pass: dx (may be null) and dw (may be null).  ws: blocks x N
// fp32 partial sums of dw when dw is wanted.
struct NormBwdArgs {
  const void* dy;
  const void* h;
  const void* w;
  const float* rstd;
  const void* dsum;
  void* dx;
  void* dw;
  int64_t M, N, lddy, ldh, ldds, lddx;
  int in_dtype, dy_dtype, w_dtype, dw_dtype;
  float offset;
  float* ws;
  int cus;
  int dw_blocks;  // set by the launcher: workgroups that take columns of dw
  bool past_caches;
  hipStream_t stream;
};

// Rows times 4-bit weights (w4.hip), and the expansion of such weights.
struct W4Weights {
  const uint8_t* q;    // N rows of (K + 1) / 2 bytes, ldq bytes apart
  const void* scales;  // (n, g) at n * lds_n + g * lds_g
  int64_t N, K, ldq, lds_n, lds_g;
  int format, scale_dtype, group;
};
struct W4Args {
  W4Weights w;
  const void* x;
  const float* row_scale;
  void* y;
  int64_t M, ldx, ldy;
  int x_dtype, out_dtype;
  float x_scale;
  hipStream_t stream;
};
struct W4ExpandArgs {
  W4Weights w;
  void* y;
  int64_t ldy;
  int out_dtype;
  bool past_caches;
  hipStream_t stream;
};

// Launcher status codes (0 = launched).
enum LaunchStatus { LS_OK = 0, LS_UNSUPPORTED = 1, LS_HIP_ERROR = 2 };

}  // namespace gt
