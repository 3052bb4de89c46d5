// The operators' entry points under sanitizers, on the stand-in device (their
// checks and descriptors; nothing is launched): eight threads at once, each
// call taken or refused as it should be, each thread's last error its own,
// the default stream set meanwhile.
#include <math.h>
#include <stdio.h>
#include <string.h>

#include <atomic>
#include <thread>
#include <vector>

#include "gemm_tune.h"
#include "gemm_tune_testing.h"

static std::atomic<int> g_fail{0};

#define CHECK(cond)                                                      \
  do {                                                                   \
    if (!(cond)) {                                                       \
      fprintf(stderr, "check failed at line %d: %s\n", __LINE__, #cond); \
      g_fail++;                                                          \
    }                                                                    \
  } while (0)

static void* const P = (void*)0x10000;

static gt_rmsnorm_desc norm(int64_t M, int64_t N) {
  gt_rmsnorm_desc d;
  memset(&d, 0, sizeof(d));
  d.x = d.weight = P;
  d.y = P;
  d.M = M;
  d.N = N;
  d.in_dtype = GT_BF16;
  d.weight_dtype = d.out_dtype = -1;
  d.eps = 1e-6f;
  return d;
}
static gt_rmsnorm_bwd_desc backward(int64_t M, int64_t N) {
  gt_rmsnorm_bwd_desc d;
  memset(&d, 0, sizeof(d));
  d.dy = d.h = P;
  d.rstd = (const float*)P;
  d.dx = d.dweight = P;
  d.M = M;
  d.N = N;
  d.in_dtype = GT_F16;
  d.dy_dtype = d.weight_dtype = d.dweight_dtype = -1;
  return d;
}
static gt_w4_desc product(int64_t M, int64_t N, int64_t K) {
  gt_w4_desc d;
  memset(&d, 0, sizeof(d));
  d.x = d.qweight = d.scales = P;
  d.y = P;
  d.M = M;
  d.N = N;
  d.K = K;
  d.x_dtype = GT_BF16;
  d.out_dtype = -1;
  d.group = 128;
  d.x_scale = 1.0f;
  return d;
}
static gt_w4_expand_desc expand(int64_t N, int64_t K) {
  gt_w4_expand_desc d;
  memset(&d, 0, sizeof(d));
  d.qweight = d.scales = P;
  d.out = P;
  d.N = N;
  d.K = K;
  d.out_dtype = GT_F16;
  d.group = 32;
  return d;
}

int main() {
  const double t = 1e-3;
  CHECK(gt_test_fake_device(1, GT_F32, &t, 1) == GT_OK);
  const int64_t far = INT64_MAX;
  std::vector<std::thread> pool;
  for (int i = 0; i < 8; ++i)
    pool.emplace_back([=] {
      for (int it = 0; it < 200; ++it) {
        CHECK(gt_set_stream((void*)(uintptr_t)(64 * (i + 1))) == GT_OK);
        gt_rmsnorm_desc n = norm(i * it, 1 + it);
        CHECK(gt_rmsnorm(&n) == GT_OK);
        n.eps = NAN;
        CHECK(gt_rmsnorm(&n) == GT_ERR_INVALID_ARG && strstr(gt_last_error(), "eps"));
        n = norm(far, 65536);
        CHECK(gt_rmsnorm(&n) == GT_ERR_INVALID_ARG && strstr(gt_last_error(), "64-bit"));
        n = norm(3, far);
        CHECK(gt_rmsnorm(&n) == GT_ERR_UNSUPPORTED);
        gt_rmsnorm_bwd_desc b = backward(1 + it, 1 + i);
        CHECK(gt_rmsnorm_backward(&b) == GT_OK);
        b.dx = b.dweight = nullptr;
        CHECK(gt_rmsnorm_backward(&b) == GT_ERR_INVALID_ARG && strstr(gt_last_error(), "neither"));
        b = backward(2, 8);
        b.ldh = far;
        CHECK(gt_rmsnorm_backward(&b) == GT_ERR_INVALID_ARG);
        gt_w4_desc w = product(1 + i, 1 + it, 1 + 37 * it);
        CHECK(gt_w4_matmul(&w) == GT_OK);
        w.group = 48;
        CHECK(gt_w4_matmul(&w) == GT_ERR_INVALID_ARG && strstr(gt_last_error(), "group"));
        w = product(1, far, far);
        CHECK(gt_w4_matmul(&w) == GT_ERR_INVALID_ARG);
        w = product(1, 2, 64);
        w.scale_ldn = w.scale_ldg = far;
        CHECK(gt_w4_matmul(&w) == GT_ERR_INVALID_ARG);
        gt_w4_expand_desc e = expand(1 + it, 1 + i);
        CHECK(gt_w4_expand(&e) == GT_OK);
        e.ldo = 1;
        e.K = 64;
        CHECK(gt_w4_expand(&e) == GT_ERR_INVALID_ARG && strstr(gt_last_error(), "out"));
        e = expand(far, 1);
        CHECK(gt_w4_expand(&e) == GT_ERR_INVALID_ARG);
      }
    });
  for (std::thread& th : pool) th.join();
  CHECK(gt_test_fake_device(0, GT_F32, nullptr, 0) == GT_OK);
  if (g_fail) return 1;
  printf("operators under sanitizer ok\n");
  return 0;
}
