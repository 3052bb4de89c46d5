// The entry points of the experts' choice, layer and adapters under
// sanitizers, on the stand-in device (their checks, workspaces and ranges;
// nothing is launched): eight threads at once, each call taken or refused as
// it should be, each thread's last error its own.
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

static gt_route_desc choice(int64_t M, int64_t E, int64_t k) {
  gt_route_desc d;
  memset(&d, 0, sizeof(d));
  d.logits = P;
  d.index = (int32_t*)P;
  d.weight = (float*)P;
  d.M = M;
  d.E = E;
  d.topk = k;
  d.dtype = GT_F32;
  d.scale = 1.0f;
  return d;
}
static gt_moe_desc layer(int64_t M, int64_t K, int64_t H, int64_t E, int64_t k, int format) {
  gt_moe_desc d;
  memset(&d, 0, sizeof(d));
  d.x = d.gate_up = d.gate_up_scales = d.down = d.down_scales = P;
  d.index = (const int32_t*)P;
  d.weight = (const float*)P;
  d.y = P;
  d.M = M;
  d.K = K;
  d.H = H;
  d.E = E;
  d.topk = k;
  d.x_dtype = GT_BF16;
  d.out_dtype = -1;
  d.format = format;
  d.group = 64;
  return d;
}
static gt_lora_desc adapters(int64_t M, int64_t K, int64_t N, int64_t rank) {
  gt_lora_desc d;
  memset(&d, 0, sizeof(d));
  d.x = d.a = d.b = P;
  d.index = (const int32_t*)P;
  d.y = (char*)P + 4096;
  d.M = M;
  d.K = K;
  d.N = N;
  d.adapters = 5;
  d.rank = rank;
  d.x_dtype = GT_F16;
  d.out_dtype = -1;
  return d;
}

int main() {
  const double t = 1e-3;
  CHECK(gt_test_fake_device(1, GT_F32, &t, 1) == GT_OK);
  const int64_t far = INT64_MAX, most = INT64_C(1) << 24;
  std::vector<std::thread> pool;
  for (int i = 0; i < 8; ++i)
    pool.emplace_back([=] {
      for (int it = 0; it < 200; ++it) {
        gt_route_desc r = choice(i * it, 8 + i, 1 + i);
        CHECK(gt_route(&r) == GT_OK);
        r.scale = NAN;
        CHECK(gt_route(&r) == GT_ERR_INVALID_ARG && strstr(gt_last_error(), "scale"));
        r = choice(far, 8, 2);
        CHECK(gt_route(&r) == GT_ERR_INVALID_ARG);
        r = choice(3, far, 2);
        CHECK(gt_route(&r) == GT_ERR_UNSUPPORTED);
        for (int f = -1; f <= 1; ++f) {
          int64_t bytes = -1, own = -1;
          gt_moe_desc m = layer(1 + it * it, 1 + 37 * i, 1 + 53 * it, 1 + i, 1 + it % 64, f);
          CHECK(gt_moe_workspace(&m, &bytes) == GT_OK && bytes > 0);
          CHECK(gt_moe(&m) == GT_OK);
          m.workspace = P;
          m.workspace_bytes = bytes;
          CHECK(gt_moe(&m) == GT_OK);
          m.workspace_bytes = bytes - 1;
          CHECK(gt_moe(&m) == GT_ERR_INVALID_ARG && strstr(gt_last_error(), "workspace"));
          // the longest rows, the most tokens
          m = layer(it ? 1 + it : INT64_C(1) << 30, most, most, 2, 64, f);
          m.gate_up_stride = m.down_stride = INT64_C(1) << 50;
          CHECK(gt_moe_workspace(&m, &own) == GT_OK && own > 0);
          m = layer(1, 64, 64, 4096, 64, f);
          m.down_stride = far;
          CHECK(gt_moe(&m) == GT_ERR_INVALID_ARG);
          m = layer(1, far, 64, 2, 1, f);
          CHECK(gt_moe(&m) == GT_ERR_UNSUPPORTED);
          m = layer(far, 64, 64, 2, 1, f);
          CHECK(gt_moe(&m) == GT_ERR_INVALID_ARG);
        }
        int64_t bytes = -1;
        gt_lora_desc l = adapters(1 + it * it, 1 + 41 * it, 1 + 29 * i, 1 + it);
        CHECK(gt_lora_workspace(&l, &bytes) == GT_OK && bytes > 0);
        CHECK(gt_lora(&l) == GT_OK);
        l.workspace = P;
        l.workspace_bytes = bytes - 1;
        CHECK(gt_lora(&l) == GT_ERR_INVALID_ARG && strstr(gt_last_error(), "workspace"));
        l = adapters(INT64_C(1) << 30, most, most, 256);
        CHECK(gt_lora_workspace(&l, &bytes) == GT_OK && bytes > 0);
        l = adapters(2, 64, 64, 16);
        l.b_stride = l.a_ld = far;
        CHECK(gt_lora(&l) == GT_ERR_INVALID_ARG);
      }
    });
  for (std::thread& th : pool) th.join();
  CHECK(gt_test_fake_device(0, GT_F32, nullptr, 0) == GT_OK);
  if (g_fail) return 1;
  printf("experts under sanitizer ok\n");
  return 0;
}
