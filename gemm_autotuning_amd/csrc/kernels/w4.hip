// w4.hip -- rows times 4-bit weights with group scales, and the expansion of
// such weights.
#include "elements.h"
#include "launchers.h"
#include "w4_mma.h"

namespace gtk {

__device__ __forceinline__ float nibble_value(uint32_t c, int format) {
  if (format == 0) return (float)((int)(c << 28) >> 28);
  const uint32_t m = c & 7u;
  const float v = m < 2 ? 0.5f * m : __uint_as_float(((m >> 1) + 126u) << 23 | (m & 1u) << 22);
  return c & 8u ? -v : v;
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

namespace {
constexpr int kRowBlock = 64;  // rows of one launch: four blocks of 16

struct W4Plan {
  int T, C, waves, S, tiles, tiles_per_wg, chunks;
  dim3 grid;
};

bool w4_plan(const W4Args& a, int64_t rows, int cus, W4Plan* p) {
  const int64_t chunks = (a.w.K + gtk::kW4Chunk - 1) / gtk::kW4Chunk, tiles = (a.w.N + 15) / 16;
  if (chunks > 0x7fffffff / 16 || tiles > 0x7fffffff / 2) return false;
  p->chunks = (int)chunks;
  p->tiles = (int)tiles;
  p->T = rows <= 16 ? 1 : (rows <= 32 ? 2 : 4);
  p->C = p->T == 1 ? (chunks <= gtk::kW4Waves ? 1 : 4) : 2;
  p->waves = (int)(chunks < gtk::kW4Waves ? chunks : gtk::kW4Waves);
  const int per = p->waves * p->C;
  p->S = (int)((chunks + per - 1) / per);
  int64_t wgs = 2 * (int64_t)cus / p->S;
  if (wgs < 1) wgs = 1;
  p->tiles_per_wg = (int)((tiles + wgs - 1) / wgs);
  p->grid = dim3((unsigned)((tiles + p->tiles_per_wg - 1) / p->tiles_per_wg), (unsigned)p->S, 1);
  return p->S <= 65535 && (p->S == 1 || (int)p->grid.x <= kMaxCounterBlocks);
}
}  // namespace

size_t w4_workspace_bytes(const W4Args& a, int cus) {
  W4Plan p;
  const int64_t rows = a.M < kRowBlock ? a.M : kRowBlock;
  if (!w4_plan(a, rows, cus, &p) || p.S == 1) return 0;
  return kCounterRegion + (size_t)p.S * rows * a.w.N * 4;
}

int launch_w4_matmul(const W4Args& all, void* ws, int cus) {
  for (int64_t m0 = 0; m0 < all.M; m0 += kRowBlock) {
    W4Args a = all;
    a.M = all.M - m0 < kRowBlock ? all.M - m0 : kRowBlock;
    a.x = static_cast<const char*>(all.x) + m0 * all.ldx * elem_bytes(all.x_dtype);
    a.y = static_cast<char*>(all.y) + m0 * all.ldy * elem_bytes(all.out_dtype);
    if (all.row_scale) a.row_scale = all.row_scale + m0;
    W4Plan pl;
    if (!w4_plan(a, a.M, cus, &pl)) return LS_UNSUPPORTED;
    gtk::W4Params p;
    p.a = a;
    p.counters = static_cast<unsigned*>(ws);
    p.ws = ws ? reinterpret_cast<float*>(static_cast<char*>(ws) + kCounterRegion) : nullptr;
    p.S = pl.S;
    p.waves = pl.waves;
    p.tiles = pl.tiles;
    p.tiles_per_wg = pl.tiles_per_wg;
    p.chunks = pl.chunks;
    const bool int4 = a.w.format == gtk::W4_INT4;
    int rc;
    switch (a.x_dtype) {
      case DT_BF16: rc = int4 ? w4_mma_bf16_int4(p, pl.grid, pl.T, pl.C) : w4_mma_bf16_e2m1(p, pl.grid, pl.T, pl.C); break;
      case DT_F16: rc = int4 ? w4_mma_f16_int4(p, pl.grid, pl.T, pl.C) : w4_mma_f16_e2m1(p, pl.grid, pl.T, pl.C); break;
      default: rc = int4 ? w4_mma_e4m3_int4(p, pl.grid, pl.T, pl.C) : w4_mma_e4m3_e2m1(p, pl.grid, pl.T, pl.C); break;
    }
    if (rc != LS_OK) return rc;
  }
  return LS_OK;
}

int launch_w4_expand(const W4ExpandArgs& a) {
  const int64_t bx = (a.w.K + 255) / 256;
  const dim3 g((unsigned)(bx < 1024 ? bx : 1024), (unsigned)(a.w.N < 65535 ? a.w.N : 65535));
  hipLaunchKernelGGL(gtk::w4_expand_kernel, g, dim3(256), 0, a.stream, a);
  return hipGetLastError() == hipSuccess ? LS_OK : LS_HIP_ERROR;
}

}  // namespace gt
