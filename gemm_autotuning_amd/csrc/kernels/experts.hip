// experts.hip -- a layer of gated experts for a few tokens: the gated product
// into fp32 activations per (token, slot) pair, the down product of each pair
// (grouped.h), and the pairs' weighted sum; single tokens in experts_token.hip.
#include "elements.h"
#include "grouped_wide.h"
#include "launchers.h"

namespace gtk {

// Weight (e, n, k) as a float.
__device__ __forceinline__ float expert_weight(const gt::ExpertWeights& w, int64_t e, int64_t n, int64_t k, int dtype, int format,
                                               int scale_dtype, int group_lg) {
  const char* row = w.p + e * w.stride + n * w.ld;
  if (format < 0) return load_any(row, k, dtype);
  const uint32_t c = (uint8_t)row[k >> 1] >> (4 * (k & 1)) & 15u;
  float v;
  if (format == W4_INT4) {
    v = (float)((int)(c << 28) >> 28);
  } else {
    const uint32_t m = c & 7u;
    v = m < 2 ? 0.5f * m : __uint_as_float(((m >> 1) + 126u) << 23 | (m & 1u) << 22);
    v = c & 8u ? -v : v;
  }
  return v * load_any(w.scales, e * w.s_lde + n * w.s_ldn + (k >> group_lg) * w.s_ldg, scale_dtype);
}

// Rows of weights too short for a lane's 16 bytes, or so far apart that a
// tile's offsets pass 32 bits: a wave to an output.
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

// y[t] = base[t] + sum_j weight[t,j] * part[t,j], four columns to a thread; a
// part has `split` slices.  A launch and one trip to the L2s: 4.1 us for 16 tokens x
// 4 parts of 4096, 4.9 for 64 x 8.
__global__ __launch_bounds__(256) void moe_join_kernel(gt::MoeArgs a, const float* part, int64_t ld, int split) {
  const int64_t n = 4 * ((int64_t)blockIdx.x * 256 + threadIdx.x), t = blockIdx.y;
  if (n >= a.K) return;
  f32x4 y = {0.f, 0.f, 0.f, 0.f};
  if (a.base) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < a.K) y[e] = load_any(a.base, t * a.ldb + n + e, a.out_dtype);
  }
  // eight slots at a time, their loads under way together; a slot that adds
  // nothing reads another's place
  for (int j0 = 0; j0 < a.topk; j0 += 8) {
    int of[8];
    float w[8];
    f32x4 v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int slot = min(j0 + j, a.topk - 1);
      of[j] = a.index[t * a.ldi + slot];
      w[j] = a.weight[t * a.ldw + slot];
      v[j] = *reinterpret_cast<const f32x4*>(part + (t * a.topk + slot) * ld + n);
    }
    for (int s = 1; s < split; ++s)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[j] += *reinterpret_cast<const f32x4*>(part + ((s * a.M + t) * a.topk + min(j0 + j, a.topk - 1)) * ld + n);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j0 + j < a.topk && of[j] >= 0 && of[j] < a.E) y += w[j] * v[j];
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (n + e < a.K) store_out(a.y, t * a.ldy + n + e, y[e], a.out_dtype);
}

}  // namespace gtk

namespace gt {
namespace {

constexpr int64_t kMostPairs = gtk::kMostRows;

int down_split(const MoeArgs& a);
bool in_tiles(const MoeArgs& a);

struct MoeSpace {
  int64_t act_ld, part_ld, split;
  size_t act, part, bytes;  // offsets; with tiles their table comes first, without there are only activations
};
MoeSpace space(MoeArgs a, int64_t tokens) {
  MoeSpace s;
  a.M = tokens;
  const int64_t pairs = tokens * a.topk;
  const bool tiles = in_tiles(a);
  s.act_ld = (a.H + 3) / 4 * 4;
  s.part_ld = (a.K + 3) / 4 * 4;
  s.act = tiles ? gtk::row_table_bytes(pairs) : 0;
  s.part = s.act + (size_t)pairs * s.act_ld * 4;
  s.split = tiles ? down_split(a) : 0;
  s.bytes = s.part + (size_t)(pairs * s.split * s.part_ld * 4);
  return s;
}

// The down product of 4-bit weights, which are exact in f16, takes the
// activations as two f16 parts whatever x is: 22 bits of them, where two of bf16
// have 16 and three more matrix-core work.
GroupedLaunch launcher(const MoeArgs& a, bool down) {
  const bool bf = a.x_dtype == DT_BF16 && !(down && a.format >= 0);
  if (a.format == gtk::W4_INT4) return bf ? grouped_bf16_int4 : grouped_f16_int4;
  if (a.format == gtk::W4_E2M1) return bf ? grouped_bf16_e2m1 : grouped_f16_e2m1;
  return bf ? grouped_bf16 : grouped_f16;
}

// Whether a matrix' rows can be walked in whole units: 16 bytes of a row at
// least, and a tile's offsets within 32 bits.
bool in_units(const MoeArgs& a, const ExpertWeights& w, int64_t K) {
  const int64_t row = a.format < 0 ? 2 * K : (K + 1) / 2;
  const int64_t most = INT64_C(1) << 31;
  if (row < 16 || w.ld > most / 16 || row > most / 2) return false;
  if (a.format < 0) return true;
  const int e = elem_bytes(a.scale_dtype);
  return w.s_ldn <= most / 32 / e && w.s_ldg <= most / 2 / e / ((K >> a.group_lg) + 1);
}
bool in_units(const MoeArgs& a) { return in_units(a, a.gate_up, a.K) && in_units(a, a.down, a.H); }

// Whether so few tokens name the same experts that each may read its own
// (experts_token.hip): up to 32 MiB of weights read again, of 4 bits 4 MiB
// (their expansion costs more than their bytes), where every choice is as
// likely.  bf16, 8 of 128 experts 2048 x 768: 1 token 18.4 us and 24.4 with
// tiles, 4 tokens (27 MB) 50 and 53, 6 (61 MB) 70 and 66; 2 of 8 experts 256 x
// 512: 8 tokens 9.7 and 16.  int4, 4 of 64 experts 4096 x 2048: 1 token 20.8 and 24.5,
// 2 (3 MB) 34.0 and 34.4, 4 (20 MB) 55 and 51; 4 of 32 experts 1024 x 512: 4 tokens
// (3 MB) 15.8 and 20.5.  More than 8 tokens would gain only where the experts are
// tiny (16 tokens, 2 of 8 experts 256 x 512: 11.4 and 17.2) and have the tiles.
// One token always does: should it name experts twice, its tiles' sums would take
// up to topk * K floats for each slice of H.
bool hardly_share(const MoeArgs& a) {
  if (a.M > 8) return false;
  if (a.M == 1) return true;
  double left = 1.0;  // the share of experts that no token names
  for (int64_t t = 0; t < a.M; ++t) left *= std::max(0.0, 1.0 - (double)a.topk / a.E);
  const double again = (double)(a.M * a.topk) - a.E * (1.0 - left);
  const double bytes = 3.0 * a.H * a.K * (a.format < 0 ? 2.0 : 0.5);
  return again * bytes <= (a.format < 0 ? 32.0 : 4.0) * (1 << 20);
}

bool in_tiles(const MoeArgs& a) { return in_units(a) && !hardly_share(a); }

// How a product's K is cut: into units, a wave's slice of them, and where one
// workgroup's waves do not hold all of them, turns (the gated product) or
// workgroups whose sums the join adds (the down product).
struct MoeCut : gtk::GroupedCut {
  int units, split;
};
MoeCut cut(const MoeArgs& a, bool down) {
  MoeCut c{};
  const int64_t K = down ? a.H : a.K;
  if (a.wide) {
    c.units = (int)((K + 127) / 128);
    // along K as many workgroups as find a CU where each expert has a tile, of four units at least
    const int64_t items = std::max<int64_t>(a.E, a.M * a.topk / 64) * ((a.K + 255) / 256);
    c.split = down ? (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(a.cus / items, c.units / 4), 8)) : 1;
    c.wk = c.turns = 1;
    c.cols = 8;
    return c;
  }
  const int unit = a.format < 0 ? 128 : 256;
  c.units = (int)((K + unit - 1) / unit);
  if (a.format >= 0) {
    c.U = down ? 1 : 2;
    c.waves = 8;
  } else if (down && a.x_dtype == DT_BF16) {  // three parts: registers for two units
    c.waves = c.units > 8 ? 8 : 4;
    c.U = 2;
  } else {
    c.waves = c.units > 16 ? 8 : 4;
    c.U = c.units > 2 * c.waves ? 4 : 2;
  }
  const int most = c.U * c.waves;
  c.split = down ? (c.units + most - 1) / most : 1;
  const int each = (c.units + c.split - 1) / c.split;  // of a workgroup
  c.wk = std::min(c.waves, (each + c.U - 1) / c.U);
  c.turns = (each + c.wk * c.U - 1) / (c.wk * c.U);
  c.cols = c.waves / c.wk;
  return c;
}

int product(const MoeArgs& a, gtk::GroupedParams& p, int phase, int64_t tiles) {
  const int pairs = phase == gtk::GROUPED_GATE_UP ? (p.N + 15) / 16 : (p.N + 31) / 32;
  const MoeCut c = cut(a, phase == gtk::GROUPED_DOWN);
  fill_cut(p, c, c.units, c.split);
  if (!fill_list(p, tiles, (pairs + c.cols - 1) / c.cols, a.cus)) return LS_UNSUPPORTED;
  return a.wide ? (a.x_dtype == DT_BF16 ? grouped_wide_bf16 : grouped_wide_f16)(p, phase, a.out_dtype == DT_F32, a.stream) : launcher(a, phase == gtk::GROUPED_DOWN)(p, phase, c, a.stream);
}

int down_split(const MoeArgs& a) { return cut(a, true).split; }

}  // namespace

int64_t moe_range(const MoeArgs& a) {
  // (a wide call's slices of K are not counted: there are some only where all
  // their sums together stay below 256 columns of 64 rows to a CU, 16 MiB)
  const int64_t slices = a.wide ? 1 : down_split(a);
  const int64_t pairs = ((int64_t)64 << 20) / (4 * (a.H + slices * a.K + 6) + (int64_t)sizeof(gtk::RowTile));
  return std::max<int64_t>(1, std::min(pairs, kMostPairs) / a.topk);
}
// Whether an expert has at least 16 rows on average: 8 experts 4096 x 2048
// bf16 take 97 us with tiles of 64 rows and 120 with tiles of 16 there (128 tokens: 115 and 166,
// 512: 274 and 582), 97 and 92 with 12 rows.  Expanding 4-bit weights less
// often gains nothing (134 us both ways with 64 rows to an expert), so they
// have tiles of 16 only.
bool moe_wide(const MoeArgs& a) {
  MoeArgs wide = a;
  wide.wide = true;
  return a.format < 0 && std::min(a.M, moe_range(wide)) * a.topk >= 16 * (int64_t)a.E;
}
size_t moe_workspace_bytes(const MoeArgs& a, int64_t tokens) { return space(a, tokens).bytes; }

int launch_moe(const MoeArgs& a) {
  const MoeSpace s = space(a, a.M);
  float* act = reinterpret_cast<float*>(a.ws + s.act);
  float* part = reinterpret_cast<float*>(a.ws + s.part);
  if (!in_units(a)) {
    hipLaunchKernelGGL(gtk::moe_up_kernel, dim3((unsigned)((a.H + 3) / 4), (unsigned)(a.M * a.topk)), dim3(256), 0, a.stream, a, act);
    hipLaunchKernelGGL(gtk::moe_down_kernel, dim3((unsigned)((a.K + 3) / 4), (unsigned)a.M), dim3(256), 0, a.stream, a, act);
    return hipGetLastError() == hipSuccess ? LS_OK : LS_HIP_ERROR;
  }
  if (!in_tiles(a)) return launch_moe_tokens(a, act, s.act_ld);
  const int64_t pairs = a.M * a.topk, tiles = most_tiles(pairs, a.E, a.wide ? 64 : 16);
  gtk::GroupedParams p{};
  p.ix = gtk::RowIndex{a.index, a.ldi, (int)pairs, a.topk, a.E, ((1u << 20) + a.topk - 1) / a.topk, 0, bits_of(a.E - 1), a.wide ? 6 : 4};
  p.table = reinterpret_cast<gtk::RowTable*>(a.ws);
  p.scale_dtype = a.scale_dtype;
  p.group = 1 << a.group_lg;
  p.activation = a.activation;
  p.w = a.gate_up;
  p.x = a.x;
  p.ldx = a.ldx;
  p.out = act;
  p.ld_out = s.act_ld;
  p.up = a.H;
  p.N = (int)a.H;
  p.K = (int)a.K;
  int rc = LS_OK;
  if (pairs > gtk::kFewRows) rc = launch_row_tiles(p.ix, p.table, a.stream);
  if (rc == LS_OK) rc = product(a, p, gtk::GROUPED_GATE_UP, tiles);
  if (rc != LS_OK) return rc;
  p.w = a.down;
  p.x = act;
  p.ldx = s.act_ld;
  p.out = part;
  p.ld_out = s.part_ld;
  p.out_slice = pairs * s.part_ld;
  p.N = (int)a.K;
  p.K = (int)a.H;
  rc = product(a, p, gtk::GROUPED_DOWN, tiles);
  if (rc != LS_OK) return rc;
  hipLaunchKernelGGL(gtk::moe_join_kernel, dim3((unsigned)((a.K + 1023) / 1024), (unsigned)a.M), dim3(256), 0, a.stream, a, part,
                     s.part_ld, (int)s.split);
  return hipGetLastError() == hipSuccess ? LS_OK : LS_HIP_ERROR;
}

}  // namespace gt
