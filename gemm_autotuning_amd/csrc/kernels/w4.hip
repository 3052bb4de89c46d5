// w4.hip -- rows times 4-bit weights with group scales, and the expansion of
// such weights.
#include "elements.h"
#include "launchers.h"
#include "w4_mma.h"

namespace gtk {

// Nibble e of u as the value it stands for.
template <int FMT>
__device__ __forceinline__ float nibble_value(uint32_t u, int e) {
  const uint32_t c = u >> (4 * e) & 15u;
  if constexpr (FMT == W4_INT4) return (float)((int)(c << 28) >> 28);
  const uint32_t m = c & 7u;
  const float v = m < 2 ? 0.5f * m : __uint_as_float(((m >> 1) + 126u) << 23 | (m & 1u) << 22);
  return c & 8u ? -v : v;
}
template <int FMT>
__device__ __forceinline__ void nibble_pair(uint32_t u, int pair, float* v) {
  if constexpr (FMT == W4_E2M1) {
    f32x2v f;
    if (pair == 0) f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u, 1.f, 0);
    if (pair == 1) f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u, 1.f, 1);
    if (pair == 2) f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u, 1.f, 2);
    if (pair == 3) f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u, 1.f, 3);
    v[0] = f[0];
    v[1] = f[1];
  } else {
    v[0] = nibble_value<FMT>(u, 2 * pair);
    v[1] = nibble_value<FMT>(u, 2 * pair + 1);
  }
}

// Rows too short for a lane's 16 bytes, or so far apart that a tile's offsets
// pass 32 bits: a thread to an output.
__global__ __launch_bounds__(256) void w4_plain_kernel(gt::W4Args a) {
  for (int64_t m = blockIdx.y; m < a.M; m += gridDim.y)
    for (int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x; n < a.w.N; n += (int64_t)gridDim.x * 256) {
      float y = 0.f;
      for (int64_t k0 = 0; k0 < a.w.K; k0 += a.w.group) {
        float sum = 0.f;
        for (int64_t k = k0; k < a.w.K && k < k0 + a.w.group; ++k) {
          const uint32_t b = a.w.q[n * a.w.ldq + (k >> 1)];
          const float v = a.w.format == W4_INT4 ? nibble_value<W4_INT4>(b, k & 1) : nibble_value<W4_E2M1>(b, k & 1);
          const int64_t i = m * a.ldx + k;
          sum += v * (a.x_dtype == DT_E4M3 ? e4m3_bits_to_f32(static_cast<const uint8_t*>(a.x)[i]) : load_any(a.x, i, a.x_dtype));
        }
        y += sum * load_any(a.w.scales, n * a.w.lds_n + k0 / a.w.group * a.w.lds_g, a.w.scale_dtype);
      }
      store_out(a.y, m * a.ldy + n, y * a.x_scale * (a.row_scale ? a.row_scale[m] : 1.f), a.out_dtype);
    }
}

// The slices' partial sums, four columns to a thread.  A launch of its own:
// joined by the last workgroup of a column block inside the product's launch,
// the sums of 61 x 11001 x 4100 were left to 85 CUs and took 10 us.
__global__ __launch_bounds__(256) void w4_join_kernel(W4Params p) {
  const gt::W4Args& a = p.a;
  const int64_t n = 4 * ((int64_t)blockIdx.x * 256 + threadIdx.x), m = blockIdx.y;
  if (n >= a.w.N) return;
  const float* at = p.ws + m * p.ws_ld + n;  // columns past N, up to a tile, are in the workspace
  const int64_t stride = a.M * p.ws_ld;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  for (int q0 = 0; q0 < p.S; q0 += 4) {
    f32x4 part[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) part[j] = *reinterpret_cast<const f32x4*>(at + min(q0 + j, p.S - 1) * stride);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (q0 + j < p.S) v += part[j];
  }
  const float f = a.row_scale ? a.row_scale[m] : 1.f;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (n + e < a.w.N) store_out(a.y, m * a.ldy + n + e, v[e] * a.x_scale * f, a.out_dtype);
}

// Expansion: out[n,k] = s[n,k/G] * v(q[n,k]) rounded once.  The stores bound
// it (four bytes written for one read at 16 bits), so a thread makes whole
// 16-byte stores, from a piece of E weights; a group is a whole number of
// pieces.  A thread takes PER pieces, all loaded before the first is stored:
// 256 pieces apart along a long row, or those of rows below each other where
// a row has no more than 256 (1 << lg threads to a row).  The last K % E
// weights of a row go one to a thread beside them.
// 16384 x 8192 to bf16: 47.9 us, 7.1 TB/s, the rate of a fill (73 with its
// stores through the caches; four and eight pieces a thread 48.4 and 51.3, and
// 32768 x 1024 with two, four and eight 14.8, 17.4 and 25.2).
template <int FMT, int OUT, bool LONG, int PER>
__global__ __launch_bounds__(256) void w4_expand_kernel(gt::W4ExpandArgs a, int lg, int group_lg) {
  typedef typename Elem<OUT>::T TO;
  constexpr int E = 16 / (int)sizeof(TO);
  const int64_t whole = a.w.K / E * E;
  const int tx = threadIdx.x & ((1 << lg) - 1), ty = threadIdx.x >> lg, per_block = 256 >> lg;
  const int64_t block_rows = LONG ? 1 : (int64_t)per_block * PER;
  const bool ends = whole < a.w.K && (!LONG || blockIdx.y == 0);
  constexpr int kEnds = LONG ? 1 : PER;  // rows of a thread
  for (int64_t n0 = blockIdx.x * block_rows; n0 < a.w.N; n0 += gridDim.x * block_rows) {
    auto row = [&](int j) { return LONG ? n0 : n0 + j * per_block + ty; };
    auto col = [&](int j) { return E * (LONG ? ((int64_t)blockIdx.y * PER + j) * 256 + tx : (int64_t)tx); };
    auto scale = [&](int64_t n, int64_t k) {
      return load_any(a.w.scales, n * a.w.lds_n + (k >> group_lg) * a.w.lds_g, a.w.scale_dtype);
    };
    uint32_t q[PER], q_end[kEnds];
    float s[PER], s_end[kEnds];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int64_t n = row(j), k = col(j);
      q[j] = 0;
      s[j] = 0.f;
      if (n < a.w.N && k < whole) {
        __builtin_memcpy(&q[j], a.w.q + n * a.w.ldq + (k >> 1), E / 2);
        s[j] = scale(n, k);
      }
    }
    const int64_t k_end = whole + tx;
    if (ends) {
#pragma unroll
      for (int j = 0; j < kEnds; ++j)
        if (row(j) < a.w.N && k_end < a.w.K) {
          q_end[j] = a.w.q[row(j) * a.w.ldq + (k_end >> 1)];
          s_end[j] = scale(row(j), k_end);
        }
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int64_t n = row(j), k = col(j);
      float v[E];
#pragma unroll
      for (int p = 0; p < E / 2; ++p) nibble_pair<FMT>(q[j], p, v + 2 * p);
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] *= s[j];
      if (n < a.w.N && k < whole) store_piece<OUT, E>(reinterpret_cast<TO*>(a.y) + n * a.ldy + k, v, a.past_caches);
    }
    if (ends) {
#pragma unroll
      for (int j = 0; j < kEnds; ++j)
        if (row(j) < a.w.N && k_end < a.w.K)
          reinterpret_cast<TO*>(a.y)[row(j) * a.ldy + k_end] =
              Elem<OUT>::put(s_end[j] * nibble_value<FMT>(q_end[j], (int)(k_end & 1)));
    }
  }
}

}  // namespace gtk

namespace gt {

namespace {
constexpr int64_t kRowBlock = 256;         // most rows of one launch
constexpr int64_t kPartials = 64ll << 20;  // most bytes of the slices' partial sums of one launch

// Whether the tiles can take these weights: 16 bytes to a row at least, and
// 16 rows (and a wave's groups of their scales) within 31-bit byte offsets.
bool w4_tiled(const W4Weights& w) {
  const int64_t far = 0x7fffffff;
  return w.K >= gtk::kW4LeastK && w.ldq <= far / 32 && w.lds_n <= far / 128 && w.lds_g <= far / 4 / 64;
}

struct W4Plan {
  int T, C, waves, groups, S, tiles, chunks;
  dim3 grid;
};

bool w4_plan(const W4Args& a, int64_t rows, int cus, W4Plan* p) {
  const int64_t chunks = (a.w.K + gtk::kW4Chunk - 1) / gtk::kW4Chunk, tiles = (a.w.N + 15) / 16;
  if (chunks > 0x7fffffff / 16 || tiles > 0x7fffffff / 2) return false;
  p->chunks = (int)chunks;
  p->tiles = (int)tiles;
  // Blocks of 16 rows to a workgroup.  More read the weights less often, but
  // take longer to begin; where one to a workgroup fits the CUs, that: 53 x 118
  // x 244 takes 5.6 us and with four 8.7, 64 x 2048 x 4096 (512 workgroups of
  // one block) 14.5 and 12.4.
  p->T = rows <= 16 ? 1 : (rows <= 32 ? 2 : 4);
  if (tiles * ((rows + 15) / 16) <= cus) p->T = 1;
  // Chunks to a wave: as few as hold K, up to four (two with more rows, for
  // registers), then slices of K.  Eight would spare the slices' second
  // launch, but leave one tile in flight: 4 x 65536 x 8192 bf16 and int4 56.6
  // us, 63.6 with eight, f16 56.4 and 57.7, 1 x 32768 x 8192 30.6 and 34.5
  // (rows of 3000 bytes through the caches, 4 x 65536 x 6000: bf16 48.2 and
  // 48.7, f16 52.0 and 49.2).
  p->C = chunks <= gtk::kW4Waves ? 1 : (p->T > 1 || chunks <= 2 * gtk::kW4Waves ? 2 : 4);
  p->waves = (int)(chunks < gtk::kW4Waves ? chunks : gtk::kW4Waves);
  const int per = p->waves * p->C;
  p->S = (int)((chunks + per - 1) / per);
  // Short K leaves waves over, which take other columns.  Workgroups a CU: as
  // many as are there at a time.  Two of one chunk a wave: 16 x 65536 x 1024
  // 13.5 us, 16.6 with one, 15.9 with four.
  p->groups = gtk::kW4Waves / p->waves;
  const int64_t most = (p->C == 1 && p->T == 1 ? 2 : 1) * (int64_t)cus / p->S, wgs = (tiles + p->groups - 1) / p->groups;
  p->grid = dim3((unsigned)(wgs < most ? wgs : (most > 1 ? most : 1)), (unsigned)p->S,
                 (unsigned)((rows + 16 * p->T - 1) / (16 * p->T)));
  return p->S <= 65535;
}

// Rows and columns of one launch: all columns of up to 256 rows, unless the
// slices' partial sums would pass kPartials (S x rows x columns floats; S
// grows with K).  Then fewer rows, in blocks of 64 as a workgroup takes them
// (256 x 65536 x 8192 524 us, 520 in one launch; in ranges of columns 567);
// where not even 64 fit, ranges of columns of equal numbers of tiles, and 16
// rows where not even one tile fits (with S at most 65535 one always does).
// A part's own plan takes no more slices than the whole's: only T falls with
// its size, and a smaller T has as many chunks to a wave or more.
struct W4Ranges {
  int64_t rows, cols;
};
bool w4_ranges(const W4Args& a, int cus, W4Ranges* r) {
  r->rows = a.M < kRowBlock ? a.M : kRowBlock;
  r->cols = a.w.N;
  W4Plan p;
  if (!w4_plan(a, r->rows, cus, &p)) return false;
  auto fits = [&] { return kPartials / (64 * (int64_t)p.S * p.tiles); };  // rows of all columns
  if (p.S == 1 || fits() >= r->rows) return true;
  r->rows = fits() >= 64 ? fits() / 64 * 64 : (r->rows < 64 ? r->rows : 64);
  while (w4_plan(a, r->rows, cus, &p)) {
    if (p.S == 1 || fits() >= r->rows) return true;
    const int64_t most = kPartials / (64 * p.S * r->rows);  // tiles
    if (most > 0) {
      const int64_t parts = (p.tiles + most - 1) / most;
      r->cols = 16 * ((p.tiles + parts - 1) / parts);
      return true;
    }
    r->rows = 16;
  }
  return false;
}
// The part of the problem at rows m0.. and columns n0...
W4Args w4_part(const W4Args& all, const W4Ranges& r, int64_t m0, int64_t n0) {
  W4Args a = all;
  a.M = all.M - m0 < r.rows ? all.M - m0 : r.rows;
  a.w.N = all.w.N - n0 < r.cols ? all.w.N - n0 : r.cols;
  a.w.q = all.w.q + n0 * all.w.ldq;
  a.w.scales = static_cast<const char*>(all.w.scales) + n0 * all.w.lds_n * elem_bytes(all.w.scale_dtype);
  a.x = static_cast<const char*>(all.x) + m0 * all.ldx * elem_bytes(all.x_dtype);
  a.y = static_cast<char*>(all.y) + (m0 * all.ldy + n0) * elem_bytes(all.out_dtype);
  if (all.row_scale) a.row_scale = all.row_scale + m0;
  return a;
}
}  // namespace

size_t w4_workspace_bytes(const W4Args& a, int cus) {
  size_t most = 0;
  W4Ranges r;
  if (!w4_tiled(a.w) || !w4_ranges(a, cus, &r)) return 0;
  // the parts that there are: whole ones and the last of either direction
  for (const int64_t m0 : {(int64_t)0, (a.M - 1) / r.rows * r.rows})
    for (const int64_t n0 : {(int64_t)0, (a.w.N - 1) / r.cols * r.cols}) {
      const W4Args part = w4_part(a, r, m0, n0);
      W4Plan p;
      if (!w4_plan(part, part.M, cus, &p) || p.S == 1) continue;
      const size_t need = kCounterRegion + (size_t)p.S * part.M * p.tiles * 64;
      most = need > most ? need : most;
    }
  return most;
}

namespace {
int w4_launch(const W4Args& a, void* ws, int cus) {
  W4Plan pl;
  if (!w4_plan(a, a.M, cus, &pl)) return LS_UNSUPPORTED;
  gtk::W4Params p;
  p.a = a;
  p.ws = ws ? reinterpret_cast<float*>(static_cast<char*>(ws) + kCounterRegion) : nullptr;
  p.ws_ld = (int64_t)pl.tiles * 16;
  p.S = pl.S;
  p.waves = pl.waves;
  p.groups = pl.groups;
  p.waves_inverse = (65536 + pl.waves - 1) / pl.waves;
  p.tiles = pl.tiles;
  p.chunks_each = pl.chunks / pl.S;
  p.chunks_rest = pl.chunks % pl.S;
  const int columns = (int)pl.grid.x * pl.groups;
  p.tiles_each = pl.tiles / columns;
  p.tiles_rest = pl.tiles % columns;
  const bool int4 = a.w.format == gtk::W4_INT4;
  int rc;
  switch (a.x_dtype) {
    case DT_BF16: rc = int4 ? w4_mma_bf16_int4(p, pl.grid, pl.T, pl.C) : w4_mma_bf16_e2m1(p, pl.grid, pl.T, pl.C); break;
    case DT_F16: rc = int4 ? w4_mma_f16_int4(p, pl.grid, pl.T, pl.C) : w4_mma_f16_e2m1(p, pl.grid, pl.T, pl.C); break;
    default: rc = int4 ? w4_mma_e4m3_int4(p, pl.grid, pl.T, pl.C) : w4_mma_e4m3_e2m1(p, pl.grid, pl.T, pl.C); break;
  }
  if (rc != LS_OK || p.S == 1) return rc;
  hipLaunchKernelGGL(gtk::w4_join_kernel, dim3((unsigned)((a.w.N + 1023) / 1024), (unsigned)a.M), dim3(256), 0, a.stream, p);
  return hipGetLastError() == hipSuccess ? LS_OK : LS_HIP_ERROR;
}
}  // namespace

int launch_w4_matmul(const W4Args& all, void* ws, int cus) {
  if (!w4_tiled(all.w)) {
    const int64_t wgs = (all.w.N + 255) / 256;
    const dim3 g((unsigned)(wgs < (1 << 22) ? wgs : 1 << 22), (unsigned)(all.M < 65535 ? all.M : 65535));
    hipLaunchKernelGGL(gtk::w4_plain_kernel, g, dim3(256), 0, all.stream, all);
    return hipGetLastError() == hipSuccess ? LS_OK : LS_HIP_ERROR;
  }
  W4Ranges r;
  if (!w4_ranges(all, cus, &r)) return LS_UNSUPPORTED;
  for (int64_t n0 = 0; n0 < all.w.N; n0 += r.cols)
    for (int64_t m0 = 0; m0 < all.M; m0 += r.rows) {
      const int rc = w4_launch(w4_part(all, r, m0, n0), ws, cus);
      if (rc != LS_OK) return rc;
    }
  return LS_OK;
}

namespace {
template <int FMT, int OUT>
int expand_launch(const W4ExpandArgs& a, int cus) {
  const int64_t pieces = a.w.K / (16 / elem_bytes(OUT));  // the rest goes to threads that have a piece
  const int group_lg = a.w.group == 32 ? 5 : (a.w.group == 64 ? 6 : 7);
  // a row's rest of up to seven weights needs as many threads
  int lg = 3;
  while (lg < 8 && (1 << lg) < pieces) ++lg;
  const bool wide = pieces > 256;
  // Two pieces a thread, or one where that leaves CUs without a workgroup
  // (500 x 2000 to bf16 in a graph: 2.3 us, 3.4 with four).
  auto blocks = [&](int per, int64_t* parts) {
    const int64_t rows = wide ? 1 : (int64_t)(256 >> lg) * per;
    *parts = wide ? (pieces + 256 * per - 1) / (256 * per) : 1;
    return (a.w.N + rows - 1) / rows;
  };
  int64_t parts = 1, wgs = blocks(2, &parts);
  const bool one = wgs * parts < 2 * (int64_t)cus;
  if (one) wgs = blocks(1, &parts);
  if (parts > 65535) return LS_UNSUPPORTED;
  const dim3 g((unsigned)(wgs < (1 << 22) ? wgs : 1 << 22), (unsigned)parts);
#define GT_EXPAND(LONG, PER) \
  hipLaunchKernelGGL((gtk::w4_expand_kernel<FMT, OUT, LONG, PER>), g, dim3(256), 0, a.stream, a, lg, group_lg)
  if (wide && one)
    GT_EXPAND(true, 1);
  else if (wide)
    GT_EXPAND(true, 2);
  else if (one)
    GT_EXPAND(false, 1);
  else
    GT_EXPAND(false, 2);
#undef GT_EXPAND
  return hipGetLastError() == hipSuccess ? LS_OK : LS_HIP_ERROR;
}
template <int FMT>
int expand_format(const W4ExpandArgs& a, int cus) {
  switch (a.out_dtype) {
    case DT_F32: return expand_launch<FMT, DT_F32>(a, cus);
    case DT_F16: return expand_launch<FMT, DT_F16>(a, cus);
    default: return expand_launch<FMT, DT_BF16>(a, cus);
  }
}
}  // namespace

int launch_w4_expand(const W4ExpandArgs& args, int cus) {
  W4ExpandArgs a = args;
  a.past_caches = (double)a.w.N * a.w.K * (0.5 + elem_bytes(a.out_dtype)) > gtk::kPastCaches;
  return a.w.format == gtk::W4_INT4 ? expand_format<gtk::W4_INT4>(a, cus) : expand_format<gtk::W4_E2M1>(a, cus);
}

}  // namespace gt
