// grouped.h -- products of a few gathered rows with the weights that each of
// them names (experts, adapters), on the matrix cores.
//
//   out[row, n] = sum_k x[row, k] * w[of(row), n, k]
//
// Rows that name the same matrix form tiles of 16 T rows, each taken by the
// workgroups of its columns.  The weights are read from HBM once per tile and
// bound the time; everything is arranged around that stream, as for the rows
// times shared 4-bit weights (w4_mma.h).  A wave owns a slice of K, at most U
// units of 256 bytes of a 16-bit row (128 of a 4-bit one), keeps the rows'
// slice in registers as operands of 16x16x32 matrix-core blocks, and walks
// pairs of tiles of 16 columns with D units of weights in flight.  A unit's
// load has neighbouring lanes on consecutive bytes of a column and is laid
// out through an LDS region of the wave's own.  The workgroup's waves hold
// consecutive slices; their sums are joined in LDS, in order, by one barrier
// a pair of tiles.
//
// Nothing is loaded under a condition in that walk (what there is nothing for
// reads one address that is read anyway), so that the wait for a unit leaves
// the later ones in flight.
#pragma once

#include <algorithm>

#include "w4_mma.h"

namespace gtk {

constexpr int kGroupWaves = 8;       // most waves of a workgroup
constexpr int kMostMatrices = 4096;  // counted in LDS
enum { GROUPED_16 = -1 };            // weights of the rows' type; else W4_INT4, W4_E2M1
enum { GROUPED_GATE_UP = 0, GROUPED_DOWN = 1, GROUPED_SHRINK = 2 };

// A tile of rows: the matrix, how many rows, which.  matrix < 0: no tile.
struct RowTile {
  int matrix, count;
  int rows[16];
};

// The rows that name matrices, for the search of a tile: row i's matrix is
// index[i / per * ld + i % per], none outside 0..matrices-1.
struct RowIndex {
  const int32_t* index;
  int64_t ld;
  int n, per, matrices;
  int none;  // whether rows without a matrix form tiles too (of matrix `matrices`)
};

struct GroupedParams {
  RowIndex ix;
  RowTile* table;      // written by the first launch (its workgroups of columns 0), read by the others
  gt::ExpertWeights w;
  const void* x;       // 16-bit rows (row i of the index is x's row i / per), or the fp32 ones of the first launch
  int64_t ldx;
  float* out;          // fp32, row i at i * ld_out; GROUPED_SHRINK: slice s at s * out_slice
  int64_t ld_out, out_slice;
  int64_t up;          // GROUPED_GATE_UP: the row of w where the second half begins
  int N, K;            // columns (of a half), length
  int scale_dtype, group_lg, activation;
  int units_each, units_rest;  // of a slice of K, a wave's in one turn: the first `rest` have one more
  int wk, turns;       // waves side by side along K; times that the x operands are loaded anew
  int pairs, pairs_each;  // pairs of column tiles; of a wave
  int wk_inverse;      // 2^16 / wk, rounded up: exact for what is divided (at most 8)
};

// The tile number `t`, in LDS: rows that name the same matrix in the order of
// their numbers, 16 T to a tile.  Up to 64 rows: one wave compares all of them
// at once; else the matrices' rows are counted, the tiles before each matrix
// summed, and the matrix's rows numbered by ballots.  Every workgroup that asks
// for a tile finds the same one.
template <int ROWS>
struct TileSearch {
  int matrix, count, first;  // first: how many of the matrix's rows come before the tile
  int rows[ROWS];
  int of_wave[kGroupWaves];
};
__device__ __forceinline__ int row_matrix(const RowIndex& ix, int i) {
  const int t = ix.per == 1 ? i : i / ix.per;
  const int e = ix.index[(int64_t)t * ix.ld + (i - t * ix.per)];
  return e >= 0 && e < ix.matrices ? e : (ix.none ? ix.matrices : -1);
}
template <int ROWS>
__device__ void find_tile(const RowIndex& ix, int t, TileSearch<ROWS>& s, uint32_t* count) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, waves = blockDim.x >> 6;
  const uint64_t before = (1ull << lane) - 1;
  if (ix.n <= 64) {
    if (wave == 0) {
      const int e = lane < ix.n ? row_matrix(ix, lane) : -1;
      uint64_t same = __ballot(e >= 0);
#pragma unroll
      for (int b = 0; b < 13; ++b) {
        const uint64_t v = __ballot(e >> b & 1);
        same &= e >> b & 1 ? v : ~v;
      }
      const int rank = __popcll(same & before);
      const bool leads = e >= 0 && rank % ROWS == 0;
      const uint64_t leaders = __ballot(leads);
      const uint64_t mine = __ballot(leads && __popcll(leaders & before) == t);
      if (mine == 0) {
        if (lane == 0) s.matrix = -1;
      } else {
        const int at = __ffsll((unsigned long long)mine) - 1;
        const int matrix = __builtin_amdgcn_readlane(e, at), first = __builtin_amdgcn_readlane(rank, at);
        const bool in = e == matrix && rank >= first && rank < first + ROWS;
        const int n = __popcll(__ballot(in));
        if (in) s.rows[rank - first] = lane;
        if (lane == 0) {
          s.matrix = matrix;
          s.count = n;
        }
      }
    }
    __syncthreads();
    return;
  }
  const int all = ix.matrices + ix.none;
  for (int e = tid; e < all; e += blockDim.x) count[e] = 0;
  __syncthreads();
  for (int i = tid; i < ix.n; i += blockDim.x) {
    const int e = row_matrix(ix, i);
    if (e >= 0) atomicAdd(&count[e], 1u);
  }
  __syncthreads();
  if (wave == 0) {
    const int per = (all + 63) / 64, e0 = min(lane * per, all), e1 = min(e0 + per, all);
    int tiles = 0;
    for (int e = e0; e < e1; ++e) tiles += ((int)count[e] + ROWS - 1) / ROWS;
    int upto = tiles;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int v = __shfl_up(upto, d);
      if (lane >= d) upto += v;
    }
    if (lane == 63 && t >= upto) s.matrix = -1;
    if (t < upto && t >= upto - tiles) {
      int left = t - (upto - tiles);
      for (int e = e0; e < e1; ++e) {
        const int c = (int)count[e], n = (c + ROWS - 1) / ROWS;
        if (left < n) {
          s.matrix = e;
          s.first = left * ROWS;
          s.count = min(c - left * ROWS, ROWS);
          break;
        }
        left -= n;
      }
    }
  }
  __syncthreads();
  const int matrix = s.matrix;
  if (matrix < 0) return;
  const int first = s.first;
  const int blocks = (ix.n + 63) / 64, each = (blocks + waves - 1) / waves;
  int found = 0;
  for (int b = wave * each; b < min((wave + 1) * each, blocks); ++b) {
    const int i = b * 64 + lane;
    found += __popcll(__ballot(i < ix.n && row_matrix(ix, i) == matrix));
  }
  if (lane == 0) s.of_wave[wave] = found;
  __syncthreads();
  int rank = 0;
  for (int w = 0; w < wave; ++w) rank += s.of_wave[w];
  if (found > 0 && rank < first + ROWS && rank + found > first)
    for (int b = wave * each; b < min((wave + 1) * each, blocks); ++b) {
      const int i = b * 64 + lane;
      const bool is = i < ix.n && row_matrix(ix, i) == matrix;
      const uint64_t v = __ballot(is);
      const int r = rank + __popcll(v & before);
      if (is && r >= first && r < first + ROWS) s.rows[r - first] = i;
      rank += __popcll(v);
    }
  __syncthreads();
}

__device__ __forceinline__ float activated(float g, float u, int activation) {
  // GELU's tanh form is g / (1 + exp(-2 z)), z = sqrt(2 / pi) (g + 0.044715 g^3)
  const float z = activation == 0 ? g : 1.5957691216057308f * (g + 0.044715f * g * g * g);
  return g / (1.f + expf(-z)) * u;
}

// 16 bytes less their first d (d >= 0), zeros behind.
__device__ __forceinline__ u32x4 bytes_from(u32x4 v, int d) {
  unsigned __int128 w;
  __builtin_memcpy(&w, &v, 16);
  w = d < 16 ? w >> (8 * d) : 0;
  __builtin_memcpy(&v, &w, 16);
  return v;
}

template <int FMT>
struct UnitOf {
  static constexpr bool k4 = FMT != GROUPED_16;
  static constexpr int kBytes = k4 ? 128 : 256;       // of a column
  static constexpr int kK = k4 ? 256 : 128;           // k of them
  static constexpr int kLanes = kBytes / 16, kCols = 64 / kLanes, kLoads = 16 / kCols;
  static constexpr int kSteps = kK / 32;              // matrix-core steps
  static constexpr int kRowUnits = kK / 128;          // 256-byte units of a 16-bit row
  static constexpr int kPitch = kBytes + 16;          // of a column in LDS: reads of 16 columns fall on different banks
};

// What a wave lays out through LDS: weights of a unit (and its scales per 32
// k), before that 16 rows' 128 elements.
struct alignas(16) GroupedStage {
  char q[16 * 272];
};
template <int FMT>
struct ScaleStage {
  float s[16][12];
};
template <>
struct ScaleStage<GROUPED_16> {};

template <int PHASE, int XT, int FMT, int WIDE, int T, int U, int D>
__global__ __launch_bounds__(64 * kGroupWaves) void grouped_kernel(GroupedParams p) {
  typedef UnitOf<FMT> Unit;
  typedef W4Operand<XT, FMT == GROUPED_16 ? W4_E2M1 : FMT> Op;  // e2m1: elements in order
  typedef typename std::conditional<WIDE, uint32_t, uint16_t>::type Scale;
  constexpr int ROWS = 16 * T;
  constexpr bool kSplit = PHASE == GROUPED_DOWN;  // fp32 rows, in two parts
  constexpr int kParts = kSplit ? 2 : 1;
  constexpr bool kScaled = kSplit && XT == DT_F16;
  static_assert((2 * U) % D == 0 || D % (2 * U) == 0, "places in the ring are known when compiled");
  static_assert(D <= 2 * U, "at most a pair ahead");
  __shared__ TileSearch<ROWS> tile;
  __shared__ union {
    uint32_t count[kMostMatrices + 1];
    GroupedStage stage[kGroupWaves];
  } u;
  __shared__ ScaleStage<FMT> scale_stage[Unit::k4 ? kGroupWaves : 1];
  __shared__ float red[2][kGroupWaves][2][T][256];
  __shared__ float unscale[kScaled ? kGroupWaves : 1][ROWS];

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, kq = lane >> 4;
  const int t = blockIdx.y;
  if constexpr (PHASE == GROUPED_DOWN) {
    const RowTile* e = p.table + t * T;
    if (tid == 0) {
      int n = 0;
      for (int j = 0; j < T; ++j) n += e[j].matrix < 0 ? 0 : e[j].count;
      tile.matrix = e->matrix;
      tile.count = n;
    }
    if (tid < ROWS) tile.rows[tid] = e[tid / 16].rows[tid % 16];
    __syncthreads();
  } else {
    find_tile<ROWS>(p.ix, t, tile, u.count);
    if (blockIdx.x == 0 && blockIdx.z == 0) {
      const int matrix = tile.matrix, count = tile.count;
      if (tid < T) {
        p.table[t * T + tid].matrix = matrix >= 0 && 16 * tid < count ? matrix : -1;
        p.table[t * T + tid].count = min(16, count - 16 * tid);
      }
      if (tid < ROWS) p.table[t * T + tid / 16].rows[tid % 16] = tid < count ? tile.rows[tid] : 0;
    }
  }
  const int matrix = __builtin_amdgcn_readfirstlane(tile.matrix);
  if (matrix < 0 || matrix >= p.ix.matrices) return;
  const int rows = __builtin_amdgcn_readfirstlane(tile.count);

  // this wave's slice of K and its columns
  const int cols = (wave * p.wk_inverse) >> 16, along = wave - cols * p.wk;
  int c0, nc;
  auto slice = [&](int turn) {
    const int s = (blockIdx.z * p.turns + turn) * p.wk + along;
    c0 = s * p.units_each + min(s, p.units_rest);
    nc = p.units_each + (s < p.units_rest);
  };
  const int waves_cols = ((int)(blockDim.x >> 6) * p.wk_inverse) >> 16;
  const int pair0 = (blockIdx.x * waves_cols + cols) * p.pairs_each, pair1 = min(pair0 + p.pairs_each, p.pairs);
  const int most_pairs = min(p.pairs - (int)blockIdx.x * waves_cols * p.pairs_each, p.pairs_each);  // of the workgroup's waves
  const uint32_t row_bytes = Unit::k4 ? (p.K + 1) / 2 : 2 * p.K;
  const uint32_t ld = (uint32_t)p.w.ld;
  const char* const wm = p.w.p + matrix * p.w.stride;
  const char* const sm = Unit::k4 ? static_cast<const char*>(p.w.scales) + matrix * p.w.s_lde * sizeof(Scale) : nullptr;
  const uint32_t s_ldn = (uint32_t)p.w.s_ldn * sizeof(Scale), s_ldg = (uint32_t)p.w.s_ldg * sizeof(Scale);
  const int groups = Unit::k4 ? (p.K + (1 << p.group_lg) - 1) >> p.group_lg : 0;

  // the first of a half's 16 columns, and how many it has less one
  auto column = [&](int pair, int half) {
    return PHASE == GROUPED_GATE_UP ? (int64_t)pair * 16 + half * p.up : (int64_t)(2 * pair + half) * 16;
  };
  auto last_of = [&](int pair, int half) {
    const int n = PHASE == GROUPED_GATE_UP ? pair * 16 : (2 * pair + half) * 16;
    return min(p.N - 1 - n, 15);  // below 0: no column
  };

  // ---- weights
  const int piece = lane % Unit::kLanes, sub = lane / Unit::kLanes;
  auto load_unit = [&](int pair, int half, int un, bool some, u32x4 (&q)[Unit::kLoads], Scale (&sc)[2]) __attribute__((always_inline)) {
    const int last = last_of(pair, half);
    some = some && un < nc && last >= 0;
    const uint32_t mask = some ? ~0u : 0u;
    const char* base = wm + (some ? column(pair, half) * p.w.ld : 0);
    const uint32_t at = min((uint32_t)(c0 + un) * Unit::kBytes + 16 * piece, row_bytes - 16);
#pragma unroll
    for (int i = 0; i < Unit::kLoads; ++i) {
      const uint32_t off = (min(i * Unit::kCols + sub, last) * ld + at) & mask;
      q[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(base + off));
    }
    if constexpr (Unit::k4) {
      const char* sb = sm + (some ? column(pair, half) * p.w.s_ldn * (int64_t)sizeof(Scale) : 0);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int k = (c0 + un) * Unit::kK + 32 * (4 * i + (lane & 3));
        const uint32_t off = (min(lane >> 2, last) * s_ldn + min(k >> p.group_lg, groups - 1) * s_ldg) & mask;
        sc[i] = *reinterpret_cast<const Scale*>(sb + off);
      }
    }
  };
  char* const st = u.stage[wave].q;
  auto stage_unit = [&](int un, u32x4 (&q)[Unit::kLoads], const Scale (&sc)[2]) __attribute__((always_inline)) {
    const uint32_t at = (uint32_t)(c0 + un) * Unit::kBytes;
    if (at + Unit::kBytes > row_bytes) {
      const uint32_t want = at + 16 * piece;
      const int d = want > row_bytes - 16 ? (int)(want - (row_bytes - 16)) : 0;
#pragma unroll
      for (int i = 0; i < Unit::kLoads; ++i) q[i] = bytes_from(q[i], d);
    }
#pragma unroll
    for (int i = 0; i < Unit::kLoads; ++i)
      *reinterpret_cast<u32x4*>(st + (i * Unit::kCols + sub) * Unit::kPitch + 16 * piece) = q[i];
    if constexpr (Unit::k4) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        Scale b = sc[i];
        float f;
        if constexpr (WIDE)
          f = __uint_as_float(b);
        else
          f = p.scale_dtype == DT_BF16 ? bf16_bits_to_f32(b) : f16_bits_to_f32(b);
        const int k = (c0 + un) * Unit::kK + 32 * (4 * i + (lane & 3));
        scale_stage[wave].s[lane >> 2][4 * i + (lane & 3)] = k >> p.group_lg < groups ? f : 0.f;  // past K: nothing, whatever the last scale is
      }
    }
    wave_lds_order();
  };

  // ---- rows, as operands: [unit][step][block of 16][part]
  Chunk xf[U][Unit::kSteps][T][kParts];
  auto row_at = [&](int m) { return tile.rows[min(m, rows - 1)]; };
  auto load_rows16 = [&](u32x4 (&raw)[U * Unit::kRowUnits][T][4]) __attribute__((always_inline)) {
#pragma unroll
    for (int t16 = 0; t16 < T; ++t16)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (16 * t16 + 4 * i < rows) {
          const int row = row_at(16 * t16 + 4 * i + kq);
          const uint16_t* x = static_cast<const uint16_t*>(p.x) + (p.ix.per == 1 ? row : row / p.ix.per) * p.ldx;
#pragma unroll
          for (int un = 0; un < U * Unit::kRowUnits; ++un) {
            const int k = (c0 * Unit::kRowUnits + un) * 128 + 8 * r;
            raw[un][t16][i] = *reinterpret_cast<const u32x4_any*>(x + min(k, p.K - 8));
          }
        }
  };
  auto place_rows16 = [&](u32x4 (&raw)[U * Unit::kRowUnits][T][4]) __attribute__((always_inline)) {
#pragma unroll
    for (int un = 0; un < U * Unit::kRowUnits; ++un) {
      const int k0 = (c0 * Unit::kRowUnits + un) * 128;
#pragma unroll
      for (int t16 = 0; t16 < T; ++t16) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (16 * t16 + 4 * i < rows) {
            u32x4 v = raw[un][t16][i];
            if (k0 + 128 > p.K) v = bytes_from(v, max(0, 2 * (k0 + 8 * r - (p.K - 8))));
            *reinterpret_cast<u32x4*>(st + (4 * i + kq) * 272 + 16 * r) = v;
          }
        wave_lds_order();
#pragma unroll
        for (int j = 0; j < 4; ++j)
          xf[un / Unit::kRowUnits][un % Unit::kRowUnits * 4 + j][t16][0] =
              Op::order(*reinterpret_cast<const u32x4*>(st + r * 272 + 16 * (4 * j + kq)));
        wave_lds_order();
      }
    }
  };
  // fp32 rows: 32 lanes to a row's 128 elements, two rows to a load
  auto load_rows32 = [&](f32x4 (&raw)[U * Unit::kRowUnits][T][8]) __attribute__((always_inline)) {
#pragma unroll
    for (int t16 = 0; t16 < T; ++t16)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (16 * t16 + 2 * i < rows) {
          const float* x = static_cast<const float*>(p.x) + row_at(16 * t16 + 2 * i + (lane >> 5)) * p.ldx;
#pragma unroll
          for (int un = 0; un < U * Unit::kRowUnits; ++un) {
            const int k = (c0 * Unit::kRowUnits + un) * 128 + 4 * (lane & 31);
            raw[un][t16][i] = *reinterpret_cast<const f32x4*>(x + min(k, (p.K - 1) & ~3));
          }
        }
  };
  auto place_rows32 = [&](f32x4 (&raw)[U * Unit::kRowUnits][T][8]) __attribute__((always_inline)) {
#pragma unroll
    for (int t16 = 0; t16 < T; ++t16)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (16 * t16 + 2 * i < rows) {
          uint32_t most = 0;
#pragma unroll
          for (int un = 0; un < U * Unit::kRowUnits; ++un) {
            const int k = (c0 * Unit::kRowUnits + un) * 128 + 4 * (lane & 31);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (k + e >= p.K || un >= nc * Unit::kRowUnits) raw[un][t16][i][e] = 0.f;
              most = max(most, __float_as_uint(raw[un][t16][i][e]) & 0x7fffffffu);
            }
          }
          if constexpr (kScaled) {
            // a power of two that brings the row's largest of this slice to 2^14..2^15; 1 for infinities and NaN
            auto largest = [](uint32_t a, uint32_t b) { return max(a, b); };
            most = largest(most, dpp<0xB1>(most));
            most = largest(most, dpp<0x4E>(most));
            most = largest(most, dpp<0x141>(most));
            most = largest(most, dpp<0x140>(most));
            const auto both = __builtin_amdgcn_permlane16_swap(most, most, false, false);
            most = largest(both[0], both[1]);
            const uint32_t ex = most >> 23;
            const uint32_t to = ex == 255 || ex == 0 ? 127u : min(253u, 268u - ex);
            if ((lane & 31) == 0) unscale[wave][16 * t16 + 2 * i + (lane >> 5)] = __uint_as_float((254u - to) << 23);
            const float s = __uint_as_float(to << 23);
#pragma unroll
            for (int un = 0; un < U * Unit::kRowUnits; ++un) raw[un][t16][i] *= s;
          }
        }
#pragma unroll
    for (int un = 0; un < U * Unit::kRowUnits; ++un)
#pragma unroll
      for (int t16 = 0; t16 < T; ++t16)
#pragma unroll
        for (int part = 0; part < 2; ++part) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (16 * t16 + 2 * i < rows) {
              f32x4 v = raw[un][t16][i];
              uint16_t h[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float back;
                if constexpr (XT == DT_BF16) {
                  // the first part is cut off, not rounded: it cannot pass bf16's range
                  const uint32_t top = __float_as_uint(v[e]) & 0xffff0000u;
                  h[e] = part == 0 ? (uint16_t)(top >> 16) : f32_to_bf16_bits(v[e]);
                  back = __uint_as_float(top);
                } else {
                  h[e] = f32_to_f16_bits(v[e]);
                  back = f16_bits_to_f32(h[e]);
                }
                const float left = v[e] - back;
                v[e] = left == left ? left : 0.f;  // of an infinity or NaN the first part has it all
              }
              raw[un][t16][i] = v;
              __builtin_memcpy(st + (2 * i + (lane >> 5)) * 272 + 8 * (lane & 31), h, 8);
            }
          wave_lds_order();
#pragma unroll
          for (int j = 0; j < 4; ++j)
            xf[un / Unit::kRowUnits][un % Unit::kRowUnits * 4 + j][t16][part] =
                Op::order(*reinterpret_cast<const u32x4*>(st + r * 272 + 16 * (4 * j + kq)));
          wave_lds_order();
        }
  };

  u32x4 ring[D][Unit::kLoads];
  Scale ring_s[D][2];
  // the unit `ahead` places after the first of a pair's (gate, then up; each its U units)
  auto load_at = [&](int pair, int ahead, bool some, int place) __attribute__((always_inline)) {
    load_unit(pair, ahead / U, ahead % U, some, ring[place], ring_s[place]);
  };
  auto rows_and_ring = [&](int pair) __attribute__((always_inline)) {
    if constexpr (kSplit) {
      f32x4 raw[U * Unit::kRowUnits][T][8];
      load_rows32(raw);
#pragma unroll
      for (int d = 0; d < D; ++d) load_at(pair, d, pair < pair1, d);
      place_rows32(raw);
    } else {
      u32x4 raw[U * Unit::kRowUnits][T][4];
      load_rows16(raw);
#pragma unroll
      for (int d = 0; d < D; ++d) load_at(pair, d, pair < pair1, d);
      place_rows16(raw);
    }
  };

  f32x4 acc[2][T], total[kScaled ? 2 : 1][kScaled ? T : 1];  // total: of the turns, each with scales of its own
  auto multiply_unit = [&](int half, int un) __attribute__((always_inline)) {
    if constexpr (!Unit::k4) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        Chunk w;
        __builtin_memcpy(&w, st + r * Unit::kPitch + 16 * (4 * j + kq), 16);
#pragma unroll
        for (int t16 = 0; t16 < T; ++t16)
#pragma unroll
          for (int part = 0; part < kParts; ++part) Op::mma(acc[half][t16], xf[un][j][t16][part], w);
      }
    } else {
      f32x4 sum[T];
#pragma unroll
      for (int t16 = 0; t16 < T; ++t16) sum[t16] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < Unit::kSteps; ++j) {
        const Chunk w = Op::weights(*reinterpret_cast<const uint32_t*>(st + r * Unit::kPitch + 4 * (4 * j + kq)));
#pragma unroll
        for (int t16 = 0; t16 < T; ++t16)
#pragma unroll
          for (int part = 0; part < kParts; ++part) Op::mma(sum[t16], xf[un][j][t16][part], w);
        if (((j + 1) * 32 & ((1 << p.group_lg) - 1)) == 0) {  // a group ends: its scale times its sum
          const float s = scale_stage[wave].s[r][j];
#pragma unroll
          for (int t16 = 0; t16 < T; ++t16)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              acc[half][t16][e] += s * sum[t16][e];
              sum[t16][e] = 0.f;
            }
        }
      }
    }
    wave_lds_order();
  };

  int buf = 0;
#pragma unroll 1
  for (int i = 0; i < most_pairs; ++i) {
    const int pair = pair0 + i;
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int t16 = 0; t16 < T; ++t16) {
        acc[half][t16] = f32x4{0.f, 0.f, 0.f, 0.f};
        if constexpr (kScaled) total[half][t16] = acc[half][t16];
      }
#pragma unroll 1
    for (int turn = 0; turn < p.turns; ++turn) {
      if (i == 0 || p.turns > 1) {
        slice(turn);
        rows_and_ring(pair);
      }
      const bool more = p.turns == 1;
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int un = 0; un < U; ++un) {
          constexpr int kAll = 2 * U;
          const int at = half * U + un;
          if (pair < pair1 && un < nc && last_of(pair, half) >= 0) {
            stage_unit(un, ring[at % D], ring_s[at % D]);
            multiply_unit(half, un);
          }
          if (at + D < kAll)
            load_at(pair, at + D, pair < pair1, at % D);
          else
            load_at(pair + 1, at + D - kAll, more && pair + 1 < pair1, at % D);
        }
      if constexpr (kScaled) {
#pragma unroll
        for (int t16 = 0; t16 < T; ++t16) {
          f32x4 s;
          __builtin_memcpy(&s, &unscale[wave][16 * t16 + 4 * kq], 16);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            total[half][t16] += acc[half][t16] * s;
            acc[half][t16] = f32x4{0.f, 0.f, 0.f, 0.f};
          }
        }
        wave_lds_order();
      }
    }
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int t16 = 0; t16 < T; ++t16)
        if (16 * t16 + 4 * kq < rows) *reinterpret_cast<f32x4*>(&red[buf][wave][half][t16][4 * lane]) = kScaled ? total[kScaled ? half : 0][kScaled ? t16 : 0] : acc[half][t16];
    __syncthreads();
    if (pair < pair1) {
      const int first = cols * p.wk;
      for (int o = along * 64 + lane; o < 256 * T; o += 64 * p.wk) {
        const int m = o / 256 * 16 + 4 * (o >> 6 & 3) + (o & 3), c = o >> 2 & 15;
        if (m >= rows) continue;
        float v[2] = {0.f, 0.f};
        for (int w = 0; w < p.wk; ++w) {
          v[0] += red[buf][first + w][0][o / 256][o & 255];
          v[1] += red[buf][first + w][1][o / 256][o & 255];
        }
        float* out = p.out + tile.rows[m] * p.ld_out;
        if constexpr (PHASE == GROUPED_GATE_UP) {
          const int n = pair * 16 + c;
          if (n < p.N) out[n] = activated(v[0], v[1], p.activation);
        } else {
          if constexpr (PHASE == GROUPED_SHRINK) out += blockIdx.z * p.out_slice;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int n = (2 * pair + half) * 16 + c;
            if (n < p.N) out[n] = v[half];
          }
        }
      }
    }
    buf ^= 1;
  }
}

// A launch of phase, T blocks of 16 rows to a tile and slices of U units; the
// sizes that there are, by phase and weights.
template <int PHASE, int XT, int FMT, int WIDE>
int grouped_sizes(const GroupedParams& p, dim3 grid, int threads, int T, int U, hipStream_t stream) {
#define GT_GROUPED(T_, U_, D_)                                                                                             \
  if (T == T_ && U == U_) {                                                                                                \
    hipLaunchKernelGGL((grouped_kernel<PHASE, XT, FMT, WIDE, T_, U_, D_>), grid, dim3(threads), 0, stream, p);             \
    return hipGetLastError() == hipSuccess ? gt::LS_OK : gt::LS_HIP_ERROR;                                                 \
  }
  if constexpr (FMT == GROUPED_16) {
    if constexpr (PHASE != GROUPED_DOWN) GT_GROUPED(1, 1, 2)
    GT_GROUPED(1, 2, 4)
    GT_GROUPED(1, 4, (PHASE == GROUPED_DOWN ? 2 : 4))
  } else {
    GT_GROUPED(1, 1, 2)
    if constexpr (PHASE != GROUPED_DOWN) GT_GROUPED(1, 2, 4)
  }
#undef GT_GROUPED
  return gt::LS_UNSUPPORTED;
}
template <int XT, int FMT>
int grouped_launch(const GroupedParams& p, dim3 grid, int threads, int phase, int T, int U, hipStream_t stream) {
  if constexpr (FMT == GROUPED_16) {
    switch (phase) {
      case GROUPED_GATE_UP: return grouped_sizes<GROUPED_GATE_UP, XT, FMT, 0>(p, grid, threads, T, U, stream);
      case GROUPED_DOWN: return grouped_sizes<GROUPED_DOWN, XT, FMT, 0>(p, grid, threads, T, U, stream);
      default: return grouped_sizes<GROUPED_SHRINK, XT, FMT, 0>(p, grid, threads, T, U, stream);
    }
  } else {
    if (phase == GROUPED_GATE_UP)
      return p.scale_dtype == DT_F32 ? grouped_sizes<GROUPED_GATE_UP, XT, FMT, 1>(p, grid, threads, T, U, stream)
                                     : grouped_sizes<GROUPED_GATE_UP, XT, FMT, 0>(p, grid, threads, T, U, stream);
    return p.scale_dtype == DT_F32 ? grouped_sizes<GROUPED_DOWN, XT, FMT, 1>(p, grid, threads, T, U, stream)
                                   : grouped_sizes<GROUPED_DOWN, XT, FMT, 0>(p, grid, threads, T, U, stream);
  }
}
// One source file per row type and format defines its launcher.
#define GT_GROUPED_LAUNCHER(name, XT, FMT)                                                                                      \
  int name(const gtk::GroupedParams& p, dim3 grid, int threads, int phase, int T, int U, hipStream_t stream) {                  \
    return gtk::grouped_launch<XT, FMT>(p, grid, threads, phase, T, U, stream);                                                 \
  }

}  // namespace gtk

namespace gt {
typedef int (*GroupedLaunch)(const gtk::GroupedParams&, dim3, int, int, int, int, hipStream_t);
int grouped_bf16(const gtk::GroupedParams& p, dim3 grid, int threads, int phase, int T, int U, hipStream_t stream);
int grouped_f16(const gtk::GroupedParams& p, dim3 grid, int threads, int phase, int T, int U, hipStream_t stream);
int grouped_bf16_int4(const gtk::GroupedParams& p, dim3 grid, int threads, int phase, int T, int U, hipStream_t stream);
int grouped_f16_int4(const gtk::GroupedParams& p, dim3 grid, int threads, int phase, int T, int U, hipStream_t stream);
int grouped_bf16_e2m1(const gtk::GroupedParams& p, dim3 grid, int threads, int phase, int T, int U, hipStream_t stream);
int grouped_f16_e2m1(const gtk::GroupedParams& p, dim3 grid, int threads, int phase, int T, int U, hipStream_t stream);

// How a product's K is dealt out: slices of at most U units, wk waves side by
// side along K, `split` workgroups and `turns` one after another.
struct GroupedCut {
  int U, wk, turns, cols;  // cols: waves side by side along the columns
};
// The rows' tiles that a launch needs workgroups for, whatever the rows name.
inline int64_t most_tiles(int64_t n, int matrices, int rows) { return std::min<int64_t>(n, n / rows + std::min<int64_t>(n, matrices)); }
inline void fill_cut(gtk::GroupedParams& p, const GroupedCut& c, int units, int split) {
  const int slices = c.wk * c.turns * split;
  p.units_each = units / slices;
  p.units_rest = units % slices;
  p.wk = c.wk;
  p.wk_inverse = (65536 + c.wk - 1) / c.wk;
  p.turns = c.turns;
}
}  // namespace gt
