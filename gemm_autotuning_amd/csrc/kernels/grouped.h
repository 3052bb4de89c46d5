// grouped.h -- products of a few gathered rows with the weights that each of
// them names (experts, adapters), on the matrix cores.
//
//   out[row, n] = sum_k x[row, k] * w[of(row), n, k]
//
// Rows that name the same matrix form tiles of 16 (grouped_wide.h: 64).  The
// weights are read once per tile and bound the time (16-bit ones at HBM's rate, 16 tokens
// of 32 experts 4096 x 1024: 103 us, 6.9 TB/s; 4-bit ones by their expansion, 64
// tokens of 64 experts 4096 x 2048: 214 to 224 us, 3.9 TB/s, vector instructions
// under way in 0.65 of a SIMD's time in the first product and 0.53 in the second,
// matrix ones in 0.11 and 0.16); everything is arranged
// around that stream, as for the rows times shared 4-bit weights (w4_mma.h).  A
// wave owns a slice of K, U units of 256 bytes of a 16-bit row (128 of a 4-bit
// one), keeps the rows' slice in registers as operands of 16x16x32 matrix-core
// blocks, and walks pairs of tiles of 16 columns with D units of weights in
// flight.
// A unit's load has neighbouring lanes on consecutive bytes of a column and is
// laid out through an LDS region of the wave's own.  The workgroup's waves
// hold consecutive slices; their sums are joined in LDS, in order, once for B
// pairs of tiles.
//
// The tiles' pairs of columns form one list, of which each workgroup takes an
// even part, about one workgroup to a CU: finding a tile's rows and loading
// them takes 4 us, which workgroups of a few columns each would spend again
// and again (64 tokens of 8 experts each, 64 int4 experts 4096 x 2048: 290 us
// with eight pairs to a workgroup, 220 so).
//
// Nothing is loaded under a condition in that walk (what there is nothing for
// reads one address), so that the wait for a unit leaves the later ones in
// flight.
#pragma once

#include <algorithm>

#include "w4_mma.h"

namespace gtk {

constexpr int kMostRows = 4096;      // of one launch
constexpr int kMostMatrices = 4096;  // counted in LDS
constexpr int kFewRows = 128;        // whose tiles every workgroup finds by itself
constexpr int kMostTileRows = 64;
enum { GROUPED_16 = -1 };            // weights of the rows' type; else W4_INT4, W4_E2M1
enum { GROUPED_GATE_UP = 0, GROUPED_DOWN = 1, GROUPED_SHRINK = 2 };

// A tile of rows: the matrix, how many rows, which.
struct RowTile {
  int matrix, count;
  int rows[kMostTileRows];
};
// All of them, made by the first launch of a call for the others.
struct RowTable {
  int tiles, unused[3];
  RowTile tile[1];
};
inline size_t row_table_bytes(int64_t tiles) { return (16 + (size_t)tiles * sizeof(RowTile) + 255) / 256 * 256; }

// The rows that name matrices, for the search of a tile: row i's matrix is
// index[i / per * ld + i % per], none outside 0..matrices-1.
struct RowIndex {
  const int32_t* index;
  int64_t ld;
  int n, per, matrices;
  uint32_t per_inverse;  // 2^20 / per, rounded up: exact for up to 4096 rows
  int none;  // whether rows without a matrix form tiles too (of matrix `matrices`)
  int bits;  // of the largest matrix's number
  int tile_lg;  // a tile has up to 2^tile_lg rows
};

// Division by a number that the host knows: with floor(2^32 / n) the quotient
// is at most one too small.
struct Divisor {
  uint32_t n, inverse;
};
inline Divisor divisor(uint32_t n) { return Divisor{n, n > 1 ? (uint32_t)((uint64_t{1} << 32) / n) : ~0u}; }
__device__ __forceinline__ uint32_t quotient(const Divisor& d, uint32_t v) {
  const uint32_t q = __umulhi(v, d.inverse);
  return q + (v - q * d.n >= d.n);
}

struct GroupedParams {
  RowIndex ix;
  RowTable* table;
  gt::ExpertWeights w;
  const void* x;       // 16-bit rows (row i of the index is x's row i / per), or the fp32 ones of the first launch
  int64_t ldx;
  float* out;          // fp32, row i at i * ld_out, of slice s of K (not GROUPED_GATE_UP) at s * out_slice
  int64_t ld_out, out_slice;
  int64_t up;          // GROUPED_GATE_UP: the row of w where the second half begins
  int N, K;            // columns (of a half), length
  int scale_dtype, group, activation;
  int units_each, units_rest;  // of a slice of K, a wave's in one turn: the first `rest` have one more
  int wk, cols, turns; // waves side by side along K, and along the columns; times that the x operands are loaded anew
  int split;           // workgroups along K (1 for GROUPED_GATE_UP, whose activation needs whole sums)
  Divisor groups;      // of pairs of column tiles: `cols` of them, one to each wave along the columns
  Divisor of_tile, workgroups;  // items of a tile: split * groups; of the launch
  int wk_inverse;      // 2^16 / wk, rounded up: exact for what is divided (at most 16)
};

// The tiles of rows: rows that name the same matrix, 16 or 64 to a tile.  Up to 128
// rows every workgroup finds by itself: one wave compares all of them at once,
// bit by bit of what they name, and the tiles have the order of their first
// rows.  For more a launch of one workgroup makes the table first (row_tiles.hip).
struct TileSearch {
  int tiles, matrix, count;
  int rows[kMostTileRows];
};
__device__ __forceinline__ int row_of(const RowIndex& ix, int i) { return (int)((uint32_t)i * ix.per_inverse >> 20); }
__device__ __forceinline__ int row_matrix(const RowIndex& ix, int i) {
  const int t = row_of(ix, i);
  const int e = ix.index[(int64_t)t * ix.ld + (i - t * ix.per)];
  return e >= 0 && e < ix.matrices ? e : (ix.none ? ix.matrices : -1);
}
// Two rows to a lane, 64 apart: what they name, their numbers among the rows
// that name it, and the rows that are the first of a tile.
struct FewRows {
  int e[2], rank[2];
  uint64_t leaders[2];
};
__device__ __forceinline__ FewRows few_rows(const RowIndex& ix) {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));  // computed where it is asked for and not kept
  const uint64_t before = (1ull << lane) - 1;
  const int in_tile = (1 << ix.tile_lg) - 1;
  FewRows f;
  f.e[0] = lane < ix.n ? row_matrix(ix, lane) : -1;
  f.e[1] = -1;
  f.rank[1] = 0;
  f.leaders[1] = 0;
  uint64_t first = __ballot(f.e[0] >= 0);
  if (ix.n <= 64) {
    uint64_t same = first;
    for (int b = 0; b < ix.bits; ++b) {
      const bool one = (f.e[0] >> b & 1) != 0;
      const uint64_t v = __ballot(one);
      same &= one ? v : ~v;
    }
    f.rank[0] = __popcll(same & before);
  } else {
    f.e[1] = 64 + lane < ix.n ? row_matrix(ix, 64 + lane) : -1;
    uint64_t same[3] = {first, first, __ballot(f.e[1] >= 0)};  // first in first, second in first, second in second
    for (int b = 0; b < ix.bits; ++b) {
      const bool one[2] = {(f.e[0] >> b & 1) != 0, (f.e[1] >> b & 1) != 0};
      const uint64_t v[2] = {__ballot(one[0]), __ballot(one[1])};
      same[0] &= one[0] ? v[0] : ~v[0];
      same[1] &= one[1] ? v[0] : ~v[0];
      same[2] &= one[1] ? v[1] : ~v[1];
    }
    f.rank[0] = __popcll(same[0] & before);
    f.rank[1] = __popcll(same[1]) + __popcll(same[2] & before);
    f.leaders[1] = __ballot(f.e[1] >= 0 && (f.rank[1] & in_tile) == 0);
  }
  f.leaders[0] = __ballot(f.e[0] >= 0 && (f.rank[0] & in_tile) == 0);
  return f;
}
__device__ __forceinline__ int few_tiles(const FewRows& f) { return __popcll(f.leaders[0]) + __popcll(f.leaders[1]); }
// Tile t of them into LDS, by one wave.
__device__ __forceinline__ void few_tile(const RowIndex& ix, const FewRows& f, int t, TileSearch& s) {
  const int lane = threadIdx.x & 63;
  const uint64_t before = (1ull << lane) - 1;
  const int n0 = __popcll(f.leaders[0]), j = t < n0 ? 0 : 1;
  const uint64_t leaders = f.leaders[j];
  const uint64_t mine = __ballot((leaders >> lane & 1) && __popcll(leaders & before) == t - j * n0);
  const int at = __ffsll((unsigned long long)mine) - 1;
  const int matrix = __builtin_amdgcn_readlane(j ? f.e[1] : f.e[0], at), first = __builtin_amdgcn_readlane(j ? f.rank[1] : f.rank[0], at);
  int n = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bool in = f.e[i] == matrix && f.rank[i] >= first && f.rank[i] < first + (1 << ix.tile_lg);
    if (in) s.rows[f.rank[i] - first] = 64 * i + lane;
    n += __popcll(__ballot(in));
  }
  if (lane == 0) {
    s.matrix = matrix;
    s.count = n;
  }
}

__device__ __forceinline__ float activated(float g, float u, int activation) {
  // GELU's tanh form is g / (1 + exp(-2 z)), z = sqrt(2 / pi) (g + 0.044715 g^3)
  const float z = activation == 0 ? g : 1.5957691216057308f * (g + 0.044715f * g * g * g);
  return g / (1.f + expf(-z)) * u;
}

// An fp32 value as 16-bit operands of the matrix core: take_part takes the
// next one off it and leaves the rest.  bf16's are cut off, eight bits each, and
// three of them are all of the value.  f16's are rounded; two leave at most 2^-22
// of it, or the least subnormal, under a power of two that brings the largest of
// the values in a sum to 2^14..2^15: row_power, the exponent field of that.
// Beside an infinity or NaN it is 2^-114, under which no finite value becomes one.
// The sums hold the power of two until they end: a group of 128 codes is up to
// 2^25 times its scale there, which fp32 has room for below scales of 2^103.
template <int XT>
struct ValueParts {
  static constexpr int n = XT == DT_BF16 ? 3 : 2;
};
template <int XT>
__device__ __forceinline__ uint16_t take_part(float& v) {
  uint16_t part;
  float back;
  if constexpr (XT == DT_BF16) {
    const uint32_t top = __float_as_uint(v) & 0xffff0000u;
    part = (uint16_t)(top >> 16);
    back = __uint_as_float(top);
  } else {
    part = f32_to_f16_bits(v);
    back = f16_bits_to_f32(part);
  }
  const float left = v - back;
  v = left == left ? left : 0.f;  // of an infinity or NaN the first part has it all
  return part;
}
__device__ __forceinline__ uint32_t row_power(uint32_t largest) { return min(253u, 268u - (largest >> 23)); }

// 16 bytes less their first d (d >= 0), zeros behind.
__device__ __forceinline__ u32x4 bytes_from(u32x4 v, int d) {
  unsigned __int128 w;
  __builtin_memcpy(&w, &v, 16);
  w = d < 16 ? w >> (8 * d) : 0;
  __builtin_memcpy(&v, &w, 16);
  return v;
}

// Its first n, zeros behind.
__device__ __forceinline__ u32x4 bytes_upto(u32x4 v, int n) {
  unsigned __int128 w;
  __builtin_memcpy(&w, &v, 16);
  w = n <= 0 ? 0 : (n >= 16 ? w : w << (8 * (16 - n)) >> (8 * (16 - n)));
  __builtin_memcpy(&v, &w, 16);
  return v;
}

template <int FMT, int BYTES>
struct UnitOf {
  static constexpr bool k4 = FMT != GROUPED_16;
  static constexpr int kBytes = BYTES;                // of a column
  static constexpr int kK = k4 ? 2 * BYTES : BYTES / 2;  // k of them
  static constexpr int kLanes = kBytes / 16, kCols = 64 / kLanes, kLoads = 16 / kCols;
  static constexpr int kSteps = kK / 32;              // matrix-core steps
  static constexpr int kRowUnits = kK / 128;          // pieces of 128 elements of a row
  static constexpr int kPitch = kBytes + 16;          // of a column in LDS: reads of 16 columns fall on different banks
};

// A workgroup's part of the list: tile by tile, slice of K by slice, groups of
// columns from g0 on, `left` of them.
struct Part {
  int left, t, slice, g0;
};
__device__ __forceinline__ Part part_of(const GroupedParams& p, int tiles) {
  Part o;
  uint32_t in;
  const uint32_t to_each = p.workgroups.n / (uint32_t)max(tiles, 1);
  if (to_each >= 4) {  // no workgroup has the ends of two tiles, though up to a fifth of them have nothing
    o.t = blockIdx.x / to_each;
    const uint32_t at = blockIdx.x - o.t * to_each, each = p.of_tile.n / to_each, rest = p.of_tile.n - each * to_each;
    in = at * each + min(at, rest);
    o.left = o.t < tiles ? each + (at < rest) : 0;
  } else {
    const uint32_t all = (uint32_t)tiles * p.of_tile.n;
    const uint32_t each = quotient(p.workgroups, all), rest = all - each * p.workgroups.n;
    const uint32_t begin = blockIdx.x * each + min(blockIdx.x, rest);
    o.left = each + (blockIdx.x < rest);
    o.t = quotient(p.of_tile, begin);
    in = begin - o.t * p.of_tile.n;
  }
  o.slice = p.split > 1 ? quotient(p.groups, in) : 0;
  o.g0 = in - o.slice * p.groups.n;
  return o;
}
// The part, and where the workgroups search by themselves its first tile.
__device__ __forceinline__ Part first_part(const GroupedParams& p, bool search, int wave, TileSearch& tile) {
  if (search) {
    if (wave == 0) {
      const FewRows f = few_rows(p.ix);
      const int tiles = few_tiles(f);
      const Part o = part_of(p, tiles);
      if (o.left > 0) few_tile(p.ix, f, o.t, tile);
      if (threadIdx.x == 0) tile.tiles = tiles;
    }
    __syncthreads();
    if (blockIdx.x == 0 && threadIdx.x == 0) p.table->tiles = tile.tiles;
  }
  return part_of(p, __builtin_amdgcn_readfirstlane(search ? tile.tiles : p.table->tiles));
}
// The part's next groups of one tile and slice, and the tile.  found: first_part has found it.
struct Stretch {
  int slice, g0, g1;
};
__device__ __forceinline__ Stretch next_stretch(const GroupedParams& p, bool search, bool found, int wave, Part& part, TileSearch& tile) {
  const int tid = threadIdx.x, t = part.t;
  const Stretch s = {part.slice, part.g0, min((int)p.groups.n, part.g0 + part.left)};
  part.left -= s.g1 - s.g0;
  part.g0 = 0;
  part.slice = s.slice + 1 == p.split ? 0 : s.slice + 1;
  part.t = t + (part.slice == 0);
  if (!found) __syncthreads();  // the last tile's rows are no longer read
  if (search) {
    if (!found) {
      if (wave == 0) few_tile(p.ix, few_rows(p.ix), t, tile);
      __syncthreads();
    }
    if (s.g0 == 0 && s.slice == 0 && tid < 1 << p.ix.tile_lg) {
      RowTile& e = p.table->tile[t];
      if (tid == 0) e.matrix = tile.matrix;
      if (tid == 0) e.count = tile.count;
      e.rows[tid] = tid < tile.count ? tile.rows[tid] : 0;
    }
  } else {
    if (tid < 2 + (1 << p.ix.tile_lg)) (&tile.matrix)[tid] = reinterpret_cast<const int*>(&p.table->tile[t])[tid];
    __syncthreads();
  }
  return s;
}

// What a wave lays out through LDS: weights of a unit (and its scales, a
// column's groups), before that 16 rows' 128 elements.
struct alignas(16) GroupedStage {
  char q[16 * 272];
};
template <int FMT>
struct ScaleStage {
  float s[16][12];
};
template <>
struct ScaleStage<GROUPED_16> {};

// A wave's weights: for group g of columns its pair of tiles of 16, each half
// in units along K, from memory into registers and from there into LDS.
template <int PHASE, int FMT, int BYTES, int G, int WIDE>
struct PairWeights {
  typedef UnitOf<FMT, BYTES> Unit;
  typedef typename std::conditional<WIDE, uint32_t, uint16_t>::type Scale;
  static constexpr int kGroups = Unit::k4 ? Unit::kK / G : 1;  // of a unit
  static constexpr int kScales = kGroups > 4 ? kGroups / 4 : 1;  // of a lane: every fourth
  const GroupedParams& p;
  const int cols, g1, lane, piece, sub;
  const uint32_t row_bytes, ld, s_ldn, s_ldg, lane_q, lane_s, bf16_scales;
  const int scale_groups;
  const char *const wm, *const sm;
  char* const st;
  float (*const ss)[12];
  const int64_t half_columns, pair_columns;
  int c0, nc;  // the slice: its first unit, and how many
  // the next pair to load from: its group, first column's weights and scales
  int load_g;
  const char *load_q, *load_s;

  __device__ __forceinline__ PairWeights(const GroupedParams& p, int matrix, int cols, int g1, int lane, char* st, float (*ss)[12])
      : p(p), cols(cols), g1(g1), lane(lane), piece(lane % Unit::kLanes), sub(lane / Unit::kLanes),
        row_bytes(Unit::k4 ? (p.K + 1) / 2 : 2 * p.K), ld((uint32_t)p.w.ld), s_ldn((uint32_t)p.w.s_ldn * sizeof(Scale)),
        s_ldg((uint32_t)p.w.s_ldg * sizeof(Scale)), lane_q(sub * ld + 16 * piece), lane_s((lane >> 2) * s_ldn + (lane & 3) * s_ldg),
        bf16_scales(p.scale_dtype == DT_BF16 ? ~0u : 0u), scale_groups((p.K + G - 1) / G), wm(p.w.p + matrix * p.w.stride),
        sm(Unit::k4 ? static_cast<const char*>(p.w.scales) + matrix * p.w.s_lde * sizeof(Scale) : nullptr), st(st), ss(ss),
        half_columns(PHASE == GROUPED_GATE_UP ? p.up : 16), pair_columns(p.cols * (PHASE == GROUPED_GATE_UP ? 16 : 32)) {}
  __device__ __forceinline__ void slice(int s) {
    c0 = s * p.units_each + min(s, p.units_rest);
    nc = p.units_each + (s < p.units_rest);
  }
  __device__ __forceinline__ int column_of(int g, int half) const {
    const int pair = g * p.cols + cols;
    return PHASE == GROUPED_GATE_UP ? pair * 16 : (2 * pair + half) * 16;
  }
  // a half's columns less one, below 0 where there is none
  __device__ __forceinline__ int last_of(int g, int half) const {
    return g < g1 && cols < p.cols ? min(p.N - 1 - column_of(g, half), 15) : -1;  // a wave may be left over
  }
  __device__ __forceinline__ void load_from(int g) {
    load_g = g;
    load_q = wm + column_of(g, 0) * p.w.ld;
    load_s = Unit::k4 ? sm + column_of(g, 0) * p.w.s_ldn * (int64_t)sizeof(Scale) : nullptr;
  }
  __device__ __forceinline__ void load_next_pair() {
    ++load_g;
    load_q += pair_columns * p.w.ld;
    if (Unit::k4) load_s += pair_columns * p.w.s_ldn * (int64_t)sizeof(Scale);
  }
  // Unit `un` of a half, or for all lanes one address.  An offset past the
  // half's last piece is cut to that; between a row's end and it there are
  // other rows, whose bytes stage() takes out.
  __device__ __forceinline__ void load(bool any, int half, int un, u32x4 (&q)[Unit::kLoads], Scale (&sc)[kScales]) const {
    const int last = last_of(load_g, half);
    any = any && un < nc && last >= 0;
    const char* const base = any ? load_q + half * half_columns * p.w.ld : wm;
    const uint32_t some = any ? ~0u : 0u, most = (last * ld + row_bytes - 16) & some, from = (uint32_t)(c0 + un) * Unit::kBytes;
#pragma unroll
    for (int i = 0; i < Unit::kLoads; ++i)
      q[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(base + min(lane_q + (i * Unit::kCols * ld + from), most)));
    if constexpr (Unit::k4) {
      const char* const scales = any ? load_s + half * half_columns * p.w.s_ldn * (int64_t)sizeof(Scale) : sm;
      const uint32_t s_most = (last * s_ldn + (scale_groups - 1) * s_ldg) & some;
#pragma unroll
      for (int i = 0; i < kScales; ++i)
        sc[i] = *reinterpret_cast<const Scale*>(scales + min(lane_s + ((c0 + un) * kGroups + 4 * i) * s_ldg, s_most));
    }
  }
  __device__ __forceinline__ void stage(int half_last, int un, u32x4 (&q)[Unit::kLoads], const Scale (&sc)[kScales]) const {
    const uint32_t from = (uint32_t)(c0 + un) * Unit::kBytes;
    if (from + Unit::kBytes > row_bytes) {  // the row ends in it
      const uint32_t most = half_last * ld + row_bytes - 16;
      const int here = (int)(row_bytes - from) - 16 * piece;  // bytes of the lane's 16 that are the row's
#pragma unroll
      for (int i = 0; i < Unit::kLoads; ++i) {
        const uint32_t want = lane_q + (i * Unit::kCols * ld + from);
        q[i] = bytes_upto(bytes_from(q[i], want > most ? (int)min(want - most, 16u) : 0), here);
      }
    }
#pragma unroll
    for (int i = 0; i < Unit::kLoads; ++i)
      *reinterpret_cast<u32x4*>(st + (i * Unit::kCols + sub) * Unit::kPitch + 16 * piece) = q[i];
    if constexpr (Unit::k4) {
#pragma unroll
      for (int i = 0; i < kScales; ++i) {
        Scale b = sc[i];
        asm volatile("" : "+v"(b));  // converted here and not where it was loaded, which would wait for it there
        float f;
        if constexpr (WIDE)
          f = __uint_as_float(b);
        else  // both conversions and a selection by bits
          f = __uint_as_float(((uint32_t)b << 16 & bf16_scales) | (__float_as_uint(f16_bits_to_f32(b)) & ~bf16_scales));
        const int g = (c0 + un) * kGroups + 4 * i + (lane & 3);
        ss[lane >> 2][4 * i + (lane & 3)] = g < scale_groups ? f : 0.f;  // past K: nothing, whatever the last scale is
      }
    }
    wave_lds_order();
  }
};

// BYTES: a unit's of a column; G: a group's k and WIDE: its scale is fp32 (4
// bits); ONE: the slices are loaded once a tile (K in one turn); W: waves.
template <int PHASE, int XT, int FMT, int BYTES, int G, int WIDE, int U, int D, int B, int W, bool ONE>
__global__ __launch_bounds__(64 * W, 2) void grouped_kernel(GroupedParams p) {
  typedef UnitOf<FMT, BYTES> Unit;
  typedef PairWeights<PHASE, FMT, BYTES, G, WIDE> Weights;
  typedef W4Operand<XT, FMT == GROUPED_16 ? W4_E2M1 : FMT> Op;  // e2m1: elements in order
  constexpr int kGroups = Weights::kGroups;
  // with a group to 128 k a lane takes its 32 of them as they lie, eight to a step; else a step's 32 k are of one group
  constexpr bool kPieces = Unit::k4 && G == 128;
  constexpr bool kSplit = PHASE == GROUPED_DOWN;  // fp32 rows, in parts
  constexpr int kParts = kSplit ? ValueParts<XT>::n : 1;
  constexpr bool kScaled = kSplit && XT == DT_F16;
  static_assert(ONE || !kScaled, "turns whose rows have scales of their own");
  constexpr int kAll = 2 * U;  // units of a pair
  static_assert((B * kAll) % D == 0 && (ONE || D <= B * kAll), "places in the ring are known when compiled");
  __shared__ TileSearch tile;
  __shared__ GroupedStage stages[W];
  __shared__ ScaleStage<Unit::k4 ? FMT : W4_INT4> scale_stage[Unit::k4 ? W : 1];
  // the waves' sums of B pairs; with one pair at a time two buffers take turns, and one barrier is enough
  constexpr int kBuffers = B == 1 ? 2 : B;
  __shared__ float red[kBuffers][W][2][256];
  __shared__ float unscale[kScaled ? W : 1][16];

  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const bool search = PHASE != GROUPED_DOWN && p.ix.n <= kFewRows;  // else there is a table
  Part part = first_part(p, search, wave, tile);
  // this wave's slice of K and its columns
  const int cols = (wave * p.wk_inverse) >> 16, along = wave - cols * p.wk;
  char* const st = stages[wave].q;
  int buf = 0;

  for (bool found = search; part.left > 0; found = false) {
    const Stretch stretch = next_stretch(p, search, found, wave, part, tile);
    const int g0 = stretch.g0, g1 = stretch.g1;
    const int matrix = __builtin_amdgcn_readfirstlane(tile.matrix);
    if (matrix >= p.ix.matrices) continue;
    const int rows = __builtin_amdgcn_readfirstlane(tile.count);
    int lane = tid & 63;
    asm volatile("" : "+v"(lane));  // what follows from it is not kept over the search above
    const int r = lane & 15, kq = lane >> 4;
    Weights w(p, matrix, cols, g1, lane, st, scale_stage[Unit::k4 ? wave : 0].s);
    auto slice = [&](int turn) { w.slice((stretch.slice * p.turns + turn) * p.wk + along); };

    // ---- rows, as operands: [unit][step][part]
    Chunk xf[U][Unit::kSteps][kParts];
    auto row_at = [&](int m) { return tile.rows[min(m, rows - 1)]; };
    auto load_rows16 = [&](u32x4 (&raw)[U * Unit::kRowUnits][4]) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (4 * i < rows) {
          const int row = row_at(4 * i + kq);
          const uint16_t* x = static_cast<const uint16_t*>(p.x) + row_of(p.ix, row) * p.ldx;
#pragma unroll
          for (int un = 0; un < U * Unit::kRowUnits; ++un) {
            const int k = (w.c0 * Unit::kRowUnits + un) * 128 + 8 * r;
            raw[un][i] = *reinterpret_cast<const u32x4_any*>(x + min(k, p.K - 8));
          }
        }
    };
    auto place_rows16 = [&](u32x4 (&raw)[U * Unit::kRowUnits][4]) __attribute__((always_inline)) {
#pragma unroll
      for (int un = 0; un < U * Unit::kRowUnits; ++un) {
        const int k0 = (w.c0 * Unit::kRowUnits + un) * 128;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (4 * i < rows) {
            u32x4 v = raw[un][i];
            if (k0 + 128 > p.K) v = bytes_from(v, max(0, 2 * (k0 + 8 * r - (p.K - 8))));
            *reinterpret_cast<u32x4*>(st + (4 * i + kq) * 272 + 16 * r) = v;
          }
        wave_lds_order();
#pragma unroll
        for (int j = 0; j < 4; ++j)
          xf[un / Unit::kRowUnits][un % Unit::kRowUnits * 4 + j][0] =
              Op::order(*reinterpret_cast<const u32x4*>(st + r * 272 + 16 * (kPieces ? 4 * kq + j : 4 * j + kq)));
        wave_lds_order();
      }
    };
    // fp32 rows: 32 lanes to a row's 128 elements, two rows to a load
    auto load_rows32 = [&](f32x4 (&raw)[U * Unit::kRowUnits][8]) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (2 * i < rows) {
          const float* x = static_cast<const float*>(p.x) + row_at(2 * i + (lane >> 5)) * p.ldx;
#pragma unroll
          for (int un = 0; un < U * Unit::kRowUnits; ++un) {
            const int k = (w.c0 * Unit::kRowUnits + un) * 128 + 4 * (lane & 31);
            raw[un][i] = *reinterpret_cast<const f32x4*>(x + min(k, (p.K - 1) & ~3));
          }
        }
    };
    auto place_rows32 = [&](f32x4 (&raw)[U * Unit::kRowUnits][8]) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (2 * i < rows) {
          uint32_t most = 0;
#pragma unroll
          for (int un = 0; un < U * Unit::kRowUnits; ++un) {
            const int k = (w.c0 * Unit::kRowUnits + un) * 128 + 4 * (lane & 31);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (k + e >= p.K || un >= w.nc * Unit::kRowUnits) raw[un][i][e] = 0.f;
              most = max(most, __float_as_uint(raw[un][i][e]) & 0x7fffffffu);
            }
          }
          if constexpr (kScaled) {
            // the row's power of two, of this slice
            auto largest = [](uint32_t a, uint32_t b) { return max(a, b); };
            most = largest(most, dpp<0xB1>(most));
            most = largest(most, dpp<0x4E>(most));
            most = largest(most, dpp<0x141>(most));
            most = largest(most, dpp<0x140>(most));
            const auto both = __builtin_amdgcn_permlane16_swap(most, most, false, false);
            most = largest(both[0], both[1]);
            const uint32_t to = row_power(most);
            if ((lane & 31) == 0) unscale[wave][2 * i + (lane >> 5)] = __uint_as_float((254u - to) << 23);
            const float s = __uint_as_float(to << 23);
#pragma unroll
            for (int un = 0; un < U * Unit::kRowUnits; ++un) raw[un][i] *= s;
          }
        }
#pragma unroll
      for (int un = 0; un < U * Unit::kRowUnits; ++un)
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (2 * i < rows) {
              f32x4 v = raw[un][i];
              uint16_t h[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float rest = v[e];
                h[e] = take_part<XT>(rest);
                v[e] = rest;
              }
              raw[un][i] = v;
              __builtin_memcpy(st + (2 * i + (lane >> 5)) * 272 + 8 * (lane & 31), h, 8);
            }
          wave_lds_order();
#pragma unroll
          for (int j = 0; j < 4; ++j)
            xf[un / Unit::kRowUnits][un % Unit::kRowUnits * 4 + j][part] =
                Op::order(*reinterpret_cast<const u32x4*>(st + r * 272 + 16 * (kPieces ? 4 * kq + j : 4 * j + kq)));
          wave_lds_order();
        }
    };

    u32x4 ring[D][Unit::kLoads];
    typename Weights::Scale ring_s[D][Weights::kScales];
    // the unit `at` places after a pair's first (a half's U units, then the other's), in order
    auto load_at = [&](int at, bool any, int place) __attribute__((always_inline)) {
      w.load(any, at / U, at % U, ring[place], ring_s[place]);
      if (at == kAll - 1) w.load_next_pair();
    };
    // the rows' slice, and the ring from group g on
    auto rows_and_ring = [&](int g) __attribute__((always_inline)) {
      auto fill = [&]() __attribute__((always_inline)) {
        w.load_from(g);
#pragma unroll
        for (int d = 0; d < D; ++d) load_at(d % kAll, true, d);
      };
      if constexpr (kSplit) {
        f32x4 raw[U * Unit::kRowUnits][8];
        load_rows32(raw);
        fill();
        place_rows32(raw);
      } else {
        u32x4 raw[U * Unit::kRowUnits][4];
        load_rows16(raw);
        fill();
        place_rows16(raw);
      }
    };

    f32x4 acc[B][2];
    auto multiply_unit = [&](f32x4& acc, int un) __attribute__((always_inline)) {
      if constexpr (!Unit::k4) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          Chunk v;
          __builtin_memcpy(&v, st + r * Unit::kPitch + 16 * (4 * j + kq), 16);
#pragma unroll
          for (int part = 0; part < kParts; ++part) Op::mma(acc, xf[un][j][part], v);
        }
      } else {
        uint32_t v[Unit::kSteps];
        if constexpr (kPieces) {
#pragma unroll
          for (int c = 0; c < Unit::kSteps / 4; ++c) __builtin_memcpy(&v[4 * c], st + r * Unit::kPitch + 16 * (4 * c + kq), 16);
        } else {
#pragma unroll
          for (int j = 0; j < Unit::kSteps; ++j) __builtin_memcpy(&v[j], st + r * Unit::kPitch + 4 * (4 * j + kq), 4);
        }
        float sc[kGroups];
#pragma unroll
        for (int g = 0; g < kGroups; ++g) sc[g] = w.ss[r][g];
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          f32x4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = g * (G / 32); j < (g + 1) * (G / 32); ++j) {
            const Chunk e = Op::weights(v[j]);
#pragma unroll
            for (int part = 0; part < kParts; ++part) Op::mma(sum, xf[un][j][part], e);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[e] += sc[g] * sum[e];
        }
      }
      wave_lds_order();
    };

    if constexpr (ONE) {
      slice(0);
      rows_and_ring(g0);
    }
#pragma unroll 1
    for (int g = g0; g < g1; g += B) {
#pragma unroll
      for (int b = 0; b < B; ++b)
#pragma unroll
        for (int half = 0; half < 2; ++half) acc[b][half] = f32x4{0.f, 0.f, 0.f, 0.f};
      const int turns = ONE ? 1 : p.turns;
#pragma unroll 1
      for (int turn = 0; turn < turns; ++turn) {
        if constexpr (!ONE) {
          slice(turn);
          rows_and_ring(g);
        }
#pragma unroll
        for (int b = 0; b < B; ++b)
#pragma unroll
          for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int un = 0; un < U; ++un) {
              const int at = b * kAll + half * U + un;
              const int last = w.last_of(g + b, half);
              if (un < w.nc && last >= 0) {
                w.stage(last, un, ring[at % D], ring_s[at % D]);
                multiply_unit(acc[b][half], un);
              }
              load_at((at + D) % kAll, ONE || at + D < B * kAll, at % D);
            }
      }
      if constexpr (B > 1) __syncthreads();  // the last sums have been read
      if (4 * kq < rows) {
        f32x4 s = {1.f, 1.f, 1.f, 1.f};
        if constexpr (kScaled) __builtin_memcpy(&s, &unscale[wave][4 * kq], 16);
#pragma unroll
        for (int b = 0; b < B; ++b)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            f32x4 v = acc[b][half];
            if constexpr (kScaled) v *= s;
            *reinterpret_cast<f32x4*>(&red[B == 1 ? buf : b][wave][half][4 * lane]) = v;
          }
      }
      __syncthreads();
      if (cols < p.cols) {
        const int first = cols * p.wk;
        for (int o = along * 64 + lane; o < 256 * B; o += 64 * p.wk) {
          const int b = o >> 8, m = 4 * (o >> 6 & 3) + (o & 3), c = o >> 2 & 15, pair = (g + b) * p.cols + cols;
          if (m >= rows || g + b >= g1) continue;
          const float* at = &red[B == 1 ? buf : b][first][0][o & 255];
          float v[2] = {0.f, 0.f};
#pragma unroll
          for (int w0 = 0; w0 < W; w0 += 4) {
            float part[4][2];
#pragma unroll
            for (int v4 = 0; v4 < 4; ++v4)
#pragma unroll
              for (int half = 0; half < 2; ++half) part[v4][half] = at[min(w0 + v4, p.wk - 1) * 512 + half * 256];
#pragma unroll
            for (int v4 = 0; v4 < 4; ++v4)
#pragma unroll
              for (int half = 0; half < 2; ++half) v[half] += w0 + v4 < p.wk ? part[v4][half] : 0.f;
          }
          float* out = p.out + tile.rows[m] * p.ld_out;
          if constexpr (PHASE == GROUPED_GATE_UP) {
            const int n = pair * 16 + c;
            if (n < p.N) out[n] = activated(v[0], v[1], p.activation);
          } else {
            out += stretch.slice * p.out_slice;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const int n = (2 * pair + half) * 16 + c;
              if (n < p.N) out[n] = v[half];
            }
          }
        }
      }
      if constexpr (B == 1) buf ^= 1;
    }
  }
}

// A launch with K cut as `c` says, among the sizes that there are.
struct GroupedCut {
  int U, wk, cols, turns, waves;  // cols: waves side by side along the columns; waves: of a workgroup
};
template <int PHASE, int XT, int FMT, int G, int WIDE>
int grouped_sizes(const GroupedParams& p, const GroupedCut& c, hipStream_t stream) {
#define GT_GROUPED(BYTES_, U_, D_, B_, W_, ONE_)                                                                               \
  if (c.U == U_ && c.waves == W_ && (c.turns == 1) == ONE_) {                                                                  \
    hipLaunchKernelGGL((grouped_kernel<PHASE, XT, FMT, BYTES_, G, WIDE, U_, D_, B_, W_, ONE_>), dim3(p.workgroups.n), dim3(64 * W_), 0, \
                       stream, p);                                                                                             \
    return hipGetLastError() == hipSuccess ? gt::LS_OK : gt::LS_HIP_ERROR;                                                     \
  }
  // bytes of a unit, U, D, B, waves, K in one turn
  if constexpr (FMT == GROUPED_16) {
    constexpr int D = PHASE == GROUPED_DOWN ? 2 : 4;
    constexpr bool kThree = PHASE == GROUPED_DOWN && ValueParts<XT>::n == 3;  // rows' parts: registers for two units
    if constexpr (PHASE == GROUPED_SHRINK) GT_GROUPED(256, 1, 2, 1, 8, true)
    if constexpr (PHASE == GROUPED_SHRINK || kThree) GT_GROUPED(256, 2, 4, 1, 8, true)
    if constexpr (!kThree) GT_GROUPED(256, 4, D, 1, 8, true)
    if constexpr (PHASE == GROUPED_GATE_UP) GT_GROUPED(256, 4, 4, 2, 8, false)
    if constexpr (PHASE == GROUPED_SHRINK) GT_GROUPED(256, 4, 4, 1, 8, false)
    if constexpr (PHASE != GROUPED_SHRINK) {
      GT_GROUPED(256, 2, 4, 1, 4, true)
      if constexpr (!kThree) GT_GROUPED(256, 4, D, 1, 4, true)
    }
  } else if constexpr (PHASE == GROUPED_DOWN) {
    GT_GROUPED(128, 1, 2, 2, 8, true)
  } else {
    GT_GROUPED(128, 2, 4, 2, 8, true)
    GT_GROUPED(128, 2, 4, 4, 8, false)
  }
#undef GT_GROUPED
  return gt::LS_UNSUPPORTED;
}
template <int PHASE, int XT, int FMT>
int grouped_scales(const GroupedParams& p, const GroupedCut& c, hipStream_t stream) {
  const bool wide = p.scale_dtype == DT_F32;
#define GT_GROUPED_G(G_)                                                                       \
  return wide ? grouped_sizes<PHASE, XT, FMT, G_, 1>(p, c, stream)                 \
              : grouped_sizes<PHASE, XT, FMT, G_, 0>(p, c, stream)
  switch (p.group) {
    case 32: GT_GROUPED_G(32);
    case 64: GT_GROUPED_G(64);
    default: GT_GROUPED_G(128);
  }
#undef GT_GROUPED_G
}
template <int XT, int FMT>
int grouped_launch(const GroupedParams& p, int phase, const GroupedCut& c, hipStream_t stream) {
  if constexpr (FMT == GROUPED_16) {
    switch (phase) {
      case GROUPED_GATE_UP: return grouped_sizes<GROUPED_GATE_UP, XT, FMT, 128, 0>(p, c, stream);
      case GROUPED_DOWN: return grouped_sizes<GROUPED_DOWN, XT, FMT, 128, 0>(p, c, stream);
      default: return grouped_sizes<GROUPED_SHRINK, XT, FMT, 128, 0>(p, c, stream);
    }
  } else {
    if (phase == GROUPED_GATE_UP) return grouped_scales<GROUPED_GATE_UP, XT, FMT>(p, c, stream);
    if constexpr (XT == DT_F16) return grouped_scales<GROUPED_DOWN, XT, FMT>(p, c, stream);  // for either type of x
    return gt::LS_UNSUPPORTED;
  }
}
// One source file per row type and format defines its launcher.
#define GT_GROUPED_LAUNCHER(name, XT, FMT)                                                                                        \
  int name(const gtk::GroupedParams& p, int phase, const gtk::GroupedCut& c, hipStream_t stream) {                \
    return gtk::grouped_launch<XT, FMT>(p, phase, c, stream);                                                         \
  }

}  // namespace gtk

namespace gt {
typedef int (*GroupedLaunch)(const gtk::GroupedParams&, int, const gtk::GroupedCut&, hipStream_t);
int grouped_bf16(const gtk::GroupedParams& p, int phase, const gtk::GroupedCut& c, hipStream_t stream);
int grouped_f16(const gtk::GroupedParams& p, int phase, const gtk::GroupedCut& c, hipStream_t stream);
int grouped_bf16_int4(const gtk::GroupedParams& p, int phase, const gtk::GroupedCut& c, hipStream_t stream);
int grouped_f16_int4(const gtk::GroupedParams& p, int phase, const gtk::GroupedCut& c, hipStream_t stream);
int grouped_bf16_e2m1(const gtk::GroupedParams& p, int phase, const gtk::GroupedCut& c, hipStream_t stream);
int grouped_f16_e2m1(const gtk::GroupedParams& p, int phase, const gtk::GroupedCut& c, hipStream_t stream);

// The table of the tiles (row_tiles.hip), for rows that the workgroups do not
// search by themselves.
int launch_row_tiles(const gtk::RowIndex& ix, gtk::RowTable* table, hipStream_t stream);

// The rows' tiles that there can be, whatever the rows name.
inline int64_t most_tiles(int64_t n, int matrices, int rows = 16) {
  return std::min<int64_t>(n, n / rows + std::min<int64_t>(n, matrices));
}
inline void fill_cut(gtk::GroupedParams& p, const gtk::GroupedCut& c, int units, int split) {
  const int slices = c.wk * c.turns * split;
  p.units_each = units / slices;
  p.units_rest = units % slices;
  p.wk = c.wk;
  p.wk_inverse = (65536 + c.wk - 1) / c.wk;
  p.cols = c.cols;
  p.turns = c.turns;
  p.split = split;
}
// The list of at most `tiles` tiles' groups of columns, and the workgroups for
// it, `at_once` of which run at once; 0 where the list is too long.
inline int fill_list(gtk::GroupedParams& p, int64_t tiles, int groups, int64_t at_once) {
  const int64_t of_tile = (int64_t)groups * p.split;
  if (of_tile * tiles >= (INT64_C(1) << 31)) return 0;
  const int64_t n = std::min(tiles * of_tile, at_once);
  p.groups = gtk::divisor((uint32_t)groups);
  p.of_tile = gtk::divisor((uint32_t)of_tile);
  p.workgroups = gtk::divisor((uint32_t)n);
  return (int)n;
}
inline int bits_of(int n) { return 32 - __builtin_clz((unsigned)n | 1u); }
}  // namespace gt
