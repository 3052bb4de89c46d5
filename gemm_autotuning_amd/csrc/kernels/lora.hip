// lora.hip -- adapters of many requests beside a shared projection: the first
// product of each row (grouped.h, slices of K to workgroups where the rows are
// few) into fp32 values, then the second one, which adds the slices, and the
// base to its results; few rows of small adapters in one launch; the first
// product row by row, or in tiles of 64 rows, where that is less.
#include "elements.h"
#include "grouped.h"
#include "launchers.h"
#include "row_tiles.h"

namespace gtk {

struct ExpandParams {
  gt::LoraArgs a;
  const RowTable* table;
  const float* mid;  // slice s, row m, rank r at (s * M + m) * ld + r
  int64_t ld, slice;
  int slices, blocks, blocks_each;  // blocks of 64 columns; of a wave
  int parts_lg;                     // a tile of the table is 2^parts_lg of 16 rows
};

// A piece that is used once.
template <int DT>
__device__ __forceinline__ void load_past_caches(const typename Elem<DT>::T* p, Piece<DT, 8>& b) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(b.w) / 16; ++i) {
    const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(p) + i);
    __builtin_memcpy(b.w + 4 * i, &v, 16);
  }
}

// The second product: a wave holds the tile's 16 rows of up to 32 R values as
// operands in 16-bit parts (ValueParts) and walks blocks of 64 columns, whose weights
// (64 rows of the rank) it loads a block ahead.  What bounds it is the weights
// with few rows (48 rows of 64 adapters rank 64, 16384 columns: 16 us, 4.4 TB/s)
// and base and y with many (4096 rows, 4096 columns bf16: 19 us, 3.5 TB/s); the
// results go through LDS so that a row's 64 columns are read and written by
// eight lanes.  PAST: base and y pass by the caches.  The waves to a SIMD are
// held to what the registers allow without spilling (4096 rows of 6 adapters rank
// 64: 45 us with four, 52 with three, which the compiler takes by itself).
template <int XT, int OUT, int R, bool NARROW, bool PAST>
__global__ __launch_bounds__(256, R == 1 ? 5 : (R == 2 ? 4 : 1)) void lora_expand_kernel(ExpandParams p) {
  typedef W4Rows<XT> Op;
  typedef typename Elem<OUT>::T TO;
  constexpr int kPitch = 68;  // floats of a row of results in LDS
  constexpr int kParts = ValueParts<XT>::n;
  __shared__ RowTile tile;
  __shared__ float h[16][32 * R + 4];
  __shared__ float out[4][16][kPitch];
  const gt::LoraArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, kq = lane >> 4;
  const int t = blockIdx.y >> p.parts_lg, row0 = 16 * (blockIdx.y - (t << p.parts_lg));
  if (t >= p.table->tiles) return;
  const RowTile& whole_tile = p.table->tile[t];
  if (tid < 16) tile.rows[tid] = whole_tile.rows[row0 + tid];
  if (tid == 16) tile.matrix = whole_tile.matrix;
  if (tid == 17) tile.count = whole_tile.count;
  __syncthreads();
  const int matrix = __builtin_amdgcn_readfirstlane(tile.matrix);
  const int rows = min(__builtin_amdgcn_readfirstlane(tile.count) - row0, 16);
  if (rows <= 0) return;
  const bool some = matrix < a.adapters;
  const int block0 = (blockIdx.x * 4 + wave) * p.blocks_each, block1 = min(block0 + p.blocks_each, p.blocks);

  const char* const wb = a.b.p + (some ? matrix : 0) * a.b.stride;
  typedef __attribute__((ext_vector_type(4))) uint32_t Raw;
  // weights of 16 columns: a column's 8 values of each step of 32
  auto load_weights = [&](int64_t n0, Raw (&w)[R]) __attribute__((always_inline)) {
    const int64_t n = min(n0 + r, a.N - 1);
    const uint16_t* row = reinterpret_cast<const uint16_t*>(wb + n * a.b.ld);
    if constexpr (NARROW) {
      uint16_t v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = kq == 0 && e < a.rank ? row[min(e, a.rank - 1)] : 0;
      __builtin_memcpy(&w[0], v, 16);
    } else {
#pragma unroll
      for (int j = 0; j < R; ++j) w[j] = *reinterpret_cast<const u32x4_any*>(row + min(32 * j + 8 * kq, a.rank - 8));
    }
  };
  auto place_weights = [&](Raw (&w)[R], Chunk (&f)[R]) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < R; ++j) {
      Raw v = w[j];
      if (!NARROW && 32 * (j + 1) > a.rank) v = bytes_from(v, max(0, 2 * (32 * j + 8 * kq - (a.rank - 8))));
      __builtin_memcpy(&f[j], &v, 16);
    }
  };
  Raw raw[4][R];
  if (some && block0 < block1)
#pragma unroll
    for (int c = 0; c < 4; ++c) load_weights(64 * (int64_t)block0 + 16 * c, raw[c]);

  // the rows' values: the slices' sums, in order
  Chunk x[R][kParts];
  float back[4] = {1.f, 1.f, 1.f, 1.f};  // of this lane's four rows of results
  if (some) {
    for (int i = tid; i < 16 * 32 * R; i += 256) {
      const int m = i / (32 * R), k = i % (32 * R);
      float v = 0.f;
      if (m < rows && k < a.rank) {
        const float* at = p.mid + tile.rows[m] * p.ld + k;
        for (int s0 = 0; s0 < p.slices; s0 += 4) {
          float part[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) part[j] = at[min(s0 + j, p.slices - 1) * p.slice];
#pragma unroll
          for (int j = 0; j < 4; ++j) v += s0 + j < p.slices ? part[j] : 0.f;
        }
      }
      h[m][k] = v;
    }
    __syncthreads();
    float v[R][8];
    uint32_t most = 0;
#pragma unroll
    for (int j = 0; j < R; ++j) {
      __builtin_memcpy(v[j], &h[r][32 * j + 8 * kq], 32);
#pragma unroll
      for (int e = 0; e < 8; ++e) most = max(most, __float_as_uint(v[j][e]) & 0x7fffffffu);
    }
    if constexpr (XT == DT_F16) {
      // the row's power of two
      const auto half = __builtin_amdgcn_permlane16_swap(most, most, false, false);
      most = max(half[0], half[1]);
      const auto both = __builtin_amdgcn_permlane32_swap(most, most, false, false);
      most = max(both[0], both[1]);
      const uint32_t to = row_power(most);
      const float s = __uint_as_float(to << 23);
#pragma unroll
      for (int j = 0; j < R; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] *= s;
#pragma unroll
      for (int e = 0; e < 4; ++e) back[e] = __shfl(__uint_as_float((254u - to) << 23), 4 * kq + e);
    }
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
      for (int part = 0; part < kParts; ++part) {
        uint16_t b[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) b[e] = take_part<XT>(v[j][e]);
        __builtin_memcpy(&x[j][part], b, 16);
      }
  }
  const float scale = some && a.scale ? a.scale[matrix] : 1.f;

  const int pass_row = lane >> 3, col = 8 * (lane & 7);
  for (int block = block0; block < block1; ++block) {
    const int64_t n0 = 64 * (int64_t)block;
    const bool whole = n0 + 64 <= a.N;
    float v[2][8];  // of rows pass_row and pass_row + 8: the base
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
      const int m = pass_row + 8 * i;
      if (a.base && m < rows) {
        const TO* at = static_cast<const TO*>(a.base) + tile.rows[m] * a.ldb + n0 + col;
        if (whole) {
          Piece<OUT, 8> b;
          if constexpr (PAST)
            load_past_caches<OUT>(at, b);
          else
            b.load(at);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[i][e] = b.get(e);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (n0 + col + e < a.N) v[i][e] = Elem<OUT>::get(at[e]);
        }
      }
    }
    if (some) {
      Chunk f[4][R];
#pragma unroll
      for (int c = 0; c < 4; ++c) place_weights(raw[c], f[c]);
      if (block + 1 < block1)
#pragma unroll
        for (int c = 0; c < 4; ++c) load_weights(n0 + 64 + 16 * c, raw[c]);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < R; ++j)
#pragma unroll
          for (int part = 0; part < kParts; ++part) Op::mma(acc, x[j][part], f[c][j]);
#pragma unroll
        for (int e = 0; e < 4; ++e) out[wave][4 * kq + e][16 * c + r] = acc[e] * back[e] * scale;
      }
      wave_lds_order();
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int m = pass_row + 8 * i;
      if (m < rows) {
        if (some) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[i][e] += out[wave][m][col + e];
        }
        TO* at = static_cast<TO*>(a.y) + tile.rows[m] * a.ldy + n0 + col;
        if (whole) {
          store_piece<OUT, 8>(at, v[i], PAST);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (n0 + col + e < a.N) at[e] = Elem<OUT>::put(v[i][e]);
        }
      }
    }
    wave_lds_order();
  }
}

// The first product of many rows: a workgroup to a tile of 64 rows and a slice
// of K, of which it takes 128 a step, the rows' and the matrix' pieces in LDS (two
// buffers in turn) and four steps of them in flight in registers.  Its waves
// are four blocks of 16 rows times two halves of the rank.  Against tiles of 16
// (grouped.h) the matrix is read a quarter as often: 4096 rows 4096 long, rank
// 32, 11.8 us for 34 MB where those take 17.9, of which the table's read, the
// rows' first load and the launch are some 6.
template <int XT, int C>
__global__ __launch_bounds__(512, 2) void lora_many_kernel(gt::LoraArgs a, const RowTable* table, float* mid, int64_t ld, int64_t slice_ld,
                                                           int split) {
  typedef W4Rows<XT> Op;
  constexpr int kPitch = 272, kAhead = 4, kLoads = 2 + C;
  __shared__ RowTile tile;
  __shared__ alignas(16) char lds[2][(64 + 32 * C) * kPitch];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, kq = lane >> 4, K = (int)a.K;
  if ((int)blockIdx.y >= table->tiles) return;
  if (tid < 2 + 64) reinterpret_cast<int*>(&tile)[tid] = reinterpret_cast<const int*>(&table->tile[blockIdx.y])[tid];
  __syncthreads();
  const int matrix = __builtin_amdgcn_readfirstlane(tile.matrix), rows = __builtin_amdgcn_readfirstlane(tile.count);
  if (matrix >= a.adapters) return;
  const int units = (K + 127) / 128, each = units / split, rest = units - each * split, slice = blockIdx.x;
  const int first = slice * each + min(slice, rest), steps = each + (slice < rest);
  // a piece is 16 bytes: of rows tid / 16 and 32 more, of the matrix' rows likewise
  const char* from[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i)
    from[i] = i < 2 ? static_cast<const char*>(a.x) + tile.rows[min(tid / 16 + 32 * i, rows - 1)] * a.ldx * 2
                    : a.a.p + matrix * a.a.stride + min(tid / 16 + 32 * (i - 2), a.rank - 1) * a.a.ld;
  u32x4 ring[kAhead][kLoads];
  auto load = [&](int step, u32x4 (&v)[kLoads]) __attribute__((always_inline)) {
    const int k = (first + min(step, steps - 1)) * 128 + 8 * (tid & 15);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) v[i] = *reinterpret_cast<const u32x4_any*>(from[i] + 2 * min(k, K - 8));
  };
  auto place = [&](int step, u32x4 (&v)[kLoads], char* at) __attribute__((always_inline)) {
    const int k0 = (first + step) * 128, k = k0 + 8 * (tid & 15);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      if (k0 + 128 > K) v[i] = bytes_from(v[i], min(max(0, 2 * (k - (K - 8))), 16));
      *reinterpret_cast<u32x4*>(at + (tid / 16 + 32 * i) * kPitch + 16 * (tid & 15)) = v[i];
    }
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) load(i, ring[i]);
  const int block = wave & 3, half = wave >> 2;
  f32x4 acc[C];
#pragma unroll
  for (int c = 0; c < C; ++c) acc[c] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int n = 0; n < steps; n += kAhead)
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (n + i >= steps) break;
      char* const at = lds[i & 1];
      place(n + i, ring[i], at);
      load(n + i + kAhead, ring[i]);
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        Chunk x, w;
        __builtin_memcpy(&x, at + (16 * block + r) * kPitch + 64 * j + 16 * kq, 16);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          __builtin_memcpy(&w, at + (64 + 16 * (C * half + c) + r) * kPitch + 64 * j + 16 * kq, 16);
          Op::mma(acc[c], x, w);
        }
      }
    }
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int m = 16 * block + 4 * kq + e, n = 16 * (C * half + c) + r;
      if (m < rows && n < a.rank) mid[slice * slice_ld + tile.rows[m] * ld + n] = acc[c][e];
    }
}

constexpr int kFewThreads = 1024;

// A few rows of small adapters in one launch: every workgroup computes its row's
// first product anew, its waves along the rank and K (16 bytes of a row of a to
// a lane, 16 rows at once), and then 1024 columns of the second, one to a
// thread, whose rows of b it has loaded meanwhile.  All in fp32.  It is a chain
// of waits (the adapter's number, its weights, two barriers) rather than of
// bytes: one row of rank 16, 4096 x 4096, 5.5 us for 0.3 MB; 77 rows of rank 12, 1001 x 999,
// 5.6 us where the tiles' two launches take 11.6.
template <int XT>
__global__ __launch_bounds__(kFewThreads) void lora_few_kernel(gt::LoraArgs a) {
  constexpr int kRows = 16, kEach = 4, kWaves = kFewThreads / 64;
  __shared__ float sums[kWaves][256], h[256];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t m = blockIdx.y, n = (int64_t)blockIdx.x * kFewThreads + tid;
  const int e = a.index[m], K = (int)a.K;
  const float base = a.base && n < a.N ? load_any(a.base, m * a.ldb + n, a.out_dtype) : 0.f;
  if (e < 0 || e >= a.adapters) {
    if (a.base != a.y && n < a.N) store_out(a.y, m * a.ldy + n, base, a.out_dtype);
    return;
  }
  const uint16_t* const b = reinterpret_cast<const uint16_t*>(a.b.p + e * a.b.stride + min(n, a.N - 1) * a.b.ld);
  u32x4 part[kEach];  // of the column's row, its first 32 ahead
  auto load_part = [&](int r) __attribute__((always_inline)) {
    if (a.rank >= 8)
#pragma unroll
      for (int i = 0; i < kEach; ++i) part[i] = *reinterpret_cast<const u32x4_any*>(b + min(r + 8 * i, a.rank - 8));
  };
  load_part(0);
  const uint16_t* const x = static_cast<const uint16_t*>(a.x) + m * a.ldx;
  const char* const w = a.a.p + e * a.a.stride;
  const int groups = (a.rank + kRows - 1) / kRows, along = kWaves / groups;  // of the rank; waves along K
  const int r0 = wave % groups * kRows, part_k = wave / groups;
  if (part_k < along) {
    float acc[kRows] = {};
    for (int k0 = 512 * part_k; k0 < K; k0 += 512 * along) {
      const int k = k0 + 8 * lane, at = min(k, K - 8);
      u32x4 v = *reinterpret_cast<const u32x4_any*>(x + at), q[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i)
        q[i] = *reinterpret_cast<const u32x4_any*>(w + (int64_t)min(r0 + i, a.rank - 1) * a.a.ld + 2 * at);
      if (k0 + 512 > K) {  // what lies past the end becomes zero
        v = bytes_from(v, min(2 * (k - at), 16));
#pragma unroll
        for (int i = 0; i < kRows; ++i) q[i] = bytes_from(q[i], min(2 * (k - at), 16));
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i] = fmaf(half_to_f32<XT>(q[i][j / 2], j & 1), half_to_f32<XT>(v[j / 2], j & 1), acc[i]);
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const float v = wave_sum(acc[i]);
      if (lane == 0 && r0 + i < a.rank) sums[part_k][r0 + i] = v;
    }
  }
  __syncthreads();
  if (tid < a.rank) {
    float v = 0.f;
    for (int i = 0; i < along; ++i) v += sums[i][tid];
    h[tid] = v;
  }
  __syncthreads();
  if (n >= a.N) return;
  float v = 0.f;
  if (a.rank < 8) {
    for (int j = 0; j < a.rank; ++j) v = fmaf(load_any(b, j, a.x_dtype), h[j], v);
  } else {
    auto add = [&](int r, const u32x4& q) __attribute__((always_inline)) {
      const int at = min(r, a.rank - 8);  // the last eight may hold some twice
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (at + j >= r) v = fmaf(half_to_f32<XT>(q[j / 2], j & 1), h[at + j], v);
    };
    for (int r = 0; r < a.rank; r += 8 * kEach) {
      if (r > 0) load_part(r);
#pragma unroll
      for (int i = 0; i < kEach; ++i)
        if (r + 8 * i < a.rank) add(r + 8 * i, part[i]);
    }
  }
  store_out(a.y, m * a.ldy + n, base + (a.scale ? a.scale[e] : 1.f) * v, a.out_dtype);
}

// The first product of rows whose adapters' matrices are small altogether,
// row by row, and beside it, in the first workgroup, the tiles' table for the
// second: 16 values of a row to a workgroup, eight waves along K times two of
// eight values.  A chain of waits (the adapter's number, its weights, a barrier):
// 48 rows of 64 adapters rank 64, 4096 long, 7.1 us for 25 MB, most of it waits.
template <int XT>
__global__ __launch_bounds__(1024) void lora_dot_kernel(gt::LoraArgs a, RowIndex ix, RowTable* table, float* mid, int64_t ld) {
  constexpr int kRows = 8, kAlong = 8;
  __shared__ float sums[kAlong][2 * kRows];
  if (blockIdx.x == 0) {
    make_row_table(ix, table);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), K = (int)a.K;
  const int groups = (a.rank + 2 * kRows - 1) / (2 * kRows), m = (blockIdx.x - 1) / groups;
  const int first = ((int)blockIdx.x - 1 - m * groups) * 2 * kRows, r0 = first + wave % 2 * kRows;
  const int e = a.index[m];
  if (e < 0 || e >= a.adapters) return;
  const uint16_t* const x = static_cast<const uint16_t*>(a.x) + m * a.ldx;
  const char* const w = a.a.p + e * a.a.stride;
  float acc[kRows] = {};
  for (int k0 = 512 * (wave / 2); k0 < K; k0 += 512 * kAlong) {
    const int k = k0 + 8 * lane, at = min(k, K - 8);
    u32x4 v = *reinterpret_cast<const u32x4_any*>(x + at), q[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      q[i] = *reinterpret_cast<const u32x4_any*>(w + (int64_t)min(r0 + i, a.rank - 1) * a.a.ld + 2 * at);
    if (k0 + 512 > K) {  // what lies past the end becomes zero
      v = bytes_from(v, min(2 * (k - at), 16));
#pragma unroll
      for (int i = 0; i < kRows; ++i) q[i] = bytes_from(q[i], min(2 * (k - at), 16));
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[i] = fmaf(half_to_f32<XT>(q[i][j / 2], j & 1), half_to_f32<XT>(v[j / 2], j & 1), acc[i]);
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const float v = wave_sum(acc[i]);
    if (lane == 0) sums[wave / 2][wave % 2 * kRows + i] = v;
  }
  __syncthreads();
  if (tid < 2 * kRows && first + tid < a.rank) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kAlong; ++i) v += sums[i][tid];
    mid[m * ld + first + tid] = v;
  }
}

// Rows of x or of the adapters' first matrices too short for a lane's 16
// bytes, or the latter so far apart that a tile's offsets pass 32 bits: a wave
// to a value.
__global__ __launch_bounds__(256) void lora_shrink_kernel(gt::LoraArgs a, float* mid, int64_t ld) {
  const int lane = threadIdx.x & 63, r = blockIdx.y * 4 + (threadIdx.x >> 6);
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    const int e = a.index[m];
    if (r >= a.rank || e < 0 || e >= a.adapters) continue;
    const char* row = a.a.p + e * a.a.stride + r * a.a.ld;
    float v = 0.f;
    for (int64_t k = lane; k < a.K; k += 64) v += load_any(a.x, m * a.ldx + k, a.x_dtype) * load_any(row, k, a.x_dtype);
    v = wave_sum(v);
    if (lane == 0) mid[m * ld + r] = v;
  }
}

__global__ __launch_bounds__(256) void copy_rows_kernel(const void* base, void* y, int64_t M, int64_t N, int64_t ldb, int64_t ldy,
                                                        int dtype) {
  for (int64_t m = blockIdx.y; m < M; m += gridDim.y)
    for (int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x; n < N; n += (int64_t)gridDim.x * 256)
      store_out(y, m * ldy + n, base ? load_any(base, m * ldb + n, dtype) : 0.f, dtype);
}

}  // namespace gtk

namespace gt {
namespace {

bool in_units(const LoraArgs& a) { return a.K >= 8 && a.a.ld <= (INT64_C(1) << 27); }

// Whether one launch that computes the first product again for every 1024
// columns is the faster: matrices a of up to 256 KB, and rows and columns for
// one workgroup to a CU, or two where the rows are so many that the tiles'
// table would be a launch of its own.  bf16, against the tiles: 1 row, rank 16, 4096 x 4096 5.5 us and
// 8.5, rank 32 7.5 and 9.3; 64 rows of rank 16 7.6 and 9.8, 128 (512 workgroups)
// 13.2 and 11.2; 256 rows 2048 x 2048 (512) 11.4 and 14.8; 1 row of rank 32 and
// 8192 x 2048 (512 KB) 10.8 and 9.5; rank 64, 1024 x 1024, 10.1 and 9.6.
bool few_rows(const LoraArgs& a) {
  const int64_t workgroups = a.M * ((a.N + gtk::kFewThreads - 1) / gtk::kFewThreads);
  return a.K >= 8 && a.rank <= 32 && a.rank * a.K <= 128 << 10 && workgroups <= (a.M > gtk::kFewRows ? 2 : 1) * a.cus;
}

// The first product's slices: one workgroup's K where the tiles alone give
// eight workgroups to a CU, more where they do not (300 rows of 2 adapters rank 32, 4096
// long: 15.4 us with 4 slices, 22.3 with one; 4096 rows of 64 adapters rank 16: 43.1 and
// 44.2; a number of slices that does not divide the waves' units loses, 50 with 3).
struct LoraCut {
  gtk::GroupedCut c;
  int units, split;
};
LoraCut cut(const LoraArgs& a) {
  LoraCut l;
  const int64_t tiles = most_tiles(a.M, a.adapters);
  l.units = (int)((a.K + 127) / 128);
  const int pairs = (a.rank + 31) / 32;
  const int64_t want = (int64_t)1 << (bits_of((int)std::min<int64_t>(std::max<int64_t>(1, 8 * a.cus / (tiles * pairs)), 16)) - 1);
  l.c.wk = std::min(8, l.units);
  l.split = (int)std::max<int64_t>(1, std::min<int64_t>(want, l.units / l.c.wk));
  const int each = (l.units + l.c.wk * l.split - 1) / (l.c.wk * l.split);  // of a wave
  l.c.U = each > 2 ? 4 : (each > 1 ? 2 : 1);
  l.c.turns = (each + l.c.U - 1) / l.c.U;
  l.c.cols = 8 / l.c.wk;
  l.c.waves = 8;
  return l;
}
// Whether the first product takes tiles of 64 rows: where an adapter has some
// 256 of them and all together fill the CUs.  4096 long, rank 32, 4096 rows of 6
// adapters 38.4 us and 42.3, rank 64 49 and 66, 2048 rows 36.0 and 38.5; 1024 rows
// of 8 adapters 22 and 18.7, 4096 of 64 adapters 51 and 47.
bool many_rows(const LoraArgs& a) {
  return a.K >= 8 && a.rank >= 8 && a.rank <= 64 && a.M >= 2048 && a.M >= 256 * (int64_t)a.adapters;
}
// Its slices: two workgroups to a CU, of two units at least (a power of two, as above).
int many_split(const LoraArgs& a) {
  const int64_t want = 2 * a.cus / most_tiles(a.M, a.adapters, 64), units = (a.K + 127) / 128;
  return 1 << (bits_of((int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(want, 16), units / 2))) - 1);
}
// Whether the first product goes row by row, which spares the table's launch
// or its search: two workgroups of 4096 long rows to a CU at most (short rows
// count as 2048).  48 rows of 64 adapters rank 64, 4096 x 16384, 24.5 us and
// 26.5 with tiles; rank 16, 4096 x 4096, 512 rows 13.3 and 16.2, 1024 rows (1024
// workgroups) 19.2 and 18.6; 1000 rows 1024 long 14.6 and 18.5; 277 rows of rank
// 34 2945 long (831) 18.0 and 17.4.
bool row_by_row(const LoraArgs& a) {
  return a.K >= 8 && a.M * ((a.rank + 15) / 16) * std::max<int64_t>(a.K, 2048) <= (int64_t)8192 * a.cus;
}
struct LoraSpace {
  int64_t ld;
  size_t mid, bytes;
};
LoraSpace space(LoraArgs a, int64_t rows) {
  LoraSpace s;
  a.M = rows;
  s.ld = (a.rank + 3) / 4 * 4;
  s.mid = gtk::row_table_bytes(most_tiles(rows, a.adapters + 1));
  s.bytes = s.mid + (size_t)(many_rows(a) ? many_split(a) : cut(a).split) * rows * s.ld * 4;
  return s;
}

template <int XT, int OUT, bool PAST>
int expand(const gtk::ExpandParams& p, dim3 grid) {
  const int rank = p.a.rank;
  hipStream_t st = p.a.stream;
  if (rank < 8)
    hipLaunchKernelGGL((gtk::lora_expand_kernel<XT, OUT, 1, true, PAST>), grid, dim3(256), 0, st, p);
  else if (rank <= 32)
    hipLaunchKernelGGL((gtk::lora_expand_kernel<XT, OUT, 1, false, PAST>), grid, dim3(256), 0, st, p);
  else if (rank <= 64)
    hipLaunchKernelGGL((gtk::lora_expand_kernel<XT, OUT, 2, false, PAST>), grid, dim3(256), 0, st, p);
  else if (rank <= 128)
    hipLaunchKernelGGL((gtk::lora_expand_kernel<XT, OUT, 4, false, PAST>), grid, dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL((gtk::lora_expand_kernel<XT, OUT, 8, false, PAST>), grid, dim3(256), 0, st, p);
  return hipGetLastError() == hipSuccess ? LS_OK : LS_HIP_ERROR;
}
// Where base and y are more than the L2s hold, b and the first product's values
// stay there if those pass by: 4096 rows of 6 adapters rank 32, 4096 x 4096 bf16 (67 MB),
// 34.6 us and 38.5, of 64 adapters 43.3 and 47.5; 1024 rows (17 MB) 19.4 and 18.7.
template <int XT, int OUT>
int expand(const gtk::ExpandParams& p, dim3 grid) {
  const bool past = p.a.M * p.a.N * elem_bytes(OUT) * (p.a.base ? 2 : 1) > 32 << 20;
  return past ? expand<XT, OUT, true>(p, grid) : expand<XT, OUT, false>(p, grid);
}
template <int XT>
int expand(const gtk::ExpandParams& p, dim3 grid) {
  switch (p.a.out_dtype) {
    case DT_F32: return expand<XT, DT_F32>(p, grid);
    case DT_F16: return expand<XT, DT_F16>(p, grid);
    default: return expand<XT, DT_BF16>(p, grid);
  }
}

unsigned at_most(int64_t n, int64_t most) { return (unsigned)(n < most ? n : most); }

}  // namespace

int64_t lora_range(const LoraArgs& a) {
  // a row has up to 16 slices where the rows are few, one where they are many
  return std::min<int64_t>(gtk::kMostRows, ((int64_t)64 << 20) / (16 * (4 * ((a.rank + 3) / 4 * 4) + 6)));
}
size_t lora_workspace_bytes(const LoraArgs& a, int64_t rows) { return space(a, rows).bytes; }

int launch_lora(const LoraArgs& a) {
  if (few_rows(a)) {
    const dim3 grid((unsigned)((a.N + gtk::kFewThreads - 1) / gtk::kFewThreads), (unsigned)a.M);
    if (a.x_dtype == DT_BF16)
      hipLaunchKernelGGL((gtk::lora_few_kernel<DT_BF16>), grid, dim3(gtk::kFewThreads), 0, a.stream, a);
    else
      hipLaunchKernelGGL((gtk::lora_few_kernel<DT_F16>), grid, dim3(gtk::kFewThreads), 0, a.stream, a);
    return hipGetLastError() == hipSuccess ? LS_OK : LS_HIP_ERROR;
  }
  const LoraSpace s = space(a, a.M);
  const int none = a.base != a.y;
  const bool many = many_rows(a);
  const int64_t tiles = most_tiles(a.M, a.adapters + none, many ? 64 : 16);
  gtk::RowTable* table = reinterpret_cast<gtk::RowTable*>(a.ws);
  float* mid = reinterpret_cast<float*>(a.ws + s.mid);
  const gtk::RowIndex ix{a.index, 1, (int)a.M, 1, a.adapters, 1u << 20, none, bits_of(a.adapters - 1 + none), many ? 6 : 4};
  int split = 1;
  const bool units = in_units(a);
  const bool dots = row_by_row(a);
  if (!dots && (!units || a.M > gtk::kFewRows)) {
    const int rc = launch_row_tiles(ix, table, a.stream);
    if (rc != LS_OK) return rc;
  }
  if (dots) {
    const dim3 grid((unsigned)(1 + a.M * ((a.rank + 15) / 16)));
    if (a.x_dtype == DT_BF16)
      hipLaunchKernelGGL((gtk::lora_dot_kernel<DT_BF16>), grid, dim3(1024), 0, a.stream, a, ix, table, mid, s.ld);
    else
      hipLaunchKernelGGL((gtk::lora_dot_kernel<DT_F16>), grid, dim3(1024), 0, a.stream, a, ix, table, mid, s.ld);
  } else if (many) {
    split = many_split(a);
    const dim3 grid((unsigned)split, (unsigned)tiles);
    if (a.x_dtype == DT_BF16) {
      if (a.rank <= 32)
        hipLaunchKernelGGL((gtk::lora_many_kernel<DT_BF16, 1>), grid, dim3(512), 0, a.stream, a, table, mid, s.ld, a.M * s.ld, split);
      else
        hipLaunchKernelGGL((gtk::lora_many_kernel<DT_BF16, 2>), grid, dim3(512), 0, a.stream, a, table, mid, s.ld, a.M * s.ld, split);
    } else {
      if (a.rank <= 32)
        hipLaunchKernelGGL((gtk::lora_many_kernel<DT_F16, 1>), grid, dim3(512), 0, a.stream, a, table, mid, s.ld, a.M * s.ld, split);
      else
        hipLaunchKernelGGL((gtk::lora_many_kernel<DT_F16, 2>), grid, dim3(512), 0, a.stream, a, table, mid, s.ld, a.M * s.ld, split);
    }
  } else if (units) {
    const LoraCut l = cut(a);
    split = l.split;
    gtk::GroupedParams p{};
    p.ix = ix;
    p.table = table;
    p.w = a.a;
    p.x = a.x;
    p.ldx = a.ldx;
    p.out = mid;
    p.ld_out = s.ld;
    p.out_slice = a.M * s.ld;
    p.N = a.rank;
    p.K = (int)a.K;
    fill_cut(p, l.c, l.units, l.split);
    const int groups = ((p.N + 31) / 32 + l.c.cols - 1) / l.c.cols;
    if (!fill_list(p, tiles, groups, tiles * l.split * groups)) return LS_UNSUPPORTED;
    const int rc = (a.x_dtype == DT_BF16 ? grouped_bf16 : grouped_f16)(
        p, gtk::GROUPED_SHRINK, l.c, a.stream);
    if (rc != LS_OK) return rc;
  } else {
    hipLaunchKernelGGL(gtk::lora_shrink_kernel, dim3(at_most(a.M, 65536), (a.rank + 3) / 4), dim3(256), 0, a.stream, a, mid, s.ld);
  }
  gtk::ExpandParams e{a, table, mid, s.ld, a.M * s.ld, split, (int)((a.N + 63) / 64), 1, many ? 2 : 0};
  const int64_t groups = (e.blocks + 3) / 4, parts = many ? 4 * tiles : tiles;
  e.blocks_each = (int)std::max<int64_t>(1, std::min<int64_t>(16, groups * parts / (4 * a.cus)));
  const dim3 grid((unsigned)((e.blocks + 4 * e.blocks_each - 1) / (4 * e.blocks_each)), (unsigned)parts);
  return a.x_dtype == DT_BF16 ? expand<DT_BF16>(e, grid) : expand<DT_F16>(e, grid);
}

int launch_copy_rows(const void* base, void* y, int64_t M, int64_t N, int64_t ldb, int64_t ldy, int dtype, hipStream_t stream) {
  if (base == y) return LS_OK;
  hipLaunchKernelGGL(gtk::copy_rows_kernel, dim3(at_most((N + 255) / 256, 1024), at_most(M, 32768)), dim3(256), 0, stream, base, y, M,
                     N, ldb, ldy, dtype);
  return hipGetLastError() == hipSuccess ? LS_OK : LS_HIP_ERROR;
}

}  // namespace gt
