// row_tiles.h -- the table of the tiles of rows that name the same matrix
// (grouped.h), by one workgroup: the matrices' rows are counted, the tiles
// before each matrix summed, and every row takes the next place of its
// matrix's tiles (512 rows 5.7 us, 4096 6 to 7, 3.5 of them the launch and the
// waits of one workgroup).  Which place depends on the order of the waves, what is
// computed for a row does not depend on its place.
#pragma once

#include "grouped.h"

namespace gtk {

// By 1024 threads.
__device__ __forceinline__ void make_row_table(const RowIndex& ix, RowTable* table) {
  __shared__ int count[kMostMatrices + 1], place[kMostMatrices + 1];  // rows; the first tile's place, then the next
  __shared__ int of_wave[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, all = ix.matrices + ix.none, in_tile = (1 << ix.tile_lg) - 1;
  constexpr int kRows = kMostRows / 1024, kEach = (kMostMatrices + 1 + 1023) / 1024;
  int e[kRows];
#pragma unroll
  for (int j = 0; j < kRows; ++j) e[j] = 1024 * j + tid < ix.n ? row_matrix(ix, 1024 * j + tid) : -1;
  for (int m = tid; m < all; m += 1024) count[m] = 0;
  __syncthreads();
  // one addition for all rows of a wave that name the same matrix (many may)
  uint64_t same[kRows];
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    same[j] = __ballot(e[j] >= 0);
    for (int b = 0; b < ix.bits; ++b) {
      const bool one = (e[j] >> b & 1) != 0;
      const uint64_t v = __ballot(one);
      same[j] &= one ? v : ~v;
    }
    if (e[j] >= 0 && __ffsll((unsigned long long)same[j]) - 1 == lane) atomicAdd(&count[e[j]], __popcll(same[j]));
  }
  __syncthreads();
  // the tiles of a thread's matrices, then those of the threads before it
  const int m0 = tid * kEach;
  int mine = 0;
#pragma unroll
  for (int m = m0; m < m0 + kEach; ++m) mine += m < all ? (count[m] + in_tile) >> ix.tile_lg : 0;
  int upto = mine;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int v = __shfl_up(upto, d);
    if (lane >= d) upto += v;
  }
  if (lane == 63) of_wave[wave] = upto;
  __syncthreads();
  int tile = upto - mine;
  for (int w = 0; w < wave; ++w) tile += of_wave[w];
  if (tid == 1023) table->tiles = tile + mine;
#pragma unroll
  for (int m = m0; m < m0 + kEach; ++m)
    if (m < all) {
      place[m] = tile << ix.tile_lg;
      tile += (count[m] + in_tile) >> ix.tile_lg;
    }
  __syncthreads();
  int at[kRows];
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const int leader = __ffsll((unsigned long long)same[j]) - 1;
    at[j] = 0;
    if (e[j] >= 0 && leader == lane) at[j] = atomicAdd(&place[e[j]], __popcll(same[j]));
    at[j] = __shfl(at[j], e[j] >= 0 ? leader : lane) + __popcll(same[j] & ((1ull << lane) - 1));
  }
  __syncthreads();
  // a tile's first row writes what the tile has; place[m] is now past the matrix's last row
#pragma unroll
  for (int j = 0; j < kRows; ++j)
    if (e[j] >= 0) {
      RowTile& t = table->tile[at[j] >> ix.tile_lg];
      t.rows[at[j] & in_tile] = 1024 * j + tid;
      if ((at[j] & in_tile) == 0) {
        t.matrix = e[j];
        t.count = min(place[e[j]] - at[j], in_tile + 1);
      }
    }
}

}  // namespace gtk
