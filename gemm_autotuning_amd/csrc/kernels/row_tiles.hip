// row_tiles.hip -- the table of row_tiles.h by a launch of its own.
#include "row_tiles.h"

namespace gtk {

__global__ __launch_bounds__(1024) void row_tiles_kernel(RowIndex ix, RowTable* table) { make_row_table(ix, table); }

}  // namespace gtk

namespace gt {

int launch_row_tiles(const gtk::RowIndex& ix, gtk::RowTable* table, hipStream_t stream) {
  if (ix.n > gtk::kMostRows || ix.matrices > gtk::kMostMatrices) return LS_UNSUPPORTED;
  hipLaunchKernelGGL(gtk::row_tiles_kernel, dim3(1), dim3(1024), 0, stream, ix, table);
  return hipGetLastError() == hipSuccess ? LS_OK : LS_HIP_ERROR;
}

}  // namespace gt
