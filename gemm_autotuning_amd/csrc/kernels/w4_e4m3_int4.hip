// w4_e4m3_int4.hip -- the 4-bit weight product's kernels for e4m3 rows and int4 weights.
#include "launchers.h"
#include "w4_mma.h"

namespace gt {
GT_W4_LAUNCHER(w4_mma_e4m3_int4, DT_E4M3, gtk::W4_INT4)
}  // namespace gt
