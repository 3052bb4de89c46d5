// w4_e4m3_e2m1.hip -- the 4-bit weight product's kernels for e4m3 rows and e2m1 weights.
#include "launchers.h"
#include "w4_mma.h"

namespace gt {
GT_W4_LAUNCHER(w4_mma_e4m3_e2m1, DT_E4M3, gtk::W4_E2M1)
}  // namespace gt
