// w4_bf16_int4.hip -- the 4-bit weight product's kernels for bf16 rows and int4 weights.
#include "launchers.h"
#include "w4_mma.h"

namespace gt {
GT_W4_LAUNCHER(w4_mma_bf16_int4, DT_BF16, gtk::W4_INT4)
}  // namespace gt
