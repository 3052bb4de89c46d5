// grouped_bf16_e2m1.hip -- grouped products of bf16 rows with e2m1 weights (grouped.h).
#include "grouped.h"

namespace gt {
GT_GROUPED_LAUNCHER(grouped_bf16_e2m1, DT_BF16, gtk::W4_E2M1)
}  // namespace gt
