// grouped_bf16_int4.hip -- grouped products of bf16 rows with int4 weights (grouped.h).
#include "grouped.h"

namespace gt {
GT_GROUPED_LAUNCHER(grouped_bf16_int4, DT_BF16, gtk::W4_INT4)
}  // namespace gt
