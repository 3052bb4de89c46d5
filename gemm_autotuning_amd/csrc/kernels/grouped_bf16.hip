// grouped_bf16.hip -- grouped products of bf16 rows with 16-bit weights (grouped.h).
#include "grouped.h"

namespace gt {
GT_GROUPED_LAUNCHER(grouped_bf16, DT_BF16, gtk::GROUPED_16)
}  // namespace gt
