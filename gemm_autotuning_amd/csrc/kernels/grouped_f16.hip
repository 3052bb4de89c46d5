// grouped_f16.hip -- grouped products of f16 rows with 16-bit weights (grouped.h).
#include "grouped.h"

namespace gt {
GT_GROUPED_LAUNCHER(grouped_f16, DT_F16, gtk::GROUPED_16)
}  // namespace gt
