// grouped_wide_f16.hip -- grouped products of many f16 rows with 16-bit weights (grouped_wide.h).
#include "grouped_wide.h"

namespace gt {
int grouped_wide_f16(const gtk::GroupedParams& p, int phase, bool whole, hipStream_t stream) { return gtk::grouped_wide_launch<DT_F16>(p, phase, whole, stream); }
}  // namespace gt
