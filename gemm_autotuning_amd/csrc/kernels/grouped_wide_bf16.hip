// grouped_wide_bf16.hip -- grouped products of many bf16 rows with 16-bit weights (grouped_wide.h).
#include "grouped_wide.h"

namespace gt {
int grouped_wide_bf16(const gtk::GroupedParams& p, int phase, bool whole, hipStream_t stream) { return gtk::grouped_wide_launch<DT_BF16>(p, phase, whole, stream); }
}  // namespace gt
