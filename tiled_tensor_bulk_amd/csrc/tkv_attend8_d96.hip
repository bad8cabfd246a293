// tkv_attend8_d96.hip -- attention over the 8-bit cache, head_dim 96.
#include "tkv_launch.h"

namespace tkv {
int launch_attend8_d96(const AttendArgs &a, int row_tile, void *stream) { return launch_group<96, 0>(a, row_tile, stream); }
}  // namespace tkv
