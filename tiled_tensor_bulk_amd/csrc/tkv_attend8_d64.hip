// tkv_attend8_d64.hip -- attention over the 8-bit cache, head_dim 64.
#include "tkv_launch.h"

namespace tkv {
int launch_attend8_d64(const AttendArgs &a, int row_tile, void *stream) { return launch_group<64, 0>(a, row_tile, stream); }
}  // namespace tkv
