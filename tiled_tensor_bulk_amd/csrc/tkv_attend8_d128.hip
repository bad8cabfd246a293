// tkv_attend8_d128.hip -- attention over the 8-bit cache, head_dim 128.
#include "tkv_launch.h"

namespace tkv {
int launch_attend8_d128(const AttendArgs &a, int row_tile, void *stream) { return launch_group<128, 0>(a, row_tile, stream); }
}  // namespace tkv
