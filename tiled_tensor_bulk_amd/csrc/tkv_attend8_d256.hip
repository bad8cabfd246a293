// tkv_attend8_d256.hip -- attention over the 8-bit cache, head_dim 256.
#include "tkv_launch.h"

namespace tkv {
int launch_attend8_d256(const AttendArgs &a, int row_tile, void *stream) { return launch_group<256, 0>(a, row_tile, stream); }
}  // namespace tkv
