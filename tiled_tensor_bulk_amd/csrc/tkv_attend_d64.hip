// tkv_attend_d64.hip -- attention over the 4-bit cache, head_dim 64.
#include "tkv_launch.h"

namespace tkv {
int launch_attend_d64(const AttendArgs &a, int row_tile, void *stream) {
    switch (a.c.group) {
        case 32: return launch_group<64, 32>(a, row_tile, stream);
        case 64: return launch_group<64, 64>(a, row_tile, stream);
    }
    return (int)hipErrorInvalidValue;
}
}  // namespace tkv
