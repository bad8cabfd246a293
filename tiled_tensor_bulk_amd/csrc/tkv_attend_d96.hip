// tkv_attend_d96.hip -- attention over the 4-bit cache, head_dim 96.
#include "tkv_launch.h"

namespace tkv {
int launch_attend_d96(const AttendArgs &a, int row_tile, void *stream) {
    switch (a.c.group) {
        case 0: return launch_attend8_d96(a, row_tile, stream);
        case 32: return launch_group<96, 32>(a, row_tile, stream);
    }
    return (int)hipErrorInvalidValue;
}
}  // namespace tkv
