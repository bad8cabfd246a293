// tkv_attend_d256.hip -- attention over the 4-bit cache, head_dim 256.
#include "tkv_launch.h"

namespace tkv {
int launch_attend_d256(const AttendArgs &a, int row_tile, void *stream) {
    switch (a.c.group) {
        case 32: return launch_group<256, 32>(a, row_tile, stream);
        case 64: return launch_group<256, 64>(a, row_tile, stream);
        case 128: return launch_group<256, 128>(a, row_tile, stream);
    }
    return (int)hipErrorInvalidValue;
}
}  // namespace tkv
