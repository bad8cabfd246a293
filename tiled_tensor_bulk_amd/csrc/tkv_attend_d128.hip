// tkv_attend_d128.hip -- attention over the 4-bit cache, head_dim 128.
#include "tkv_launch.h"

namespace tkv {
int launch_attend_d128(const AttendArgs &a, int row_tile, void *stream) {
    switch (a.c.group) {
        case 0: return launch_attend8_d128(a, row_tile, stream);
        case 32: return launch_group<128, 32>(a, row_tile, stream);
        case 64: return launch_group<128, 64>(a, row_tile, stream);
        case 128: return launch_group<128, 128>(a, row_tile, stream);
    }
    return (int)hipErrorInvalidValue;
}
}  // namespace tkv
