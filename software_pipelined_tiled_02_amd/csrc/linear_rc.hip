// linear_rc.hip -- layers: both factors with K along their rows.
#include "linear_tile.h"

namespace pg {

const void* linear_rc_kernel(int xt, int tile, bool rows16, bool pair) {
    return pair ? linear_by_type<END_LINEAR, true, true, 1>(xt, tile, rows16) : linear_by_type<END_LINEAR, true, true, 0>(xt, tile, rows16);
}

}  // namespace pg
