// linear_backward.hip -- the gradients of an activation's or a gate's arguments.
#include "linear_tile.h"

namespace pg {

const void* gated_backward_kernel(int xt, int tile, bool rows16) {
    return linear_by_type<END_GATED_BACKWARD, true, false, 0>(xt, tile, rows16);
}

}  // namespace pg
