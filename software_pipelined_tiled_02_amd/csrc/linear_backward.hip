// linear_backward.hip -- the gradients of an activation's or a gate's arguments.
#include "linear_few.h"

namespace pg {

namespace {

template <int END, bool AIN, bool BIN, int EXTRA>
const void* kernel(int xt, int tile) {
    return linear_few_tile(tile) ? few_by_type<END, AIN, BIN, EXTRA>(xt, tile) : linear_by_type<END, AIN, BIN, EXTRA>(xt, tile);
}

}  // namespace

const void* gated_backward_kernel(int xt, int tile) {
    return kernel<END_GATED_BACKWARD, true, false, 0>(xt, tile);
}

}  // namespace pg
