// linear_weight.hip -- gradients of weights: K across the rows of both factors.
#include "linear_tile.h"

namespace pg {

const void* weight_gradient_kernel(int xt, int tile, bool rows16, bool sums) {
    return sums ? linear_by_type<END_WEIGHT, false, false, 1>(xt, tile, rows16)
                : linear_by_type<END_WEIGHT, false, false, 0>(xt, tile, rows16);
}

}  // namespace pg
