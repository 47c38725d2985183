// linear_weight.hip -- gradients of weights: K across the rows of both factors.
#include "linear_few.h"

namespace pg {

namespace {

template <int END, bool AIN, bool BIN, int EXTRA>
const void* kernel(int xt, int tile) {
    return linear_few_tile(tile) ? few_by_type<END, AIN, BIN, EXTRA>(xt, tile) : linear_by_type<END, AIN, BIN, EXTRA>(xt, tile);
}

}  // namespace

const void* weight_gradient_kernel(int xt, int tile, bool sums) {
    return sums ? kernel<END_WEIGHT, false, false, 1>(xt, tile) : kernel<END_WEIGHT, false, false, 0>(xt, tile);
}

}  // namespace pg
