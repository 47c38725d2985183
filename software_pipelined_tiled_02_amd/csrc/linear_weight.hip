// linear_weight.hip -- gradients of weights: K across the rows of both factors.
#include "linear_few.h"

namespace pg {

namespace {

template <int END, bool AIN, bool BIN, int EXTRA>
const void* kernel(int xt, int tile, bool rows4) {
    if (linear_few_tile(tile)) return rows4 ? few_by_type<END, AIN, BIN, EXTRA>(xt, tile) : nullptr;
    return linear_by_type<END, AIN, BIN, EXTRA>(xt, tile, rows4);
}

}  // namespace

const void* weight_gradient_kernel(int xt, int tile, bool rows4, bool sums) {
    return sums ? kernel<END_WEIGHT, false, false, 1>(xt, tile, rows4) : kernel<END_WEIGHT, false, false, 0>(xt, tile, rows4);
}

}  // namespace pg
