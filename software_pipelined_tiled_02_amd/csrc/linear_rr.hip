// linear_rr.hip -- products with a weight as it lies: K across its rows.
#include "linear_few.h"

namespace pg {

namespace {

template <int END, bool AIN, bool BIN, int EXTRA>
const void* kernel(int xt, int tile) {
    return linear_few_tile(tile) ? few_by_type<END, AIN, BIN, EXTRA>(xt, tile) : linear_by_type<END, AIN, BIN, EXTRA>(xt, tile);
}

}  // namespace

const void* linear_rr_kernel(int xt, int tile, bool pair) {
    return pair ? kernel<END_LINEAR, true, false, 1>(xt, tile) : kernel<END_LINEAR, true, false, 0>(xt, tile);
}

}  // namespace pg
