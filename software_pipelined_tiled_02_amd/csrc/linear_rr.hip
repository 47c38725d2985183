// linear_rr.hip -- products with a weight as it lies: K across its rows.
#include "linear_few.h"

namespace pg {

namespace {

template <int END, bool AIN, bool BIN, int EXTRA>
const void* kernel(int xt, int tile, bool rows4) {
    if (linear_few_tile(tile)) return rows4 ? few_by_type<END, AIN, BIN, EXTRA>(xt, tile) : nullptr;
    return linear_by_type<END, AIN, BIN, EXTRA>(xt, tile, rows4);
}

}  // namespace

const void* linear_rr_kernel(int xt, int tile, bool rows4, bool pair) {
    return pair ? kernel<END_LINEAR, true, false, 1>(xt, tile, rows4) : kernel<END_LINEAR, true, false, 0>(xt, tile, rows4);
}

}  // namespace pg
