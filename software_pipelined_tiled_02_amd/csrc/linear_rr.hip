// linear_rr.hip -- products with a weight as it lies: K across its rows.
#include "linear_few.h"

namespace pg {

namespace {

template <int END, bool AIN, bool BIN, int EXTRA>
const void* kernel(int xt, int tile, bool rows16) {
    if (linear_few_tile(tile)) return rows16 ? few_by_type<END, AIN, BIN, EXTRA>(xt, tile) : nullptr;
    return linear_by_type<END, AIN, BIN, EXTRA>(xt, tile, rows16);
}

}  // namespace

const void* linear_rr_kernel(int xt, int tile, bool rows16, bool pair) {
    return pair ? kernel<END_LINEAR, true, false, 1>(xt, tile, rows16) : kernel<END_LINEAR, true, false, 0>(xt, tile, rows16);
}

}  // namespace pg
