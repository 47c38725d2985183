// linear_gated.hip -- gated layers: two products of one input.
#include "linear_few.h"

namespace pg {

namespace {

template <int END, bool AIN, bool BIN, int EXTRA>
const void* kernel(int xt, int tile, bool rows4) {
    if (linear_few_tile(tile)) return rows4 ? few_by_type<END, AIN, BIN, EXTRA>(xt, tile) : nullptr;
    return linear_by_type<END, AIN, BIN, EXTRA>(xt, tile, rows4);
}

}  // namespace

const void* gated_kernel(int xt, int tile, bool rows4) { return kernel<END_GATED, true, true, 0>(xt, tile, rows4); }

}  // namespace pg
