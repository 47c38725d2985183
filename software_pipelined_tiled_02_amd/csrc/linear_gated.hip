// linear_gated.hip -- gated layers: two products of one input.
#include "linear_few.h"

namespace pg {

namespace {

template <int END, bool AIN, bool BIN, int EXTRA>
const void* kernel(int xt, int tile) {
    return linear_few_tile(tile) ? few_by_type<END, AIN, BIN, EXTRA>(xt, tile) : linear_by_type<END, AIN, BIN, EXTRA>(xt, tile);
}

}  // namespace

const void* gated_kernel(int xt, int tile) { return kernel<END_GATED, true, true, 0>(xt, tile); }

}  // namespace pg
