// linear_rc.hip -- layers: both factors with K along their rows.
#include "linear_few.h"

namespace pg {

namespace {

template <int END, bool AIN, bool BIN, int EXTRA>
const void* kernel(int xt, int tile) {
    return linear_few_tile(tile) ? few_by_type<END, AIN, BIN, EXTRA>(xt, tile) : linear_by_type<END, AIN, BIN, EXTRA>(xt, tile);
}

}  // namespace

const void* linear_rc_kernel(int xt, int tile, bool pair) {
    return pair ? kernel<END_LINEAR, true, true, 1>(xt, tile) : kernel<END_LINEAR, true, true, 0>(xt, tile);
}

}  // namespace pg
