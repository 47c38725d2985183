// linear_rr.hip -- products with a weight as it lies: K across its rows.
#include "linear_tile.h"

namespace pg {

const void* linear_rr_kernel(int xt, int tile, bool rows16, bool pair) {
    return pair ? linear_by_type<END_LINEAR, true, false, 1>(xt, tile, rows16) : linear_by_type<END_LINEAR, true, false, 0>(xt, tile, rows16);
}

}  // namespace pg
