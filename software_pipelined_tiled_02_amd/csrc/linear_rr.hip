// linear_rr.hip -- products with a weight as it lies: K across its rows.
#include "linear_tile.h"

namespace pg {

const void* linear_rr_kernel(int xt, int tile, bool rows16) {
    return linear_by_type<END_LINEAR, true, false, false>(xt, tile, rows16);
}

}  // namespace pg
