// linear_gated.hip -- gated layers: two products of one input.
#include "linear_tile.h"

namespace pg {

const void* gated_kernel(int xt, int tile, bool rows16) { return linear_by_type<END_GATED, true, true, 0>(xt, tile, rows16); }

}  // namespace pg
