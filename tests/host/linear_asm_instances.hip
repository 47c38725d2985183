// Instances with transposing LDS reads, for tests/test_linear_asm_waits.py.
#include "linear_few.h"

namespace pg {

const void* instances(int t, bool rr, bool backward, bool sums, bool pair) {
    if (pair) return linear_by_tile<XT_F16, END_LINEAR, true, false, 1>(t);
    if (rr) return linear_by_tile<XT_BF16, END_LINEAR, true, false, 0>(t);
    if (backward) return linear_by_tile<XT_F16, END_GATED_BACKWARD, true, false, 0>(t);
    if (sums) return linear_by_tile<XT_BF16, END_WEIGHT, false, false, 1>(t);
    return linear_by_tile<XT_F16, END_WEIGHT, false, false, 0>(t);
}

const void* few_instances(int t, bool rr, bool backward, bool sums, bool pair) {
    if (pair) return few_by_tile<XT_F16, END_LINEAR, true, false, 1>(t);
    if (rr) return few_by_tile<XT_BF16, END_LINEAR, true, false, 0>(t);
    if (backward) return few_by_tile<XT_F16, END_GATED_BACKWARD, true, false, 0>(t);
    if (sums) return few_by_tile<XT_BF16, END_WEIGHT, false, false, 1>(t);
    return few_by_tile<XT_F16, END_WEIGHT, false, false, 0>(t);
}

}  // namespace pg
