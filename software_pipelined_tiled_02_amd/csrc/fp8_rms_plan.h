// fp8_rms_plan.h -- which form of its kernels the norm and its backward pass
// take.  Plain constexpr C++ with no HIP dependency: the launchers, the checks,
// the workspace's size and a host test share it.
#ifndef PIPEGEMM_FP8_RMS_PLAN_H
#define PIPEGEMM_FP8_RMS_PLAN_H

#include <stdint.h>

namespace pg {

// `tpr` threads hold a row in `nc` steps of 8 values each.
struct RmsForm {
    int tpr, nc;
};
struct RmsBackwardForm {
    bool by_columns;         // dw by columns beside the rows, else in the rows' groups
    int parts;               // of dw, left in the workspace (0: it needs none)
    int tpr, nc;
    bool ahead;              // groups: the next row is loaded before the current one's sum
    bool whole;              // groups, not ahead: D a multiple of 8, or else any D
};

constexpr int64_t rms_parts_row(int64_t D) { return (D + 3) / 4 * 4; }

constexpr RmsForm rms_form(int64_t M, int64_t D) {
    if (D <= 512) return {64, 1};
    // Few rows: more threads each, a chunk per thread (us in a graph, 1 x 8192:
    // 3.4, at four chunks 5.3; 256 x 8192 4.8 and 6.5; 1 x 1000 2.6 and 3.1);
    // with many the bytes on their way count (8192 x 8192: 91 at four chunks).
    if (M <= 512 && D <= 8192) return D <= 2048 ? RmsForm{256, 1} : D <= 4096 ? RmsForm{512, 1} : RmsForm{1024, 1};
    if (D <= 1024) return {64, 2};
    if (D <= 2048) return {256, 1};
    if (D <= 4096) return {256, 2};
    if (D <= 8192) return {256, 4};
    if (D <= 16384) return {1024, 2};
    return {1024, 4};
}

// Workgroups hold whole rows, 256 threads at least.
constexpr int rms_group_threads(int tpr) { return tpr < 256 ? 256 : tpr; }
constexpr int64_t rms_row_groups(int64_t M, int tpr) {
    return (M + rms_group_threads(tpr) / tpr - 1) / (rms_group_threads(tpr) / tpr);
}
// Lanes across the columns of dw that a workgroup of the form by columns takes.
constexpr int columns_lanes(int tpr) { return tpr <= 256 ? 8 : 16; }

// A launch takes less than 2^32 threads (the forms in groups have few).
constexpr int64_t kLaunchThreads = (int64_t)1 << 32;
constexpr bool rms_launches(int64_t M, int64_t D) {
    const RmsForm f = rms_form(M, D);
    return rms_row_groups(M, f.tpr) * rms_group_threads(f.tpr) < kLaunchThreads;
}
constexpr bool rms_backward_launches(const RmsBackwardForm& f, int64_t M, int64_t D) {
    if (!f.by_columns) return true;
    const int64_t across = 8 * columns_lanes(f.tpr);
    return (rms_row_groups(M, f.tpr) + (D + across - 1) / across * (f.parts > 0 ? f.parts : 1)) * rms_group_threads(f.tpr) <
           kLaunchThreads;
}

// The backward pass's form for M rows of D values.  by_columns and parts, which the workspace
// goes by, do not depend on the type (`f32`).
constexpr RmsBackwardForm rms_backward_form(int64_t M, int64_t D, bool f32, int num_cus) {
    // us in groups and by columns, bf16 with dh: 560 x 4096 14.3 and 9.2, 1024
    // x 4096 15.6 and 13.5, 1300 x 4096 16.1 and 16.7; 560 x 8192 15.9 and
    // 14.7, 1024 x 8192 20.0 and 21.3, 2000 x 8192 32.5 and 36; 2000 x 1024
    // 12.7 and 8.8, 8192 x 1024 19.4 and 20.9.  Groups hold 16384 columns at
    // most (1500 x 20000, read twice with registers in scratch: 171 us, by
    // columns 77), and above 12288 multiples of 8.
    if (M <= 1024 || (D <= 1024 && M <= 4096) || D > 16384 || (D > 12288 && D % 8 != 0)) {
        const int parts = M <= 512 ? 0 : (int)((M + 255) / 256 < 64 ? (M + 255) / 256 : 64);
        return D <= 512 ? RmsBackwardForm{true, parts, 64, 1, false, false}
             : D <= 1024 ? RmsBackwardForm{true, parts, 64, 2, false, false}
             : D <= 2048 ? RmsBackwardForm{true, parts, 256, 1, false, false}
             : D <= 4096 ? RmsBackwardForm{true, parts, 256, 2, false, false}
             : D <= 8192 ? RmsBackwardForm{true, parts, 512, 2, false, false}
             : D <= 16384 ? RmsBackwardForm{true, parts, 1024, 2, false, false}
                          : RmsBackwardForm{true, parts, 1024, 4, false, false};
    }
    // two workgroups of 256 or 512 threads per CU (one of more), each with as
    // many groups as it holds rows at a time: more groups leave more parts
    // (8192 x 8192: 512 groups 110 us, 256 105; 8192 x 2048: 1024 39, 512 31),
    // fewer have too little on the way (8192 x 4096: 512 52, 256 62; 16384 x
    // 256: 1536 18.0, 1024 21.3)
    const int64_t most = (int64_t)num_cus * (D <= 512 ? 6 : D <= 1024 ? 4 : D <= 4096 ? 2 : 1);
    const int parts = (int)(M < most ? M : most);
    if (D <= 512) return {false, parts, 64, 1, true, false};
    if (D <= 1024) return {false, parts, 128, 1, true, false};
    if (D <= 2048) return {false, parts, 256, 1, true, false};
    if (D <= 4096) return {false, parts, 512, 1, true, false};
    if (D <= 8192) return {false, parts, 1024, 1, true, false};
    // 16-bit rows up to 12288 in 512 threads, the next one ahead, take 11
    // registers to scratch.  Rows that end inside a thread's 8 values gain by it
    // (us at 1030, 2000 and 8192 x 9300: 36, 51 and 161; held, with 19 registers
    // in scratch, 39, 55 and 166; by columns 35, 61 and 230), multiples of 8 do
    // not (8192 x 8200: 147, held 118; 8192 x 10240: 149 and 135; 8192 x 12288: 178
    // and 157; 2000 x 10240: 49 and 44; 1030 x 12288: 40 and 36).
    if (!f32 && D <= 12288 && D % 8 != 0) return {false, parts, 512, 3, true, false};
    // fp32 rows that end inside a thread's 8 values: settling them takes 9
    // registers to scratch, and is still faster than by columns with many
    // rows (8192 x 9300: 254 us, 348 by columns; 2000 x 9300: 78 and 90; 1030 x
    // 9300: 52 and 49; 8192 x 8200: 223, 204 as multiples of 8).
    return {false, parts, 1024, 2, false, D % 8 == 0};
}

}  // namespace pg

#endif
