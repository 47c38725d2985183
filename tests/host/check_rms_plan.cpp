// The forms that the norm and its backward pass take, over both sides of every border of
// M and D and both kinds of type: one that exists and takes the D it is given,
// with parts of dw that fit the workspace whatever the type.
#include <cstdio>
#include <initializer_list>
#include <vector>

#include "fp8_rms_plan.h"

using pg::RmsBackwardForm;

// The kernels compiled for a type: 16-bit types hold 8193 to 12288 columns ahead in 512 threads; fp32 any
// D in the held form.
static bool exists(const RmsBackwardForm& f, bool f32) {
    const int k = 8 * f.tpr + f.nc;
    if (f.by_columns) {
        for (int c : {8 * 64 + 1, 8 * 64 + 2, 8 * 256 + 1, 8 * 256 + 2, 8 * 512 + 2, 8 * 1024 + 2, 8 * 1024 + 4})
            if (k == c) return true;
        return false;
    }
    if (f.ahead) {
        for (int c : {8 * 64 + 1, 8 * 128 + 1, 8 * 256 + 1, 8 * 512 + 1, 8 * 1024 + 1})
            if (k == c) return !f.whole;
        return k == 8 * 512 + 3 && !f32 && !f.whole;
    }
    return k == 8 * 1024 + 2 && (f.whole || f32);
}

int main() {
    std::vector<int64_t> ms, ds;
    for (int64_t m : {1, 64, 128, 256, 512, 1024, 1536, 2048, 4096, 8192, 65536, 1 << 22})
        for (int64_t d = -1; d <= 1; ++d) ms.push_back(m + d);
    for (int64_t d : {8, 512, 1024, 2048, 4096, 8192, 9300, 10000, 12288, 16384, 20000, 32768})
        for (int64_t e = -9; e <= 9; ++e)
            if (d + e >= 1 && d + e <= 32768) ds.push_back(d + e);
    // launches: one row below the last refused one, and everything of fewer rows or shorter ones
    const int64_t most = 1 << 22;
    bool launches = pg::rms_launches(most, 8192) && pg::rms_launches(most - 1, 32768) && !pg::rms_launches(most, 8193);
    const auto back = [](int64_t m, int64_t d) {
        return pg::rms_backward_launches(pg::rms_backward_form(m, d, false, 256), m, d);
    };
    launches = launches && back(most, 8192) && back(most, 16384) && back(most - 16385, 32768) && !back(most - 16384, 32768);
    // 16-bit rows of 8193 to 12288: only those that are no multiple of 8 spill
    const bool spills = pg::rms_backward_form(2000, 10241, false, 256).ahead && !pg::rms_backward_form(2000, 10240, false, 256).ahead &&
                        !pg::rms_backward_form(2000, 8200, false, 256).ahead && !pg::rms_backward_form(2000, 12288, false, 256).ahead;
    long bad = launches && spills ? 0 : 1, seen = 0;
    for (int64_t m : ms)
        for (int64_t d : ds) {
            if (m > (1 << 22)) continue;
            const RmsBackwardForm half = pg::rms_backward_form(m, d, false, 256);
            const pg::RmsForm fw = pg::rms_form(m, d);
            if ((int64_t)fw.tpr * fw.nc * 8 < d) ++bad;
            for (bool f32 : {false, true}) {
                const RmsBackwardForm f = pg::rms_backward_form(m, d, f32, 256);
                ++seen;
                const bool ok = exists(f, f32) && (int64_t)f.tpr * f.nc * 8 >= d && (!f.whole || d % 8 == 0) &&
                                f.by_columns == half.by_columns && f.parts == half.parts &&
                                (f.by_columns ? f.parts >= 0 && f.parts <= 64 && (m > 512 || f.parts == 0)
                                              : f.parts >= 1 && f.parts <= m);
                if (!ok && ++bad <= 10)
                    std::printf("%lld x %lld %s: %s, %d threads, %d steps, %s%s, %d parts\n", (long long)m, (long long)d,
                                f32 ? "fp32" : "16-bit", f.by_columns ? "columns" : "groups", f.tpr, f.nc,
                                f.ahead ? "ahead" : "held", f.whole ? ", multiples of 8" : "", f.parts);
            }
        }
    std::printf("%ld forms, %ld wrong\n", seen, bad);
    std::puts(bad == 0 ? "OK" : "FAILED");
    return bad == 0 ? 0 : 1;
}
