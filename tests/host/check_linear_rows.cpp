// pg::rows_meet against every byte of the two matrices, over all small ones and
// some at large addresses and steps.
#include <stdio.h>
#include <stdint.h>

#include <random>

#include "linear_rows.h"

static bool by_bytes(const pg::ByteRows& x, const pg::ByteRows& y) {
    for (int64_t i = 0; i < x.count; ++i)
        for (int64_t j = 0; j < y.count; ++j) {
            const int64_t a = x.at + i * x.step, b = y.at + j * y.step;
            if (x.width > 0 && y.width > 0 && a < b + y.width && b < a + x.width) return true;
        }
    return false;
}

static int wrong = 0, met = 0, apart = 0;

static void check(const pg::ByteRows& x, const pg::ByteRows& y) {
    const bool want = by_bytes(x, y);
    (want ? met : apart) += 1;
    if (pg::rows_meet(x, y) != want || pg::rows_meet(y, x) != want) {
        if (++wrong < 10)
            printf("wrong: %lld %lld %lld %lld, %lld %lld %lld %lld: %d\n", (long long)x.at, (long long)x.count, (long long)x.width,
                   (long long)x.step, (long long)y.at, (long long)y.count, (long long)y.width, (long long)y.step, want);
    }
}

int main() {
    for (int64_t xc = 0; xc < 5; ++xc)
        for (int64_t xw = 0; xw < 5; ++xw)
            for (int64_t xs = xw > 1 ? xw : 1; xs < 9; ++xs)
                for (int64_t yc = 0; yc < 5; ++yc)
                    for (int64_t yw = 0; yw < 5; ++yw)
                        for (int64_t ys = yw > 1 ? yw : 1; ys < 9; ++ys)
                            for (int64_t at = 60; at < 140; at += 1 + (xc + xw + ys) % 3) check({100, xc, xw, xs}, {at, yc, yw, ys});
    std::mt19937_64 rng(1);
    auto pick = [&](int64_t n) { return (int64_t)(rng() % (uint64_t)n); };
    for (int k = 0; k < 200000; ++k) {
        pg::ByteRows x{((int64_t)1 << 46) + pick(3000), 1 + pick(12), 1 + pick(60), 0}, y{((int64_t)1 << 46) + pick(3000), 1 + pick(12), 1 + pick(60), 0};
        x.step = x.width + pick(400);
        y.step = pick(4) == 0 ? (x.step >= y.width ? x.step : y.width) : y.width + pick(400);
        check(x, y);
    }
    const int64_t far = (int64_t)1 << 33;                    // rows far apart: 2^33 bytes, of them 2^10
    check({0, 1000, 64, far}, {128, 900, 64, far});
    check({0, 1000, 64, far}, {128, 900, 64, far + 2});
    check({0, 1000, 64, far}, {128, 900, 64, far - 2});
    printf("%d meet, %d apart, %d wrong\n%s\n", met, apart, wrong, wrong == 0 && met > 1000 && apart > 1000 ? "OK" : "FAILED");
    return wrong != 0;
}
