// extents_check.cpp -- host-side checks of dense_gemm_06_amd/csrc/extents.h at sizes up to
// 2^31 - 1 (built by tests/test_extents_host.py as plain C++). Prints "0 failures" when every
// count and walk agrees with 64-bit arithmetic.
#include <stdint.h>
#include <stdio.h>

#include <initializer_list>

#include "../dense_gemm_06_amd/csrc/extents.h"

static int fails = 0;
#define CHECK(c, ...)                            \
    do {                                         \
        if (!(c)) {                              \
            if (fails < 20) printf(__VA_ARGS__); \
            ++fails;                             \
        }                                        \
    } while (0)

constexpr int64_t kTop = ((int64_t)1 << 31) - 1;

template <int of>
void pieces_at(int64_t n) {
    if (n < 0 || n > kTop) return;
    CHECK(dg::pieces<of>((int)n) == (n + of - 1) / of, "pieces<%d>(%lld) = %d\n", of, (long long)n, dg::pieces<of>((int)n));
}

void walk_at(int64_t first, int64_t end, int64_t step) {
    int64_t want = first, calls = 0;
    dg::stride_walk(first, end, step, [&](int at) {
        CHECK(at == want && at < end, "walk %lld %lld %lld: %d\n", (long long)first, (long long)end, (long long)step, at);
        want += step;
        ++calls;
    });
    CHECK(calls == (end > first ? (end - first + step - 1) / step : 0), "walk %lld %lld %lld: %lld calls\n",
          (long long)first, (long long)end, (long long)step, (long long)calls);
}

int main() {
    for (int64_t base : {(int64_t)0, (int64_t)1 << 20, ((int64_t)1 << 31) - 4096, (int64_t)1 << 31})
        for (int64_t d = -4200; d <= 4200; ++d) {
            pieces_at<16>(base + d);
            pieces_at<128>(base + d);
            pieces_at<256>(base + d);
        }
    for (int64_t end : {kTop, kTop - 1, kTop - 63, kTop - 2047, kTop - (1 << 20), (int64_t)5, (int64_t)0})
        for (int64_t step : {(int64_t)2048, (int64_t)1 << 20, ((int64_t)1 << 24) - 7})
            for (int64_t first : {(int64_t)0, (int64_t)1, step - 1, kTop - 3 * step, kTop - 1, kTop}) walk_at(first, end, step);
    // 2^20 experts whose offsets alternate between the first row and the last of 2^20, 64 at a time
    const int tiles = (1 << 20) / 128 + (1 << 20);
    int total = 0;
    for (int e = 0; e < 1 << 20; e += 64) total = dg::capped_sum(total, 32 * ((1 << 20) / 128), tiles);
    CHECK(total == tiles, "capped sum %d, not %d\n", total, tiles);
    CHECK(dg::capped_sum(5, 6, 12) == 11 && dg::capped_sum(5, 8, 12) == 12, "capped sum\n");
    printf("%d failures\n", fails);
    return fails != 0;
}
