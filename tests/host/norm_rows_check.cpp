// Host check of the norm's split of a batch into launches (kernels.h): for every
// row count the ABI takes, the largest included, the launches' rows follow each
// other from row 0 to row T - 1, none is empty, and none holds 2^32 lanes.
#include <cstdio>
#include <cstdlib>

#include "kernels.h"

using namespace moe;

static void check(int64_t T) {
    const int n = norm_launches((int32_t)T);
    int64_t next = 0;
    for (int i = 0; i < n; ++i) {
        const NormLaunch p = norm_launch((int32_t)T, i);
        if (p.first != next || p.rows < 1 || p.first + p.rows > T || (uint64_t)p.rows * 1024 >= 1ull << 32) {
            std::printf("FAIL T=%lld launch %d: rows %lld + %d\n", (long long)T, i, (long long)p.first, p.rows);
            std::exit(1);
        }
        next += p.rows;
    }
    if (next != T) {
        std::printf("FAIL T=%lld: %lld rows in %d launches\n", (long long)T, (long long)next, n);
        std::exit(1);
    }
}

int main() {
    const int64_t unit = kNormLaunchRows, last = INT32_MAX;
    for (int64_t T = 0; T < 70; ++T) check(T);
    for (int64_t i = 1; i * unit <= last + 1; ++i)
        for (int64_t d = -3; d <= 3; ++d)
            if (i * unit + d <= last) check(i * unit + d);
    for (int64_t T = last - 3; T <= last; ++T) check(T);
    std::printf("ok\n");
    return 0;
}
