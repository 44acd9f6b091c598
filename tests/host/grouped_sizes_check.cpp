// Host check of the grouped products' arithmetic on sizes, built to trap on signed
// overflow: the pieces of an expert's rows, to the largest row count.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <initializer_list>

#include "grouped.h"
#include "moe_glue.h"

using namespace moe;

static void check_pieces(int64_t n, int64_t piece) {
    const int64_t want = n == 0 ? 1 : (n + piece - 1) / piece;
    if (pieces_of((int)n, (int)piece) != want) {
        std::printf("FAIL %lld rows in pieces of %lld: %d\n", (long long)n, (long long)piece,
                    pieces_of((int)n, (int)piece));
        std::exit(1);
    }
}

int main() {
    const int64_t last = INT32_MAX;
    for (int64_t piece : {1024, 1056, 4096, 1 << 20, 4194304, 1 << 30})
        for (int64_t n : {(int64_t)0, (int64_t)1, piece - 1, piece, piece + 1, 2 * piece, 2 * piece + 1, last / piece * piece,
                          last / piece * piece + 1, last - 7, last - 1, last})
            if (n <= last) check_pieces(n, piece);

    // The largest batch of the narrowest rows: in pieces, with room for each one's sums.
    const int32_t R = INT32_MAX - 7;
    const GroupedRows rows = {nullptr, nullptr, 1, R};
    const size_t need = grouped_grad_w_workspace_bytes(rows, 8, 8);
    if (need == 0 || need != moe_grouped_linear_grad_w_workspace_bytes(R, 1, 8, 8)) {
        std::printf("FAIL workspace of %d rows: %zu\n", R, need);
        return 1;
    }
    std::printf("ok\n");
    return 0;
}
