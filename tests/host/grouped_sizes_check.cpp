// Host check of the grouped products' arithmetic on sizes, built to trap on signed
// overflow: the pieces of an expert's rows, to the largest row count (for which the
// workspace has a size), and widths near 2^31, refused before
// anything is computed from them.
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

static void expect(moe_status got, moe_status want, const char* what, int32_t N, int32_t K) {
    if (got != want) {
        std::printf("FAIL %s N=%d K=%d: status %d\n", what, N, K, (int)got);
        std::exit(1);
    }
}

int main() {
    const int64_t last = INT32_MAX;
    for (int64_t piece : {1024, 1056, 4096, 1 << 20, 4194304, 1 << 30})
        for (int64_t n : {(int64_t)0, (int64_t)1, piece - 1, piece, piece + 1, 2 * piece, 2 * piece + 1, last / piece * piece,
                          last / piece * piece + 1, last - 7, last - 1, last})
            if (n <= last) check_pieces(n, piece);

    std::printf("pieces\n");
    std::fflush(stdout);
    auto* p = reinterpret_cast<uint16_t*>(4096);  // never read: every call here is refused
    auto* b = reinterpret_cast<uint8_t*>(4096);
    auto* i = reinterpret_cast<int32_t*>(4096);
    for (int32_t w : {(1 << 20) + 32, 1 << 21, INT32_MAX - 127, INT32_MAX - 31}) {  // multiples of 32
        for (int swap = 0; swap < 2; ++swap) {
            const int32_t N = swap ? w : 64, K = swap ? 64 : w;
            expect(moe_grouped_linear(p, 4, i, nullptr, p, 4, N, K, nullptr, MOE_ACT_NONE, nullptr, nullptr, p, nullptr),
                   MOE_ERR_UNSUPPORTED, "linear", N, K);
            expect(moe_grouped_linear(p, 4, i, nullptr, p, 4, N, K, nullptr, MOE_ACT_SWIGLU, nullptr, nullptr, p, nullptr),
                   MOE_ERR_UNSUPPORTED, "swiglu", N, K);
            expect(moe_grouped_linear_mxfp8(b, b, 4, i, nullptr, b, b, 4, N, K, nullptr, MOE_ACT_NONE, nullptr, nullptr, p,
                                            nullptr),
                   MOE_ERR_UNSUPPORTED, "mxfp8", N, K);
            expect(moe_grouped_linear_grad_x(p, 4, i, nullptr, p, 4, N, K, p, nullptr), MOE_ERR_UNSUPPORTED, "grad_x", N, K);
            expect(moe_grouped_linear_grad_w(p, p, 4, i, nullptr, 4, N, K, 0, p, nullptr, nullptr, 0, nullptr),
                   MOE_ERR_UNSUPPORTED, "grad_w", N, K);
            if (moe_grouped_linear_grad_w_workspace_bytes(4, 4, N, K) != 0) {
                std::printf("FAIL workspace N=%d K=%d\n", N, K);
                return 1;
            }
        }
    }
    std::printf("widths\n");
    std::fflush(stdout);
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
