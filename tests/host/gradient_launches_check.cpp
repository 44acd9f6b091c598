// Host check of the launches behind the experts' products and the gradients, at the
// largest sizes that the calls take: the library's host code, with the runtime's launch
// replaced by one that writes down grid and arguments.  A launch holds fewer than 2^32 lanes
// (the runtime refuses more), and a routing gradient's launches cover its tokens in order.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdio>
#include <cstdlib>

#include "moe_glue.h"

namespace {

struct Launch {
    uint64_t lanes;
    const int32_t* ids;  // a routing gradient's first and fourth argument
    int tokens;
};
Launch launches[1 << 12];
int count = 0;
dim3 grid_now, block_now;
const char* what = "";
bool routing = false;

[[noreturn]] void failed(const char* why, long long a, long long b) {
    std::printf("FAIL %s: %s (%lld, %lld)\n", what, why, a, b);
    std::exit(1);
}

// Runs one call; every launch fits.
template <class Call>
void call(const char* name, int least, Call&& f) {
    what = name;
    count = 0;
    const moe_status s = f();
    if (s != MOE_OK) failed(moe_last_error(), s, 0);
    if (count < least) failed("launches", count, least);
    for (int i = 0; i < count; ++i)
        if (launches[i].lanes >= 1ull << 32) failed("lanes of a launch", i, (long long)launches[i].lanes);
}

}  // namespace

extern "C" {
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t, hipStream_t) {
    grid_now = grid;
    block_now = block;
    return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* shared, hipStream_t* stream) {
    *grid = grid_now;
    *block = block_now;
    *shared = 0;
    *stream = nullptr;
    return hipSuccess;
}
hipError_t hipLaunchKernel(const void*, dim3 grid, dim3 block, void** args, size_t, hipStream_t) {
    if (count == 1 << 12) failed("too many launches", count, 0);
    Launch& l = launches[count++];
    l.lanes = (uint64_t)grid.x * block.x * grid.y * block.y;
    if (routing) {
        l.ids = *static_cast<const int32_t**>(args[0]);
        l.tokens = *static_cast<const int*>(args[3]);
    }
    return hipSuccess;
}
hipError_t hipGetLastError() { return hipSuccess; }
}

int main() {
    auto* h = reinterpret_cast<uint16_t*>(4096);  // never read
    auto* b = reinterpret_cast<uint8_t*>(4096);
    auto* f = reinterpret_cast<float*>(4096);
    auto* i = reinterpret_cast<int32_t*>(4096);
    const int32_t most = INT32_MAX - 1;

    call("swiglu_backward", 1, [&] { return moe_swiglu_backward(h, h, most, 8, h, h, nullptr); });
    call("combine_backward", 1, [&] { return moe_combine_backward(h, h, f, i, most, 8, 1, h, f, nullptr); });
    call("combine_backward, wide", 1, [&] { return moe_combine_backward(h, h, f, i, most / 128, 1024, 16, h, f, nullptr); });
    call("expand_rows_backward", 1, [&] { return moe_expand_rows_backward(h, i, h, most, 8, 1, h, nullptr); });
    // most tiles: 2^22
    const int32_t rows = ((1 << 22) - 8) * 64;
    call("grouped_linear", 1, [&] {
        return moe_grouped_linear(h, rows, i, nullptr, h, 8, 64, 64, nullptr, MOE_ACT_NONE, nullptr, nullptr, h, nullptr);
    });
    call("grouped_linear, dense", 1, [&] {
        return moe_grouped_linear(h, 1 << 16, nullptr, nullptr, h, 1, 1 << 20, 64, nullptr, MOE_ACT_SWIGLU, nullptr, h, h,
                                  nullptr);
    });
    call("grouped_linear_mxfp8", 1, [&] {
        return moe_grouped_linear_mxfp8(b, b, rows, i, i, b, b, 8, 64, 64, nullptr, MOE_ACT_NONE, nullptr, nullptr, h,
                                        nullptr);
    });
    call("grouped_linear_grad_x", 1, [&] { return moe_grouped_linear_grad_x(h, rows, i, nullptr, h, 8, 64, 64, h, nullptr); });
    call("grouped_linear_grad_w", 1, [&] {
        return moe_grouped_linear_grad_w(h, h, 1 << 20, i, nullptr, 512, 1 << 20, 8, 1, h, f, nullptr, 0, nullptr);
    });
    call("grouped_linear_grad_w, pieces", 2, [&] {
        return moe_grouped_linear_grad_w(h, h, most - 6, nullptr, nullptr, 1, 8, 8, 1, h, f, h, SIZE_MAX, nullptr);
    });

    routing = true;
    for (int32_t E : {1, 2, 7, 8, 31, 64, 512})
        for (int32_t T : {1, 5, INT32_MAX / 2 / E, (INT32_MAX - 1) / E, 1 << 22}) {
            if ((int64_t)T * E >= INT32_MAX) continue;
            call("route_backward", 1, [&] { return moe_route_backward(i, f, f, T, E, 1, f, nullptr, nullptr); });
            int64_t next = 0;
            for (int l = 0; l < count; ++l) {
                const int64_t at = launches[l].ids - i;
                if (at != next || launches[l].tokens < 1) failed("tokens of a launch", at, next);
                next += launches[l].tokens;
                if (launches[l].lanes < (uint64_t)launches[l].tokens * 64) failed("a wave a token", l, next);
            }
            if (next != T) failed("tokens", next, T);
        }
    std::printf("ok\n");
    return 0;
}
