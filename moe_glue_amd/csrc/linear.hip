// moe_linear_mxfp4 on gfx950: y = x W^T for up to 64 tokens, W in MXFP4.
//
// Bound by the stream of W (17 bits for 4 weights), which is read once: a
// workgroup owns 16 rows of W for every token, its eight waves split K, and
// their partial sums meet in LDS.  Products as in mfma_rows.h.
#include "kernels.h"
#include "mfma_rows.h"

namespace moe {
namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / kWave;

constexpr int kTiles = 4;  // row tiles of a workgroup: 16 rows of W

template <int NT>
__global__ __launch_bounds__(kThreads) void linear_mxfp4_kernel(const uint16_t* __restrict__ x, int T, int K,
                                                                const uint8_t* __restrict__ w,
                                                                const uint8_t* __restrict__ sc, int N,
                                                                uint16_t* __restrict__ y) {
    using W = Mxfp4Weights;
    __shared__ float s_sums[kWaves][NT][kTiles][16];
    const int lane = (int)(threadIdx.x % kWave);
    const int wave = wave_index();
    const int n0 = (int)blockIdx.x * (4 * kTiles);
    const int c0 = (int)blockIdx.y * (4 * NT);
    const uint32_t row_bytes = W::bytes_of((uint32_t)K), row_scales = W::row_scales(K);
    RowTiles<kTiles> rows;
    uint32_t col[NT];
    f32x4 acc[kTiles][NT];
#pragma unroll
    for (int r = 0; r < kTiles; ++r) {
        const int first = min(r * 4, N - 1 - n0);  // a tile past W: its last row
        rows.at[r] = (uint32_t)first * row_bytes;
        rows.scales[r] = sc + (size_t)(n0 + first) * row_scales;
        rows.last[r] = (uint32_t)min(3, N - 1 - n0 - first);
#pragma unroll
        for (int c = 0; c < NT; ++c) acc[r][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
#pragma unroll
    for (int c = 0; c < NT; ++c) {
        const int t = c0 + c * 4 + lane % 16 / 4;
        col[c] = t < T ? (uint32_t)t * (uint32_t)K * 2 : kNowhere;
    }
    const int steps = steps_of<W>(K);
    const __amdgpu_buffer_rsrc_t wb = buffer_of(w + (size_t)n0 * row_bytes, (size_t)(N - n0) * row_bytes);
    multiply_rows<W, kTiles, NT, (NT == 4 ? 2 : 4)>(wb, wb, rows, buffer_of(x, (size_t)T * K * 2), col, K,
                                                    steps * wave / kWaves, steps * (wave + 1) / kWaves, acc);
#pragma unroll
    for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int r = 0; r < kTiles; ++r) {
            const float v = diagonal_sum(acc[r][c]);
            if (lane % 4 == r) s_sums[wave][c][r][lane / 16 * 4 + lane % 16 / 4] = v;
        }
    __syncthreads();
    for (int o = (int)threadIdx.x; o < NT * 64; o += kThreads) {
        const int c = o / 64, r = o / 16 % 4, at = o % 16;
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < kWaves; ++k) sum += s_sums[k][c][r][at];
        const int t = c0 + c * 4 + at % 4, n = n0 + r * 4 + at / 4;
        if (t < T && n < N) y[(size_t)t * N + n] = (uint16_t)(pack_bf16x2(sum, 0.0f) & 0xFFFFu);
    }
}

template <int NT>
hipError_t launch_nt(const void* x, int T, int K, const uint8_t* w, const uint8_t* scales, int N, void* y,
                     hipStream_t stream) {
    linear_mxfp4_kernel<NT><<<dim3((N + 15) / 16, (T + 4 * NT - 1) / (4 * NT)), kThreads, 0, stream>>>(static_cast<const uint16_t*>(x), T, K, w, scales,
                                                                    N, static_cast<uint16_t*>(y));
    return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_mxfp4(const void* x, int T, int K, const uint8_t* w, const uint8_t* scales, int N, void* y,
                               hipStream_t stream) {
    if (T <= 4) return launch_nt<1>(x, T, K, w, scales, N, y, stream);
    if (T <= 8) return launch_nt<2>(x, T, K, w, scales, N, y, stream);
    return launch_nt<4>(x, T, K, w, scales, N, y, stream);
}

}  // namespace moe
