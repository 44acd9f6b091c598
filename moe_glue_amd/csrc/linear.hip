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

template <int NT>
__global__ __launch_bounds__(kThreads) void linear_mxfp4_kernel(const uint16_t* __restrict__ x, int T, int K,
                                                                const uint8_t* __restrict__ w,
                                                                const uint8_t* __restrict__ sc, int N,
                                                                uint16_t* __restrict__ y) {
    __shared__ f32x4 s_part[kWaves][NT][kWave];
    const int lane = (int)(threadIdx.x % kWave);
    const int wave = (int)(threadIdx.x / kWave);
    const int n0 = (int)blockIdx.x * 16;
    const size_t row = (size_t)min(n0 + lane % 16, N - 1);
    const WeightRow rows[1] = {{w + row * Mxfp4Weights::row_bytes(K), sc + row * Mxfp4Weights::row_scales(K)}};
    const uint16_t* cols[NT];
    f32x4 acc[1][NT];
#pragma unroll
    for (int c = 0; c < NT; ++c) {
        cols[c] = x + (size_t)min(c * 16 + lane % 16, T - 1) * K;
        acc[0][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    const int steps = (K + Mxfp4Weights::STEP - 1) / Mxfp4Weights::STEP;
    multiply_rows<Mxfp4Weights, 1, NT>(rows, cols, K, steps * wave / kWaves, steps * (wave + 1) / kWaves, acc);
#pragma unroll
    for (int c = 0; c < NT; ++c) s_part[wave][c][lane] = acc[0][c];
    __syncthreads();
    for (int i = (int)threadIdx.x; i < NT * 256; i += kThreads) {
        const int c = i / 256, l = i % 256 / 4, v = i % 4;
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < kWaves; ++k) sum += s_part[k][c][l][v];
        const int t = c * 16 + l % 16, n = n0 + l / 16 * 4 + v;
        if (t < T && n < N) y[(size_t)t * N + n] = (uint16_t)(pack_bf16x2(sum, 0.0f) & 0xFFFFu);
    }
}

template <int NT>
hipError_t launch_nt(const void* x, int T, int K, const uint8_t* w, const uint8_t* scales, int N, void* y,
                     hipStream_t stream) {
    linear_mxfp4_kernel<NT><<<(N + 15) / 16, kThreads, 0, stream>>>(static_cast<const uint16_t*>(x), T, K, w, scales,
                                                                    N, static_cast<uint16_t*>(y));
    return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_mxfp4(const void* x, int T, int K, const uint8_t* w, const uint8_t* scales, int N, void* y,
                               hipStream_t stream) {
    if (T <= 16) return launch_nt<1>(x, T, K, w, scales, N, y, stream);
    if (T <= 32) return launch_nt<2>(x, T, K, w, scales, N, y, stream);
    return launch_nt<4>(x, T, K, w, scales, N, y, stream);
}

}  // namespace moe
