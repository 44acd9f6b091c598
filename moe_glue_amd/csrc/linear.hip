// moe_linear_mxfp4 on gfx950: y = x W^T for up to 64 tokens, W in MXFP4.
//
// Bound by the stream of W (17 bits for 4 weights) as long as tokens are few: a
// workgroup owns 16 rows of W, its eight waves split K, their partial sums meet
// in LDS, and products are those of mfma_rows.h: every wave loads its operands
// straight to registers.  x is then read once per 16 rows of W and column tile,
// which grows with T x N until it outweighs W; from there on (launch_linear_mxfp4
// has the sizes) both are staged through LDS.
#include "kernels.h"
#include "mfma_rows.h"

namespace moe {
namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / kWave;

constexpr int kCus = 256;
constexpr int kTiles = 4;  // row tiles of a workgroup: 16 rows of W

template <int NT>
__global__ __launch_bounds__(kThreads, NT == 1 ? 4 : 2) void linear_mxfp4_kernel(
    const uint16_t* __restrict__ x, int T, int K, const uint8_t* __restrict__ w, const uint8_t* __restrict__ sc, int N,
    uint16_t* __restrict__ y) {
    using W = Mxfp4Weights;
    __shared__ float s_sums[kWaves][NT][kTiles][16];
    const int lane = (int)(threadIdx.x % kWave);
    const int wave = wave_index();
    const int n0 = (int)blockIdx.x * (4 * kTiles);
    const int c0 = (int)blockIdx.y * (4 * NT);
    const uint32_t row_bytes = W::bytes_of((uint32_t)K), row_scales = W::row_scales(K);
    RowTiles<kTiles> rows;
    uint32_t col[1][NT];
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
        col[0][c] = t < T ? (uint32_t)t * (uint32_t)K * 2 : kNowhere;
    }
    const int steps = steps_of<W>(K);
    const __amdgpu_buffer_rsrc_t wb = buffer_of(w + (size_t)n0 * row_bytes, (size_t)(N - n0) * row_bytes);
    multiply_rows<W, kTiles, NT, (NT == 2 ? 4 : 2), kCacheNt, 1>(
        wb, wb, rows, buffer_of(x, (size_t)T * K * 2), col, K, steps * wave / kWaves, steps * (wave + 1) / kWaves, acc);
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

// More tokens: W and x staged through LDS, tiles of v_mfma_f32_16x16x32_bf16 in
// their plain form (row and column l % 16, k quarter l / 16).  A workgroup owns
// 16 R rows of W and all tokens (16 NT of them); a chunk is 256 k of both, and
// each of the eight waves takes 32 k of it, one scale block, so the operands are
// read from LDS once per 16 R x 16 NT products.  Chunks are fetched kAhead ahead
// into registers and pass through two LDS buffers with one barrier each.  Rows
// of LDS are padded by 16 bytes: the 16 rows a fragment read touches then fall
// into different banks.  A chunk's LDS writes, loads, LDS reads and products go
// by turns, a fourth of each at a time: all of one kind and then all of the next
// queue up behind each other (64 tokens, 7168 x 16384: 31.0 us, by turns 27.7;
// without any loads 21, so LDS and products are most of it).  Waves with chunks
// and LDS of their own, without barriers, measured 10 to 15 % less below 8192
// rows of W and 25 % more above, where their shorter pieces of a row cost HBM.
constexpr int kChunk = 256;
// chunks in flight, by registers
template <int NT>
constexpr int kAheadOf = NT == 1 ? 8 : NT == 2 ? 4 : 2;
constexpr int kXStride = kChunk * 2 + 16;
constexpr int kWStride = kChunk / 2 + 16;

template <int R, int NT>
struct WideShared {
    union {
        struct {
            uint8_t x[2][16 * NT][kXStride];
            uint8_t w[2][16 * R][kWStride];
            uint8_t sc[2][16 * R][kChunk / 32];
        };
        f32x4 part[kWaves][R][kWave];  // the waves' sums of one column tile
    };
};

template <int R, int NT>
__global__ __launch_bounds__(kThreads) void linear_mxfp4_wide_kernel(const uint16_t* __restrict__ x, int T, int K,
                                                                     const uint8_t* __restrict__ w,
                                                                     const uint8_t* __restrict__ sc, int N,
                                                                     uint16_t* __restrict__ y) {
    static_assert(R * 128 <= kThreads, "a piece of w and a scale byte a thread");
    constexpr int kAhead = kAheadOf<NT>;
    __shared__ __align__(16) WideShared<R, NT> sh;
    const int tid = (int)threadIdx.x;
    const int lane = tid % kWave;
    const int wave = wave_index();
    const int n0 = (int)blockIdx.x * (16 * R);
    const int chunks = (K + kChunk - 1) / kChunk;

    // this thread's pieces: 16 bytes of one row of w, one of its scale bytes, 16
    // bytes of NT rows of x.  Rows past the last repeat it, and are not stored.
    const int w_row = tid / 8 % (16 * R), w_piece = tid % 8;
    const bool has_w = tid < R * 128;
    const uint32_t row_bytes = Mxfp4Weights::bytes_of((uint32_t)K), row_scales = Mxfp4Weights::row_scales(K);
    const __amdgpu_buffer_rsrc_t wb = buffer_of(w + (size_t)n0 * row_bytes, (size_t)(N - n0) * row_bytes);
    const __amdgpu_buffer_rsrc_t sb = buffer_of(sc + (size_t)n0 * row_scales, (size_t)(N - n0) * row_scales);
    const __amdgpu_buffer_rsrc_t xb = buffer_of(x, (size_t)T * K * 2);
    const uint32_t w_at = (uint32_t)min(w_row, N - 1 - n0) * row_bytes + (uint32_t)w_piece * 16;
    const uint32_t s_at = (uint32_t)min(w_row, N - 1 - n0) * row_scales + (uint32_t)w_piece;
    const int x_piece = tid % 32;
    uint32_t x_at[NT];
#pragma unroll
    for (int c = 0; c < NT; ++c)
        x_at[c] = (uint32_t)min(c * 16 + tid / 32, T - 1) * (uint32_t)K * 2 + (uint32_t)x_piece * 16;
    u32x4 wv[kAhead], xv[kAhead][NT];
    uint8_t sv[kAhead];
    const auto fetch_w = [&](auto index, int chunk) {
        constexpr int j = decltype(index)::value;
        // past K: zeros (codes of zero under scale byte 0).  With R < 4 several waves
        // load the same piece, and the first of them stages it.
        const bool in_w = chunk * kChunk + w_piece * 32 < K;
        wv[j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                              wb, (int)(in_w ? w_at : kNowhere), chunk * (kChunk / 2), kCacheNt));
        sv[j] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(sb, (int)(in_w ? s_at : kNowhere),
                                                             chunk * (kChunk / 32), 0);
    };
    const auto fetch_x = [&](auto index, int chunk, int c) {
        constexpr int j = decltype(index)::value;
        const bool in_x = chunk * kChunk + x_piece * 8 < K;
        xv[j][c] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                 xb, (int)(in_x ? x_at[c] : kNowhere), chunk * (kChunk * 2), 0));
    };
    const auto fetch = [&](auto index, int chunk) {
        fetch_w(index, chunk);
#pragma unroll
        for (int c = 0; c < NT; ++c) fetch_x(index, chunk, c);
    };
    f32x4 acc[R][NT];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < NT; ++c) acc[r][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    const auto to_lds_w = [&](auto index, int buf) {
        constexpr int j = decltype(index)::value;
        if (has_w) {
            *reinterpret_cast<u32x4*>(&sh.w[buf][w_row][w_piece * 16]) = wv[j];
            sh.sc[buf][w_row][w_piece] = sv[j];
        }
    };
    const auto to_lds_x = [&](auto index, int buf, int c) {
        constexpr int j = decltype(index)::value;
        *reinterpret_cast<u32x4*>(&sh.x[buf][c * 16 + tid / 32][x_piece * 16]) = xv[j][c];
    };
    const auto to_lds = [&](auto index, int buf) {
        to_lds_w(index, buf);
#pragma unroll
        for (int c = 0; c < NT; ++c) to_lds_x(index, buf, c);
    };
    // this wave's operands of a chunk, out of LDS a chunk ahead of their use
    uint32_t codes[2][R], scale[2][R];
    u32x4 b[2][NT];
    const auto from_lds_w = [&](int buf, int r) {
        const int row = r * 16 + lane % 16;
        codes[buf][r] = *reinterpret_cast<const uint32_t*>(&sh.w[buf][row][wave * 16 + lane / 16 * 4]);
        scale[buf][r] = sh.sc[buf][row][wave];
    };
    const auto from_lds_x = [&](int buf, int c) {
        b[buf][c] = *reinterpret_cast<const u32x4*>(&sh.x[buf][c * 16 + lane % 16][wave * 64 + lane / 16 * 16]);
    };
    const auto from_lds = [&](int buf) {
#pragma unroll
        for (int r = 0; r < R; ++r) from_lds_w(buf, r);
#pragma unroll
        for (int c = 0; c < NT; ++c) from_lds_x(buf, c);
    };
    // Chunk c: its operands are in registers, chunk c + 1 is in LDS (all waves
    // past the barrier have its pieces in, and have read chunk c out).  Chunk
    // c + 2 takes chunk c's buffer, and its registers chunk c + 2 + kAhead.
    const auto step = [&](auto index, int chunk) {
        constexpr int buf = decltype(index)::value % 2;
        const int next = min(chunk + 2 + kAhead, chunks - 1);  // (behind the last: the last again, not used)
        const auto products = [&](int r) {
            const bf16x8 a = Mxfp4Weights::values<0>(u32x2{codes[buf][r], 0u},
                                                     __builtin_bit_cast(float, scale[buf][r] << 23));
#pragma unroll
            for (int c = 0; c < NT; ++c)
                acc[r][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8, b[buf][c]),
                                                                    acc[r][c], 0, 0, 0);
        };
        __syncthreads();  // chunk + 1 is in LDS, and all have read this one out
#pragma unroll
        for (int i = 0; i < (R > NT ? R : NT); ++i) {
            if (i == 0) to_lds_w(index, buf);
            if (i < NT) to_lds_x(index, buf, i);
            if (i == 0) fetch_w(index, next);
            if (i < NT) fetch_x(index, next, i);
            if (i < R) from_lds_w(1 - buf, i);
            if (i < NT) from_lds_x(1 - buf, i);
            if (i < R) products(i);
            __builtin_amdgcn_sched_barrier(0);  // (the compiler would gather them by kind)
        }
    };
    constexpr std::integral_constant<int, 0> first{};
    constexpr std::integral_constant<int, 1> second{};
    fetch(first, 0);
    fetch(second, min(1, chunks - 1));
    to_lds(first, 0);
    to_lds(second, 1);
    unrolled<kAhead>([&](auto index) { fetch(index, min(2 + (int)index, chunks - 1)); });
    __syncthreads();
    from_lds(0);
    // whole rounds without a condition on their loads (see multiply_rows), then
    // the chunks that are left
    int chunk0 = 0;
    for (; chunk0 + kAhead <= chunks; chunk0 += kAhead)
        unrolled<kAhead>([&](auto index) { step(index, chunk0 + index); });
    unrolled<kAhead>([&](auto index) {
        if (chunk0 + index < chunks) step(index, chunk0 + index);
    });
    // the waves' sums, a column tile at a time; a thread adds up four rows of one
    // token, 16 bytes from each wave
    const auto sum_column = [&](auto index) {
        constexpr int c = decltype(index)::value;
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r) sh.part[wave][r][lane] = acc[r][c];
        __syncthreads();
        const int t = c * 16 + lane % 16, n = n0 + wave * 16 + lane / 16 * 4;
        if (wave < R && t < T) {
            f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < kWaves; ++k) sum += sh.part[k][wave][lane];
            uint16_t* to = y + (size_t)t * N + n;
            if (N % 4 == 0 && reinterpret_cast<uint64_t>(y) % 8 == 0) {  // uniform; then n + 3 < N where n < N
                if (n < N)
                    *reinterpret_cast<u32x2*>(to) = u32x2{pack_bf16x2(sum[0], sum[1]), pack_bf16x2(sum[2], sum[3])};
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (n + i < N) to[i] = (uint16_t)(pack_bf16x2(sum[i], 0.0f) & 0xFFFFu);
            }
        }
    };
    unrolled<NT>(sum_column);
}

template <int R, int NT>
hipError_t launch_wide(const void* x, int T, int K, const uint8_t* w, const uint8_t* scales, int N, void* y,
                       hipStream_t stream) {
    linear_mxfp4_wide_kernel<R, NT><<<(N + 16 * R - 1) / (16 * R), kThreads, 0, stream>>>(
        static_cast<const uint16_t*>(x), T, K, w, scales, N, static_cast<uint16_t*>(y));
    return hipGetLastError();
}

template <int NT>
hipError_t launch_nt(const void* x, int T, int K, const uint8_t* w, const uint8_t* scales, int N, void* y,
                     hipStream_t stream) {
    linear_mxfp4_kernel<NT><<<dim3((N + 15) / 16, (T + 4 * NT - 1) / (4 * NT)), kThreads, 0, stream>>>(
        static_cast<const uint16_t*>(x), T, K, w, scales, N, static_cast<uint16_t*>(y));
    return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_mxfp4(const void* x, int T, int K, const uint8_t* w, const uint8_t* scales, int N, void* y,
                               hipStream_t stream) {
    // The two kernels at K x N (us, rows kernel / staged one, T = 8, 16, 32, 64):
    // 1024 x 1024 4.2 / 5.1, 4.9 / 4.6, 5.0 / 5.1, 5.0 / 6.6; 7168 x 2048 7.2 /
    // 10.6, 9.9 / 11.3, 9.7 / 14.7, 16.7 / 20.7; 7168 x 4096 7.8 / 11.1, 10.2 / 11.9,
    // 17.7 / 15.5, 34 / 21.6; 2048 x 7168 7.4 / 6.9, 9.5 / 7.0, 15.1 / 8.0, 25 / 11.1;
    // 7168 x 16384 (T = 4: 15.8 / 18) 26 / 18.4, 36 / 19.6, 67 / 22.7, 129 / 27.7.
    // The rule goes by N and T alone; K was not varied at one N.
    const int from = N <= 8 * kCus ? MOE_DECODE_T_MAX : N <= 16 * kCus ? 16 : N <= 32 * kCus ? 8 : 4;
    if (T > from) {
        const int rows = N <= 16 * kCus ? 1 : N <= 32 * kCus ? 2 : 4;  // one workgroup per CU as far as N reaches
        const auto nt = [&](auto r) {
            constexpr int R = decltype(r)::value;
            if constexpr (R > 1)  // (with R = 1 the rows kernel has the batches up to 16)
                if (T <= 16) return launch_wide<R, 1>(x, T, K, w, scales, N, y, stream);
            if (T <= 32) return launch_wide<R, 2>(x, T, K, w, scales, N, y, stream);
            return launch_wide<R, 4>(x, T, K, w, scales, N, y, stream);
        };
        if (rows == 1) return nt(std::integral_constant<int, 1>{});
        if (rows == 2) return nt(std::integral_constant<int, 2>{});
        return nt(std::integral_constant<int, 4>{});
    }
    if (T <= 4) return launch_nt<1>(x, T, K, w, scales, N, y, stream);
    if (T <= 8) return launch_nt<2>(x, T, K, w, scales, N, y, stream);
    return launch_nt<4>(x, T, K, w, scales, N, y, stream);
}

}  // namespace moe
