// moe_grouped_linear, moe_grouped_linear_mxfp8 and moe_grouped_linear_grad_x on
// gfx950: rows in expert order times their experts' weights, with bias, SwiGLU
// and residual in the epilogue (forward), or times the weights' rows (dx = dy W).
#include "grouped.h"

namespace moe {
namespace {

constexpr int NT = 4;               // 16-column tiles of a wave
constexpr int kCols = 64 * NT;      // columns of a workgroup's tile
constexpr int kScalePieces = 16;    // scale bytes of a row fetched at a time: 4 steps

template <int MT, bool BT, bool MX>
struct Shape {
    static constexpr int AJ = (MT + 1) / 2;
    static constexpr int A_BYTES = AJ * 64 * kStepBytes;
    static constexpr int STAGE = A_BYTES + kCols * kStepBytes;
    static constexpr int SCALES = MX ? 2 * (AJ * 64 + kCols) * kScalePieces : 0;
    static constexpr int FIT = (kLdsBytes - SCALES) / STAGE;
    static constexpr int STAGES = FIT > 4 ? 4 : FIT;
    static constexpr int LOADS = AJ + NT;  // of a wave, per stage
    static_assert(STAGES >= 2, "a stage in flight beside the one multiplied");
};

// silu(g) u in fp32, as moe_swiglu has it.
__device__ __forceinline__ float silu_mul(float g, float u) {
    const float e = __builtin_amdgcn_exp2f(-g * 1.4426950408889634f);
    return g * __builtin_amdgcn_rcpf(1.0f + e) * u;
}

__device__ __forceinline__ u32x4 load8(const uint16_t* p) { return *reinterpret_cast<const u32x4*>(p); }
__device__ __forceinline__ void add8(float (&v)[8], const u32x4& b) {
    float w[8];
    unpack8(b, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += w[i];
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) { *reinterpret_cast<u32x4*>(p) = pack8(v); }

// 16 scale bytes from byte `at` of a row of n on; bytes past the row are 0.
__device__ __forceinline__ u32x4 load_scale_piece(const uint8_t* row, int at, int n) {
    u32x4 v = {0, 0, 0, 0};
    if (at + kScalePieces <= n) {
        __builtin_memcpy(&v, row + at, kScalePieces);
    } else {
#pragma unroll
        for (int i = 0; i < kScalePieces; ++i)
            if (at + i < n) v[i / 4] |= (uint32_t)row[at + i] << (i % 4 * 8);
    }
    return v;
}

template <int MT, bool BT, bool MX, bool SWIGLU>
__device__ __forceinline__ void product(const GroupedArgs& g, const Tile& t, uint8_t* lds) {
    using S = Shape<MT, BT, MX>;
    const int lane = (int)(threadIdx.x % kWave), wave = (int)uniform(threadIdx.x / kWave);
    const int wm = wave / 4, wn = wave % 4;
    constexpr int EL = MX ? 1 : 2;
    const int out_cols = SWIGLU ? g.N / 2 : g.N;
    const int col0 = t.col * (SWIGLU ? kCols / 2 : kCols);  // of the output
    const uint32_t lda = (uint32_t)g.K * EL;
    const int steps = (int)((lda + kStepBytes - 1) / kStepBytes);

    RowsOperand<S::AJ> a;
    a.set(static_cast<const uint8_t*>(g.x) + (int64_t)t.first * lda, (int64_t)t.rows * lda, lda, wave * 8, 64);
    RowsOperand<BT ? 1 : NT> br;
    ColumnsOperand<BT ? NT : 1> bc;
    const uint8_t* w = static_cast<const uint8_t*>(g.w) + (int64_t)t.e * g.N * g.K * EL;
    if constexpr (BT) {  // w [K, N], the sum over its rows
        bc.set(w + (int64_t)col0 * EL, (int64_t)g.K * g.N * EL - (int64_t)col0 * EL, (uint32_t)g.N * EL);
    } else if constexpr (SWIGLU) {
        // LDS rows 64 j + 0..31 are gate rows, 64 j + 32..63 the up rows of the same columns
        const int64_t row = (int64_t)(wave / 4) * out_cols + col0;
        br.set(w + row * lda, (int64_t)(out_cols - col0) * lda, lda, wave % 4 * 8, 32);
    } else {
        br.set(w + (int64_t)col0 * lda, (int64_t)(g.N - col0) * lda, lda, wave * 8, 64);
    }

    // MXFP8: thread i fetches the scales of LDS row i (of x, then of w), four
    // steps at a time, one such piece ahead
    const int scale_row = (int)threadIdx.x;
    const bool has_scales = MX && scale_row < S::AJ * 64 + kCols;
    const uint8_t* scale_base = nullptr;
    u32x4 scale_next = {0, 0, 0, 0};
    const int scale_n = g.K / 32;
    if constexpr (MX) {
        if (scale_row < S::AJ * 64) {
            scale_base = g.xs + (int64_t)(t.first + min(scale_row, t.rows - 1)) * scale_n;
        } else {
            const int r = scale_row - S::AJ * 64;
            const int row = SWIGLU ? min(col0 + r / 64 * 32 + r % 32, out_cols - 1) + (r % 64 / 32) * out_cols
                                   : min(col0 + r, g.N - 1);
            scale_base = g.ws + ((int64_t)t.e * g.N + (has_scales ? row : 0)) * scale_n;
        }
        if (has_scales) scale_next = load_scale_piece(scale_base, 0, scale_n);
    }
    uint8_t* const lds_scales = lds + S::STAGES * S::STAGE;
    constexpr int SCALE_BUF = (S::AJ * 64 + kCols) * kScalePieces;

    const auto load = [&](int step, int buf) {
        uint8_t* p = lds + buf * S::STAGE;
        a.load(step, p);
        if constexpr (BT)
            bc.load(step, p + S::A_BYTES);
        else
            br.load(step, p + S::A_BYTES);
    };

    f32x4 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    const uint32_t a_at = (uint32_t)(wm * MT * 16) * kStepBytes + rows_at(lane % 16, lane / 16);
    const uint32_t b_at = S::A_BYTES + (BT ? columns_at<kCols * 2>()
                                           : (uint32_t)(wn * NT * 16) * kStepBytes + rows_at(lane % 16, lane / 16));

#pragma unroll
    for (int s = 0; s < S::STAGES - 1; ++s)
        if (s < steps) load(s, s);
    int buf = 0;
    for (int step = 0; step < steps; ++step) {
        if constexpr (MX) {
            if (step % 4 == 0 && has_scales)
                *reinterpret_cast<u32x4*>(lds_scales + step / 4 % 2 * SCALE_BUF + scale_row * kScalePieces) = scale_next;
        }
        if (step + S::STAGES - 1 <= steps)
            wait_and_meet<(S::STAGES - 2) * S::LOADS>();
        else
            wait_and_meet<0>();
        if constexpr (MX) {
            if (step % 4 == 0 && has_scales && step + 4 < steps)
                scale_next = load_scale_piece(scale_base, (step / 4 + 1) * kScalePieces, scale_n);
        }
        const int ahead = buf == 0 ? S::STAGES - 1 : buf - 1;
        if (step + S::STAGES - 1 < steps) load(step + S::STAGES - 1, ahead);
        const uint8_t* p = lds + buf * S::STAGE;
        if constexpr (MX) {
            const uint8_t* sp = lds_scales + step / 4 % 2 * SCALE_BUF + step % 4 * 4 + lane / 16;
            i32x8 bv[NT];
            int bs[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const i32x4 lo = *reinterpret_cast<const i32x4*>(p + b_at + j * 2048);
                const i32x4 hi = *reinterpret_cast<const i32x4*>(p + ((b_at + j * 2048) ^ 64));
                bv[j] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
                bs[j] = sp[(S::AJ * 64 + wn * NT * 16 + j * 16 + lane % 16) * kScalePieces];
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const i32x4 lo = *reinterpret_cast<const i32x4*>(p + a_at + i * 2048);
                const i32x4 hi = *reinterpret_cast<const i32x4*>(p + ((a_at + i * 2048) ^ 64));
                const i32x8 av = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
                const int as = sp[(wm * MT * 16 + i * 16 + lane % 16) * kScalePieces];
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bv[j], av, acc[i][j], 0, 0, 0, bs[j],
                                                                                0, as);
            }
        } else {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                bf16x8 av[MT], bv[NT];
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    if constexpr (BT)
                        bv[j] = columns_fragment<kCols * 2>(p, (b_at + s * 32 * kCols * 2) ^ (wn * NT + j) * 32);
                    else
                        bv[j] = *reinterpret_cast<const bf16x8*>(p + ((b_at + j * 2048) ^ s * 64));
                }
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    av[i] = *reinterpret_cast<const bf16x8*>(p + ((a_at + i * 2048) ^ s * 64));
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bv[j], av[i], acc[i][j], 0, 0, 0);
            }
        }
        buf = buf + 1 == S::STAGES ? 0 : buf + 1;
    }

    // epilogue: 8 columns of one row a lane and tile pair
    const int pc = pair_column();
    u32x4 bias[NT / 2];  // of the pairs' columns; behind SwiGLU of gate and up
    if (g.bias != nullptr) {
#pragma unroll
        for (int j = 0; j < NT / 2; ++j) {
            const int c = col0 + (SWIGLU ? wn * 32 : wn * NT * 16 + j * 32) + pc;
            if (c < out_cols) bias[j] = load8(g.bias + (int64_t)t.e * g.N + c + (SWIGLU ? j * out_cols : 0));
        }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int m = wm * MT * 16 + i * 16 + lane % 16;
        const int64_t row = t.first + m;
        if constexpr (SWIGLU) {
            float gate[8], up[8];
            pair_values(acc[i][0], acc[i][1], gate);
            pair_values(acc[i][2], acc[i][3], up);
            const int c = col0 + wn * 32 + pc;
            if (m < t.rows && c < out_cols) {
                if (g.bias != nullptr) {
                    add8(gate, bias[0]);
                    add8(up, bias[1]);
                }
                if (g.pre != nullptr) {
                    store8(g.pre + row * g.N + c, gate);
                    store8(g.pre + row * g.N + out_cols + c, up);
                }
#pragma unroll
                for (int q = 0; q < 8; ++q) gate[q] = silu_mul(gate[q], up[q]);
                if (g.residual != nullptr) add8(gate, load8(g.residual + row * out_cols + c));
                store8(g.out + row * out_cols + c, gate);
            }
        } else {
#pragma unroll
            for (int j = 0; j < NT; j += 2) {
                float v[8];
                pair_values(acc[i][j], acc[i][j + 1], v);
                const int c = col0 + (wn * NT + j) * 16 + pc;
                if (m < t.rows && c < out_cols) {
                    if (g.bias != nullptr) add8(v, bias[j / 2]);
                    if (g.residual != nullptr) add8(v, load8(g.residual + row * out_cols + c));
                    store8(g.out + row * out_cols + c, v);
                }
            }
        }
    }
}

template <bool BT, bool MX, bool SWIGLU>
__global__ __launch_bounds__(kGroupedThreads) void grouped_kernel(GroupedArgs g, int col_tiles) {
    __shared__ __align__(16) uint8_t lds[kLdsBytes];
    const Tile t = find_tile(g.rows, col_tiles);
    if (t.e < 0) return;
    if (t.last_rows > 192)
        product<8, BT, MX, SWIGLU>(g, t, lds);
    else if (t.last_rows > 128)
        product<6, BT, MX, SWIGLU>(g, t, lds);
    else if (t.last_rows > 64)
        product<4, BT, MX, SWIGLU>(g, t, lds);
    else if (t.last_rows > 32)
        product<2, BT, MX, SWIGLU>(g, t, lds);
    else
        product<1, BT, MX, SWIGLU>(g, t, lds);
}

template <bool BT, bool MX, bool SWIGLU>
hipError_t launch(const GroupedArgs& g, hipStream_t stream) {
    const int cols = SWIGLU ? kCols / 2 : kCols, out_cols = SWIGLU ? g.N / 2 : g.N;
    const int col_tiles = (out_cols + cols - 1) / cols;
    const int64_t tiles = grouped_tiles(g.rows, col_tiles);
    const uint32_t grid = (uint32_t)((tiles + 7) / 8 * 8);
    grouped_kernel<BT, MX, SWIGLU><<<grid, kGroupedThreads, 0, stream>>>(g, col_tiles);
    return hipGetLastError();
}

}  // namespace

int64_t grouped_linear_tiles(const GroupedRows& rows, int cols, bool swiglu) {
    return grouped_tiles(rows, swiglu ? (cols / 2 + kCols / 2 - 1) / (kCols / 2) : (cols + kCols - 1) / kCols);
}

hipError_t launch_grouped_linear(const GroupedArgs& g, bool swiglu, hipStream_t stream) {
    if (g.xs != nullptr) return swiglu ? launch<false, true, true>(g, stream) : launch<false, true, false>(g, stream);
    return swiglu ? launch<false, false, true>(g, stream) : launch<false, false, false>(g, stream);
}

hipError_t launch_grouped_grad_x(const GroupedArgs& g, hipStream_t stream) {
    return launch<true, false, false>(g, stream);
}

}  // namespace moe
