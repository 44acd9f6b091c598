// moe_grouped_linear, moe_grouped_linear_mxfp8 and moe_grouped_linear_grad_x on
// gfx950: rows in expert order times their experts' weights, with bias, SwiGLU
// and residual in the epilogue (forward), or times the weights' rows (dx = dy W).
//
// What bounds the products of many rows: neither the matrix cores nor LDS is near full (busy 31
// to 57 % and 15 to 30 % of a busy CU's cycles, bank conflicts 4 % at most); waves stand at
// waits and barriers for 26 to 44 % of theirs, and one workgroup a CU leaves a tile's
// first loads and its epilogue uncovered.  32768 x 1536 x 2048 over 128 experts 253 to 293 us by how
// long the card has been under load, 8192 x 7168 x 2048 222 to 241.
//
// MXFP8 operands are multiplied by the block-scaled instruction, at twice bf16's rate.  Its
// accumulators are fp32, but it adds eight neighbours along k in fixed point: of each product
// it cuts off, towards zero, what lies 2^-13 below the power of two of the largest.  (Measured:
// of 2^16 - 2^16 + 2^j in one eight 2^3 is kept and 2^2 is not, and sums formed in 64 bits with
// this cut give the kernel's every output of 256 x 256 x 2048 and 192 x 256 x 4096 normal ones.)
// Those sums are off by 1.5e-5 of their rms, 2.3e-6 of sum |x w| at the worst; the outputs' own
// rounding is 1.7e-3, and with fp32 sums it is the same to four digits.  Where the sum cancels the cut
// shows.  The way that keeps fp32's 24 bits (measured: 2^-8 beside 2^16 - 2^16) is moe_grouped_linear
// on the values, which are exact in bf16 as far as its exponents reach: 32768 x 1536 x 2048 over
// 128 experts 253 us, 161 in MXFP8.
//
// Scale rows that are not whole aligned dwords (K % 128 != 0, or a pointer off one) pass through
// registers, four byte loads a lane, whose wait every fourth step empties the loads in flight:
// 32768 x 1536 over 128 experts, K = 2880: 294 us, where 2816 takes 207 and 2944 219; dense 8192 x
// 7168: 212, 167 and 174.
#include "grouped.h"

namespace moe {
namespace {

constexpr int kCols = 256;       // columns of a workgroup's tile
constexpr int kRows = 256;       // and up to so many rows
constexpr int kScalePiece = 16;  // MXFP8 scale bytes of a row that pass through LDS at a time:
constexpr int kScaleSteps = 4;   // those of so many steps

constexpr int kBBytes = kCols * kStepBytes;
constexpr int kShortMH = 1;      // tiles of up to 64 of these rows take the short steps

// A piece of the scale bytes of 16 LDS rows into LDS, a dword a lane: lane l has
// bytes 4 (l % 4) .. + 3 of the row of scales that starts at byte `row` from base on.
__device__ __forceinline__ void load_scale_piece(const uint8_t* base, int64_t bytes, uint32_t row, int piece, uint32_t ld,
                                                 bool dwords, uint8_t* lds) {
    const uint32_t lane = threadIdx.x % kWave;
    const uint32_t k = (uint32_t)piece * kScalePiece + lane % 4 * 4;
    if (dwords) {
        load_dword_to_lds(buffer_words(base, bytes), k < ld ? row + k : kPastEnd, lds);
        return;
    }
    const __amdgpu_buffer_rsrc_t buf = grouped_buffer(base, bytes);
    uint32_t v = 0;
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) {
        const uint32_t b = __builtin_amdgcn_raw_buffer_load_b8(buf, (int)(k + i < ld ? row + k + i : kPastEnd), 0, 0);
        v |= (b & 0xFFu) << (i * 8);
    }
    *reinterpret_cast<uint32_t*>(lds + lane * 4) = v;
}

template <int MH, bool BT, bool MX, bool SWIGLU>
__device__ __forceinline__ void product(const GroupedArgs& g, const Tile& t, uint8_t* lds) {
    constexpr int EL = MX ? 1 : 2;
    constexpr int A_BYTES = MH * 64 * kStepBytes;
    constexpr int SCALE_BUF = (MH * 64 + kCols) * kScalePiece;
    constexpr bool SHORT = MH <= kShortMH;
    constexpr int STAGES = SHORT ? (kLdsBytes - (MX ? 2 * SCALE_BUF : 0)) / (A_BYTES + kBBytes) : 2;
    constexpr int B_AT = STAGES * A_BYTES, SCALES_AT = B_AT + STAGES * kBBytes;
    static_assert(STAGES >= (SHORT ? 3 : 2) && SCALES_AT + (MX ? 2 * SCALE_BUF : 0) <= kLdsBytes, "the steps in LDS");
    const int lane = (int)(threadIdx.x % kWave), wave = (int)uniform(threadIdx.x / kWave);
    const int wm = wave / 4, wn = wave % 4;
    const int out_cols = SWIGLU ? g.N / 2 : g.N;
    const int col0 = t.col * (SWIGLU ? kCols / 2 : kCols);  // of the output
    const uint32_t ld = (uint32_t)g.K * EL;
    const int steps = (int)((ld + kStepBytes - 1) / kStepBytes);

    // The tile's columns are in halves of 128, those of the rows of w from w_row[h] on:
    // with SwiGLU the gates and the ups of the same 128.  A wave has 32 of either.
    const int w_left = out_cols - col0;
    const int64_t w_row = (int64_t)t.e * g.N + col0;
    const int64_t w_row1 = w_row + (SWIGLU ? out_cols : 128);
    const int w_left1 = SWIGLU ? w_left : max(w_left - 128, 0);
    const uint8_t* w = static_cast<const uint8_t*>(g.w);

    RowsOperand<MH> a;
    a.set(ld);
    const BufferWords a_buf =
        buffer_words(static_cast<const uint8_t*>(g.x) + (int64_t)t.first * ld, (int64_t)t.rows * ld);
    RowsOperand<2> br;
    ColumnsOperand<kCols * 2, 64, 8> bc;
    BufferWords b_buf[2];
    if constexpr (BT) {  // w [K, N], the sum over its rows
        bc.set(w + ((int64_t)t.e * g.K * g.N + col0) * 2, ((int64_t)g.K * g.N - col0) * 2, (uint32_t)g.N * 2);
    } else {
        br.set(ld);
        b_buf[0] = buffer_words(w + w_row * ld, (int64_t)w_left * ld);
        b_buf[1] = buffer_words(w + w_row1 * ld, (int64_t)w_left1 * ld);
    }

    // MXFP8 scales of the steps from `step` on: 16 LDS rows a load
    const auto load_scales = [&](int step) {
        const int piece = step / kScaleSteps;
        const uint32_t n = (uint32_t)g.K / 32;
        uint8_t* p = lds + SCALES_AT + piece % 2 * SCALE_BUF;
#pragma unroll
        for (int j = 0; j < (MH + 1) / 2; ++j) {
            const int block = j * 8 + wave;
            if (MH % 2 == 0 || block < 4 * MH)
                load_scale_piece(g.xs + (int64_t)t.first * n, (int64_t)t.rows * n,
                                 (uint32_t)(block * 16 + lane / 4) * n, piece, n, g.scale_dwords, p + block * 256);
        }
        p += MH * 64 * kScalePiece;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            load_scale_piece(g.ws + (h == 0 ? w_row : w_row1) * n, (int64_t)(h == 0 ? w_left : w_left1) * n,
                             (uint32_t)(wave * 16 + lane / 4) * n, piece, n, g.scale_dwords, p + (h * 8 + wave) * 256);
        }
    };

    f32x4 acc[2][MH][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < MH; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[h][i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    using BFragment = std::conditional_t<BT, ColumnsFragment<kCols * 2, 64>, RowsFragment>;
    const uint32_t a_at = (uint32_t)(wm * MH * 16) * kStepBytes + RowsFragment::at();
    const uint32_t b_at = B_AT + BFragment::at() + (BT ? 0u : (uint32_t)(wn * 32) * kStepBytes);
    const uint32_t a_scale_at = SCALES_AT + (uint32_t)(wm * MH * 16 + lane % 16) * kScalePiece + lane / 16;
    const uint32_t b_scale_at = SCALES_AT + (uint32_t)(MH * 64 + wn * 32 + lane % 16) * kScalePiece + lane / 16;
    RowsFragment av[MH];
    BFragment bv[2][2];
    int a_scale[MH], b_scale[2][2];
    int read_step = 0;

    // Rows 0 of A are its first 32 MH: whole loads if MH is even; else the load that
    // has both kinds of rows is quarter 3's, as rows 1 are.
    constexpr int A1 = MH / 2, A3 = MH - A1;
    constexpr int B1 = BT ? 0 : 2, B2 = BT ? 4 : 2;
    // What quarter 0 does not need of a step: columns 1 and rows 1, or rows 1 alone, or
    // rows 1 but for their first load.
    constexpr int LEFT0 = MH % 2 == 1 ? A3 - 1 : BT ? A3 : B2 + A3;
    const auto read_a = [&](auto half, int buf) {
        constexpr int h = decltype(half)::value;
        const uint8_t* p = lds + buf * A_BYTES;
#pragma unroll
        for (int i = 0; i < MH; ++i) av[i].read(p, a_at + (h * 2 * MH + i) * 2048);
        if constexpr (MX) {
            const uint8_t* sp = lds + read_step / kScaleSteps % 2 * SCALE_BUF + read_step % kScaleSteps * 4;
#pragma unroll
            for (int i = 0; i < MH; ++i) a_scale[i] = sp[a_scale_at + (h * 2 * MH + i) * 16 * kScalePiece];
            read_step += h;
        }
    };
    const auto read_b = [&](auto half, int buf) {
        constexpr int h = decltype(half)::value;
        const uint8_t* p = lds + buf * kBBytes;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if constexpr (BT)
                bv[h][j].read(p, b_at ^ (h * 8 + wn * 2 + j) * 32);
            else
                bv[h][j].read(p, b_at + (h * 8 + j) * 2048);
        }
        if constexpr (MX) {
            const uint8_t* sp = lds + read_step / kScaleSteps % 2 * SCALE_BUF + read_step % kScaleSteps * 4;
#pragma unroll
            for (int j = 0; j < 2; ++j) b_scale[h][j] = sp[b_scale_at + (h * 8 + j) * 16 * kScalePiece];
        }
    };
    const auto multiply = [&](auto half_a, auto half_b) {
        constexpr int ha = decltype(half_a)::value, hb = decltype(half_b)::value;
        if constexpr (MX) {
#pragma unroll
            for (int i = 0; i < MH; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[ha][i][hb * 2 + j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        bv[hb][j].whole(), av[i].whole(), acc[ha][i][hb * 2 + j], 0, 0, 0, b_scale[hb][j], 0,
                        a_scale[i]);
        } else {
#pragma unroll
            for (int i = 0; i < MH; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[ha][i][hb * 2 + j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        bv[hb][j].template half<0>(), av[i].template half<0>(), acc[ha][i][hb * 2 + j], 0, 0, 0);
#pragma unroll
            for (int i = 0; i < MH; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[ha][i][hb * 2 + j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        bv[hb][j].template half<1>(), av[i].template half<1>(), acc[ha][i][hb * 2 + j], 0, 0, 0);
        }
    };
    const auto load = [&](auto quarter, int step, int buf) {
        constexpr int q = decltype(quarter)::value;
        uint8_t* pa = lds + buf * A_BYTES;
        uint8_t* pb = lds + B_AT + buf * kBBytes;
        if constexpr (q == 1) {
            if constexpr (MX) {
                if (step % kScaleSteps == 0) load_scales(step);
            }
            a.template load<0, A1>(a_buf, step, pa);
            if constexpr (!BT) br.template load<0, 2>(b_buf[0], step, pb);
        } else if constexpr (q == 2) {
            if constexpr (BT)
                bc.load(step, pb);
            else
                br.template load<0, 2>(b_buf[1], step, pb + kBBytes / 2);
        } else {
            a.template load<A1, MH>(a_buf, step, pa + A1 * 64 * kStepBytes);
        }
    };
    if constexpr (SHORT) {
        constexpr std::integral_constant<int, 0> h0{};
        constexpr std::integral_constant<int, 1> h1{};
        run_short_steps<STAGES, MH + 4>(
            steps,
            [&](int buf) {
                read_b(h0, buf);
                read_b(h1, buf);
                read_a(h0, buf);
                multiply(h0, h0);
                multiply(h0, h1);
                read_a(h1, buf);
                multiply(h1, h0);
                multiply(h1, h1);
            },
            [&](int step, int buf) {
                load(h1, step, buf);
                load(std::integral_constant<int, 2>{}, step, buf);
                load(std::integral_constant<int, 3>{}, step, buf);
            });
    } else {
        run_steps<A1 + B1, B2, A3, LEFT0, A3>(steps, read_a, read_b, multiply, load);
    }

    // epilogue: eight columns of one row a lane, of two tiles of 16, once behind SwiGLU
    // and twice without.  Bias and residual are all asked for before the first use: one
    // after the other, behind the stores, they took a third of the time (8192 x 7168 x
    // 2048 with a residual: 276 us, now 261).  Rows are loaded and stored line by line
    // (to_lines()).
    constexpr int OUT = SWIGLU ? 1 : 2;
    const int bias_col = col0 + wn * 32 + pair_column(), col = col0 + wn * 32 + line_column();
    u32x4 bias[2], residual[2][MH][OUT];  // bias behind SwiGLU: of gate and up
    if (g.bias != nullptr) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int c = SWIGLU ? bias_col : bias_col + j * 128;
            if (c < out_cols) bias[j] = load8(g.bias + (int64_t)t.e * g.N + c + (SWIGLU ? j * out_cols : 0));
        }
    }
    const auto row_of = [&](int h, int i) { return ((h * 2 + wm) * MH + i) * 16 + line_row(); };
    if (g.residual != nullptr) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < MH; ++i)
#pragma unroll
                for (int j = 0; j < OUT; ++j) {
                    const int m = row_of(h, i), c = col + j * 128;
                    if (m < t.rows && c < out_cols)
                        residual[h][i][j] = load8(g.residual + (int64_t)(t.first + m) * out_cols + c);
                }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < MH; ++i) {
            const int m = row_of(h, i);
            const int64_t row = t.first + m;
            float v[2][8];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                pair_values(acc[h][i][2 * j], acc[h][i][2 * j + 1], v[j]);
                if (g.bias != nullptr) add8(v[j], bias[j]);
            }
            if constexpr (SWIGLU) {
                if (g.pre != nullptr) {
                    const u32x4 gate = to_lines(pack8(v[0])), up = to_lines(pack8(v[1]));
                    if (m < t.rows && col < out_cols) {
                        store(g.pre + row * g.N + col, gate);
                        store(g.pre + row * g.N + out_cols + col, up);
                    }
                }
#pragma unroll
                for (int q = 0; q < 8; ++q) v[0][q] = silu_mul(v[0][q], v[1][q]);
            }
#pragma unroll
            for (int j = 0; j < OUT; ++j) {
                const int c = col + j * 128;
                if (g.residual != nullptr) add8(v[j], from_lines(residual[h][i][j]));
                const u32x4 o = to_lines(pack8(v[j]));
                if (m < t.rows && c < out_cols) store(g.out + row * out_cols + c, o);
            }
        }
}

template <bool BT, bool MX, bool SWIGLU>
__global__ __launch_bounds__(kGroupedThreads, 2) void grouped_kernel(GroupedArgs g, int col_tiles, int whole) {
    __shared__ __align__(16) uint8_t lds[kLdsBytes];
    const Tile t = find_tile(g.rows, col_tiles, whole);
    if (t.rows == 0) return;
    if (t.rows > 192)
        product<4, BT, MX, SWIGLU>(g, t, lds);
    else if (t.rows > 128)
        product<3, BT, MX, SWIGLU>(g, t, lds);
    else if (t.rows > 64)
        product<2, BT, MX, SWIGLU>(g, t, lds);
    else
        product<1, BT, MX, SWIGLU>(g, t, lds);
}

// From so many tiles of 64 rows by 256 columns on those keep enough CUs at work.  Dense, 512 x
// 1024 x 7168 (32 tiles): 63 us with them, 23 in grouped_few.hip; 64 tiles (8 experts, 1024 x 1024 x
// 2048): 23.4 and 22.0, MXFP8 17.9 and 20.9; 88 (512 x 2816 x 2048): 24.0 and 25.8.
constexpr int kFewTiles = 64;

template <bool BT, bool MX, bool SWIGLU>
hipError_t launch(const GroupedArgs& g, hipStream_t stream) {
    const int cols = SWIGLU ? kCols / 2 : kCols, out_cols = SWIGLU ? g.N / 2 : g.N;
    const int col_tiles = (out_cols + cols - 1) / cols;
    // Rows spread evenly over the experts, as far as the host can know.
    const int experts = g.rows.E < g.rows.R ? g.rows.E : g.rows.R;
    const auto tiles = [&](int whole) {
        return (int64_t)experts * ((g.rows.R / experts + whole - 1) / whole) * col_tiles;
    };
    if (tiles(64) < kFewTiles) return launch_grouped_few(g, BT, SWIGLU, tiles(64), stream);
    // Fewer rows a tile where whole ones would leave CUs without work (1023 x 2816 x 4096, tiles of
    // 64 rows: 41 us, 80 of 256; 4096 x 2048 x 2048, of 128: 41 and 48).
    int whole = kRows;
    while (whole > 64 && tiles(whole) < kCus) whole /= 2;
    grouped_kernel<BT, MX, SWIGLU><<<grouped_grid(grouped_tiles(g.rows, whole, col_tiles)), kGroupedThreads, 0, stream>>>(
        g, col_tiles, whole);
    return hipGetLastError();
}

}  // namespace

int64_t grouped_linear_tiles(const GroupedRows& rows, int cols) {
    return grouped_tiles(rows, 64, (cols + kCols - 1) / kCols);
}

hipError_t launch_grouped_linear(const GroupedArgs& g, bool swiglu, hipStream_t stream) {
    if (g.xs != nullptr) return swiglu ? launch<false, true, true>(g, stream) : launch<false, true, false>(g, stream);
    return swiglu ? launch<false, false, true>(g, stream) : launch<false, false, false>(g, stream);
}

hipError_t launch_grouped_grad_x(const GroupedArgs& g, hipStream_t stream) {
    return launch<true, false, false>(g, stream);
}

}  // namespace moe
