// The products of grouped_linear.hip where they have few tiles: few rows in all, or few
// columns, so that tiles of 64 rows by 256 columns would leave most CUs without work.
//
// A workgroup takes up to 64 rows by 16 or 32 columns, and its eight waves every eighth
// step of 128 bytes of the summed index each; their sums meet in LDS and are added in the
// order of the waves.  Bound by the bytes that a CU gets from its L2, (rows + columns) x steps, so
// columns are few until every CU has a tile; then by the latency of the few steps of a wave.
// Loads of two or three steps are in flight in registers, without barriers; a step goes
// through a piece of LDS of the wave's own, for neighbouring lanes have to read neighbouring
// bytes: with the lanes where the matrix instruction wants them, each beside lanes of 15 other
// rows, 32 rows by 2048 columns of 7168 took 28 us, 14.3 so (61 in tiles of 64 by 256).
// For dx the weights' rows are the steps, and ds_read_b64_tr_b16 turns them.
#include "grouped.h"

namespace moe {
namespace {

constexpr int kFewRows = 64;
constexpr int kFewWaves = kGroupedThreads / kWave;

template <int NC>
constexpr int kSumRow = NC * 16 + 4;  // floats of a row of sums in LDS: rows start at different banks
template <int NC>
constexpr int kTurnRow = NC * 32 + 16;  // bytes of a row of weights that is to be turned
// bytes of LDS: the waves' steps, 64 rows of one operand and NC times 16 rows or 64 rows to be
// turned of the other, and in their place their sums
template <int NC>
constexpr int kFewStep = kFewRows * kStepBytes + 64 * kTurnRow<NC>;
template <int NC>
constexpr int kFewLds = kFewWaves * (kFewStep<NC> > kFewRows * kSumRow<NC> * 4 ? kFewStep<NC> : kFewRows * kSumRow<NC> * 4);

// A step of NR times 16 rows on its way to LDS: 16 bytes of each of 2 NR rows a lane, and
// the scale bytes of its rows of the operand.  Loads past a row's end read its beginning (a branch
// round them would make every wait one for all loads), and clear() makes zeros of it.
template <int NR, bool MX>
struct FewRowsOperand {
    struct Step {
        i32x4 v[2 * NR];
        int scale[NR];
    };
    const uint8_t* at[2 * NR];
    const uint8_t* scale_at[NR];
    // row(i): the tile's row i, 0 .. 16 NR - 1, in the operand
    template <class Row>
    __device__ __forceinline__ void set(const uint8_t* base, const uint8_t* scales, int64_t ld, const Row& row) {
        const int lane = threadIdx.x % kWave;
#pragma unroll
        for (int i = 0; i < 2 * NR; ++i) at[i] = base + row(i * 8 + lane / 8) * ld;
        if constexpr (MX) {
#pragma unroll
            for (int i = 0; i < NR; ++i) scale_at[i] = scales + row(i * 16 + lane % 16) * (ld / 32);
        }
    }
    static __device__ __forceinline__ uint32_t piece(int step) {
        return (uint32_t)step * kStepBytes + threadIdx.x % 8 * 16;
    }
    static __device__ __forceinline__ uint32_t block(int step) {
        return (uint32_t)step * (kStepBytes / 32) + threadIdx.x % kWave / 16;
    }
    __device__ __forceinline__ void load(Step& s, int step, uint32_t ld) const {
        const uint32_t k = piece(step) < ld ? piece(step) : 0;
#pragma unroll
        for (int i = 0; i < 2 * NR; ++i) s.v[i] = *reinterpret_cast<const i32x4*>(at[i] + k);
        if constexpr (MX) {
            const uint32_t b = block(step) < ld / 32 ? block(step) : 0;
#pragma unroll
            for (int i = 0; i < NR; ++i) s.scale[i] = scale_at[i][b];
        }
    }
    static __device__ __forceinline__ void clear(Step& s, int step, uint32_t ld) {
        const i32x4 none = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 2 * NR; ++i) s.v[i] = piece(step) < ld ? s.v[i] : none;
        if constexpr (MX) {
#pragma unroll
            for (int i = 0; i < NR; ++i) s.scale[i] = block(step) < ld / 32 ? s.scale[i] : 0;
        }
    }
    static __device__ __forceinline__ void write(const Step& s, uint8_t* lds) {
        const uint32_t lane = threadIdx.x % kWave;
#pragma unroll
        for (int i = 0; i < 2 * NR; ++i) {
            const uint32_t row = i * 8 + lane / 8;
            *reinterpret_cast<i32x4*>(lds + row * kStepBytes + (lane % 8 ^ (row / 2 % 8)) * 16) = s.v[i];
        }
    }
    static __device__ __forceinline__ void read(const uint8_t* lds, RowsFragment (&f)[NR]) {
#pragma unroll
        for (int i = 0; i < NR; ++i) f[i].read(lds + i * 16 * kStepBytes, RowsFragment::at());
    }
};

// The same of 64 rows of weights by NC times 16 columns, turned on their way
// back from LDS.  Columns past the end are others.
template <int NC>
struct FewColumnsOperand {
    struct Step {
        i32x4 v[2 * NC];
    };
    const uint8_t* base;
    int row[2 * NC];  // of a step
    uint32_t column;  // byte of a row; a lane's pieces are of one column
    __device__ __forceinline__ void set(const uint8_t* base_, int cols) {
        const int lane = threadIdx.x % kWave, piece = lane % (2 * NC);
        base = base_;
        column = piece * 8 < cols ? piece * 16 : 0;
#pragma unroll
        for (int i = 0; i < 2 * NC; ++i) row[i] = (i * kWave + lane) / (2 * NC);
    }
    __device__ __forceinline__ void load(Step& s, int step, int rows, int64_t ld) const {
#pragma unroll
        for (int i = 0; i < 2 * NC; ++i)
            s.v[i] = *reinterpret_cast<const i32x4*>(base + min(step * 64 + row[i], rows - 1) * ld + column);
    }
    __device__ __forceinline__ void clear(Step& s, int step, int rows) const {
        const i32x4 none = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 2 * NC; ++i) s.v[i] = step * 64 + row[i] < rows ? s.v[i] : none;
    }
    __device__ __forceinline__ void write(const Step& s, uint8_t* lds) const {
#pragma unroll
        for (int i = 0; i < 2 * NC; ++i)
            *reinterpret_cast<i32x4*>(lds + row[i] * kTurnRow<NC> + threadIdx.x % (2 * NC) * 16) = s.v[i];
    }
    static __device__ __forceinline__ void read(const uint8_t* lds, RowsFragment (&f)[NC]) {
        const int lane = threadIdx.x % kWave;
        const uint8_t* p = lds + (lane / 16 * 8 + lane % 16 / 4) * kTurnRow<NC> + lane % 4 * 8;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            s16x4 t[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                t[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (MOE_LDS s16x4*)(p + (i / 2 * 32 + i % 2 * 4) * kTurnRow<NC> + j * 32));
            f[j].lo = __builtin_bit_cast(i32x4, __builtin_shufflevector(t[0], t[1], 0, 1, 2, 3, 4, 5, 6, 7));
            f[j].hi = __builtin_bit_cast(i32x4, __builtin_shufflevector(t[2], t[3], 0, 1, 2, 3, 4, 5, 6, 7));
        }
    }
};

template <int MR, int NC, bool BT, bool MX, bool SWIGLU>
__device__ __forceinline__ void few_product(const GroupedArgs& g, const Tile& t, uint8_t* lds) {
    constexpr int C = NC * 16, OUT_COLS = SWIGLU ? C / 2 : C;
    constexpr int STAGES = MR + NC <= 4 ? 3 : 2;  // (of 8 (MR + NC) registers each)
    const int lane = (int)(threadIdx.x % kWave), wave = (int)uniform(threadIdx.x / kWave);
    const int out_cols = SWIGLU ? g.N / 2 : g.N;
    const int col0 = t.col * OUT_COLS;
    const int64_t lda = (int64_t)g.K * (MX ? 1 : 2);
    const int steps = (int)((lda + kStepBytes - 1) / kStepBytes);

    // Rows and columns past the tile's are others of it: what they give is not stored.
    using A = FewRowsOperand<MR, MX>;
    using B = std::conditional_t<BT, FewColumnsOperand<NC>, FewRowsOperand<NC, MX>>;
    A a;
    B b;
    a.set(static_cast<const uint8_t*>(g.x), g.xs, lda, [&](int i) { return (int64_t)t.first + min(i, t.rows - 1); });
    if constexpr (BT) {
        b.set(static_cast<const uint8_t*>(g.w) + ((int64_t)t.e * g.K * g.N + col0) * 2, g.N - col0);
    } else {
        b.set(static_cast<const uint8_t*>(g.w), g.ws, lda, [&](int c) {
            const int col = min(col0 + (SWIGLU ? c % OUT_COLS : c), out_cols - 1);
            return (int64_t)t.e * g.N + col + (c < OUT_COLS ? 0 : out_cols);
        });
    }

    f32x4 acc[MR][NC];
#pragma unroll
    for (int i = 0; i < MR; ++i)
#pragma unroll
        for (int j = 0; j < NC; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    struct Step {
        typename A::Step a;
        typename B::Step b;
    };
    uint8_t* own = lds + wave * kFewStep<NC>;
    uint8_t* own_b = own + MR * 16 * kStepBytes;
    const auto load = [&](Step& s, int step) {
        step = min(step, steps - 1);
        a.load(s.a, step, (uint32_t)lda);
        if constexpr (BT)
            b.load(s.b, step, g.K, (int64_t)g.N * 2);
        else
            b.load(s.b, step, (uint32_t)lda);
    };
    const auto multiply = [&](Step& s, int step) {
        if ((step + 1) * kStepBytes > lda) {  // the last, with a row's end in it
            a.clear(s.a, step, (uint32_t)lda);
            if constexpr (BT)
                b.clear(s.b, step, g.K);
            else
                b.clear(s.b, step, (uint32_t)lda);
        }
        a.write(s.a, own);
        b.write(s.b, own_b);
        reads_done();  // lanes read what others wrote
        RowsFragment av[MR], bv[NC];
        a.read(own, av);
        b.read(own_b, bv);
        reads_done();  // before the next step's writes
#pragma unroll
        for (int i = 0; i < MR; ++i)
#pragma unroll
            for (int j = 0; j < NC; ++j) {
                if constexpr (MX) {
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        bv[j].whole(), av[i].whole(), acc[i][j], 0, 0, 0, s.b.scale[j], 0, s.a.scale[i]);
                } else {
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bv[j].template half<0>(),
                                                                       av[i].template half<0>(), acc[i][j], 0, 0, 0);
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bv[j].template half<1>(),
                                                                       av[i].template half<1>(), acc[i][j], 0, 0, 0);
                }
            }
    };
    Step s[STAGES];
    unrolled<STAGES - 1>([&](auto n) { load(s[n], wave + n * kFewWaves); });
    for (int step = wave; step < steps; step += STAGES * kFewWaves) {
        unrolled<STAGES>([&](auto n) {
            const int here = step + n * kFewWaves;
            load(s[(n + STAGES - 1) % STAGES], here + (STAGES - 1) * kFewWaves);
            if (here < steps) multiply(s[n], here);
        });
    }

    __syncthreads();  // the waves' sums take the place of their steps
    float* sums = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int i = 0; i < MR; ++i)
#pragma unroll
        for (int j = 0; j < NC; ++j)
            *reinterpret_cast<f32x4*>(sums + ((wave * MR + i) * 16 + lane % 16) * kSumRow<NC> + j * 16 + lane / 16 * 4) =
                acc[i][j];
    __syncthreads();
    // eight columns of a row a thread
    const int m = (int)threadIdx.x / (OUT_COLS / 8), c = (int)threadIdx.x % (OUT_COLS / 8) * 8;
    const int col = col0 + c;
    if (m >= t.rows || col >= out_cols) return;
    const auto sum8 = [&](int c, float(&v)[8]) {
        const float* p = sums + m * kSumRow<NC> + c;
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = 0.0f;
#pragma unroll
        for (int w = 0; w < kFewWaves; ++w)
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] += p[w * MR * 16 * kSumRow<NC> + q];
    };
    const int64_t row = t.first + m;
    float v[8];
    sum8(c, v);
    if (g.bias != nullptr) add8(v, load8(g.bias + (int64_t)t.e * g.N + col));
    if constexpr (SWIGLU) {
        float u[8];
        sum8(c + OUT_COLS, u);
        if (g.bias != nullptr) add8(u, load8(g.bias + (int64_t)t.e * g.N + out_cols + col));
        if (g.pre != nullptr) {
            store(g.pre + row * g.N + col, pack8(v));
            store(g.pre + row * g.N + out_cols + col, pack8(u));
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = silu_mul(v[q], u[q]);
    }
    if (g.residual != nullptr) add8(v, load8(g.residual + row * out_cols + col));
    store(g.out + row * out_cols + col, pack8(v));
}

template <int NC, bool BT, bool MX, bool SWIGLU>
__global__ __launch_bounds__(kGroupedThreads, 2) void few_kernel(GroupedArgs g, int col_tiles) {
    __shared__ __align__(16) uint8_t lds[kFewLds<NC>];
    static_assert(kFewLds<NC> <= kLdsBytes && NC * 16 * kStepBytes <= 64 * kTurnRow<NC>, "a step fits its LDS");
    static_assert(kFewRows * NC * 16 / 8 <= kGroupedThreads, "a thread for each eight columns of the tile");
    const Tile t = find_tile(g.rows, col_tiles, kFewRows);
    if (t.rows == 0) return;
    if (t.rows > 32)
        few_product<4, NC, BT, MX, SWIGLU>(g, t, lds);
    else if (t.rows > 16)
        few_product<2, NC, BT, MX, SWIGLU>(g, t, lds);
    else
        few_product<1, NC, BT, MX, SWIGLU>(g, t, lds);
}

template <int NC, bool BT, bool MX, bool SWIGLU>
hipError_t few_launch(const GroupedArgs& g, hipStream_t stream) {
    const int cols = SWIGLU ? NC * 8 : NC * 16, out_cols = SWIGLU ? g.N / 2 : g.N;
    const int col_tiles = (out_cols + cols - 1) / cols;
    few_kernel<NC, BT, MX, SWIGLU><<<grouped_grid(grouped_tiles(g.rows, kFewRows, col_tiles)), kGroupedThreads, 0, stream>>>(
        g, col_tiles);
    return hipGetLastError();
}

template <bool BT, bool MX, bool SWIGLU>
hipError_t few(const GroupedArgs& g, int64_t tiles, hipStream_t stream) {
    // 32 columns if that is a tile for every CU (512 x 1024 x 7168: 22.0 us, 34.2 in tiles of 16;
    // 32 x 2048 x 7168 in tiles of 16, one for every other CU: 14.3)
    if (tiles * 8 >= kCus) return few_launch<2, BT, MX, SWIGLU>(g, stream);
    return few_launch<1, BT, MX, SWIGLU>(g, stream);
}

}  // namespace

hipError_t launch_grouped_few(const GroupedArgs& g, bool transposed, bool swiglu, int64_t tiles, hipStream_t stream) {
    if (transposed) return few<true, false, false>(g, tiles, stream);
    if (g.xs != nullptr)
        return swiglu ? few<false, true, true>(g, tiles, stream) : few<false, true, false>(g, tiles, stream);
    return swiglu ? few<false, false, true>(g, tiles, stream) : few<false, false, false>(g, tiles, stream);
}

}  // namespace moe
