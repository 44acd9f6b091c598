// moe_grouped_linear_grad_w on gfx950: dw_e = dy_e^T x_e and db_e = the column
// sums of dy_e, the sum running over an expert's rows.
//
// Both operands lie with the sum across their rows (grouped.h, "columns"); rows past
// the segment's end read as zeros.  An expert has a few hundred rows, so a tile of 256
// by 256 is a handful of steps and its stores: bound by the bytes of dw, and by what a
// workgroup does before its first and behind its last product.  So one workgroup a CU
// stays and takes tile after tile: the loads, two steps ahead, run on into the next
// tile, and a tile's stores drain while the next is multiplied.  db is summed from the
// fragments of dy, by the waves of the first column tiles that hold columns 0.  Every
// expert's gradient is written, zeros for one without rows; a tile is one workgroup's,
// so the sums run in one order.
#include "grouped.h"

namespace moe {
namespace {

constexpr int kTile = 256;  // of dw's rows (N) and columns (K)
constexpr int MH = kTile / 64;
constexpr int kOperand = 64 * kTile * 2;  // bytes of LDS of one operand's step
constexpr int kLoads = 4;                 // of a wave, of either operand
using Operand = ColumnsOperand<kLoads>;
using Fragment = ColumnsFragment<Operand::W>;
static_assert(Operand::LDS_BYTES == kOperand && Operand::W == kTile * 2, "a tile's columns");

// The tiles of a workgroup: the `i`-th is number blockIdx + i * workgroups, expert by
// expert, row tile by row tile, so that each XCD has a share of every expert whatever
// their rows.
struct GradTiles {
    int k_tiles, per_expert;
    uint32_t tiles;
    struct Place {
        int e, n0, k0;
    };
    __device__ __forceinline__ Place place(uint32_t u) const {
        const int at = (int)(u % (uint32_t)per_expert);
        return {(int)(u / (uint32_t)per_expert), at / k_tiles * kTile, at % k_tiles * kTile};
    }
};

// Rows of expert e as the arrays hold them; asked for a tile ahead, made a segment
// when it has arrived.
struct RawSegment {
    int first, end_or_n;
};
__device__ __forceinline__ RawSegment raw_segment(const GroupedRows& g, int e) {
    if (g.offsets == nullptr) return {0, g.R};
    return {g.offsets[e], g.counts != nullptr ? g.counts[e] : g.offsets[e + 1]};
}
__device__ __forceinline__ Segment as_segment(const GroupedRows& g, const RawSegment& r) {
    const int first = min(max(r.first, 0), g.R);
    const int n = g.counts != nullptr ? r.end_or_n : min(max(r.end_or_n, 0), g.R) - first;
    return {first, min(max(n, 0), g.R - first)};
}
// (A tile of an expert without rows is a step of zeros.)
__device__ __forceinline__ int steps_of(const Segment& s) { return max((s.n + 63) / 64, 1); }

template <bool WIDE, bool DB>
__global__ __launch_bounds__(kGroupedThreads, 2) void grad_w_kernel(GroupedGradArgs g, GradTiles tiles) {
    __shared__ __align__(16) uint8_t lds[4 * kOperand];
    const int lane = (int)(threadIdx.x % kWave), wave = (int)uniform(threadIdx.x / kWave);
    const int wm = wave / 4, wn = wave % 4;
    const uint32_t lda = (uint32_t)g.N * 2, ldb = (uint32_t)g.K * 2;

    // The stream of loads.
    uint32_t load_tile = blockIdx.x;  // and its rows, and those of the next
    Segment load_rows = as_segment(g.rows, raw_segment(g.rows, tiles.place(load_tile).e));
    int load_step = 0, load_steps = steps_of(load_rows);
    RawSegment ahead = raw_segment(g.rows, tiles.place(min(load_tile + gridDim.x, tiles.tiles - 1)).e);
    Operand a, b;
    const auto set = [&] {
        const GradTiles::Place at = tiles.place(load_tile);
        const int64_t n = load_tile < tiles.tiles ? load_rows.n : 0;
        a.set(reinterpret_cast<const uint8_t*>(g.dy) + (int64_t)load_rows.first * lda + at.n0 * 2,
              n * lda - at.n0 * 2, lda);
        b.set(reinterpret_cast<const uint8_t*>(g.x) + (int64_t)load_rows.first * ldb + at.k0 * 2,
              n * ldb - at.k0 * 2, ldb);
    };
    set();
    const auto load_b = [&](int buf) {
        if (load_step == load_steps) {  // on to the next tile; behind the last one zeros
            load_tile += gridDim.x;
            load_rows = as_segment(g.rows, ahead);
            load_step = 0;
            load_steps = steps_of(load_rows);
            ahead = raw_segment(g.rows, tiles.place(min(load_tile + gridDim.x, tiles.tiles - 1)).e);
            set();
        }
        b.load(load_step, lds + (2 + buf) * kOperand);
    };
    const auto load_a = [&](int buf) { a.load(load_step++, lds + buf * kOperand); };

    const uint32_t at = Fragment::at();
    Fragment av[MH], bv[2][2];
    const auto read_a = [&](int h, int buf) {
#pragma unroll
        for (int i = 0; i < MH; ++i) av[i].read(lds + buf * kOperand, at ^ ((h * 2 + wm) * MH + i) * 32);
    };
    const auto read_b = [&](int h, int buf) {
#pragma unroll
        for (int j = 0; j < 2; ++j) bv[h][j].read(lds + (2 + buf) * kOperand, at ^ (h * 8 + wn * 2 + j) * 32);
    };
    f32x4 acc[2][MH][4];
    float sums[2][MH];
    const auto quarter = [&](auto half_a, auto half_b) {
        constexpr int ha = decltype(half_a)::value, hb = decltype(half_b)::value;
        meet();
        __builtin_amdgcn_s_setprio(1);
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
        __builtin_amdgcn_s_setprio(0);
        meet();
    };
    constexpr std::integral_constant<int, 0> h0{};
    constexpr std::integral_constant<int, 1> h1{};

    // Stores of a tile: always STORES a lane, those of rows and columns past dw's end
    // through an offset past its buffer's, so that the waits can count them.
    constexpr int STORES = 2 * MH * 2 * (WIDE ? 2 : 1);
    const auto store = [&](const GradTiles::Place& p) {
        constexpr int EL = WIDE ? 4 : 2;
        const int rows = min(g.N - p.n0, kTile);
        const __amdgpu_buffer_rsrc_t out =
            grouped_buffer(static_cast<uint8_t*>(g.dw) + ((int64_t)p.e * g.N + p.n0) * g.K * EL, (int64_t)rows * g.K * EL);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < MH; ++i) {
                const int n = ((h * 2 + wm) * MH + i) * 16 + lane % 16;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int k = p.k0 + j * 128 + wn * 32 + pair_column();
                    const uint32_t to = n < rows && k < g.K ? ((uint32_t)n * (uint32_t)g.K + (uint32_t)k) * EL : kPastEnd;
                    float v[8];
                    pair_values(acc[h][i][2 * j], acc[h][i][2 * j + 1], v);
                    if constexpr (WIDE) {
                        __builtin_amdgcn_raw_buffer_store_b128(
                            __builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]}), out, (int)to, 0, 0);
                        __builtin_amdgcn_raw_buffer_store_b128(
                            __builtin_bit_cast(u32x4, f32x4{v[4], v[5], v[6], v[7]}), out, (int)to, 16, 0);
                    } else {
                        __builtin_amdgcn_raw_buffer_store_b128(pack8(v), out, (int)to, 0, 0);
                    }
                }
                if constexpr (DB) {
                    if (p.k0 == 0 && wn == 0) {  // a lane has summed its quarter of the rows
                        const float s = __builtin_bit_cast(float, across_rows(__builtin_bit_cast(uint32_t, sums[h][i])));
                        if (lane < 16 && n < rows) g.db[(int64_t)p.e * g.N + p.n0 + n] = s;
                    }
                }
            }
    };
    const auto add_rows = [&](auto half) {
        constexpr int h = decltype(half)::value;
#pragma unroll
        for (int i = 0; i < MH; ++i) {
            float f[8];
            unpack8(__builtin_bit_cast(u32x4, av[i].template half<0>()), f);
            sums[h][i] += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
            unpack8(__builtin_bit_cast(u32x4, av[i].template half<1>()), f);
            sums[h][i] += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
        }
    };

#pragma unroll
    for (int s = 0; s < 2; ++s) {
        load_b(s);
        load_a(s);
    }
    loads_done<2 * kLoads>();
    meet();
    const bool late = wave >= 4;
    if (late) meet();
    int buf = 0;
    uint32_t tile = blockIdx.x;
    RawSegment next = raw_segment(g.rows, tiles.place(tile).e);
    for (; tile < tiles.tiles; tile += gridDim.x) {
        const GradTiles::Place p = tiles.place(tile);
        const int steps = steps_of(as_segment(g.rows, next));
        next = raw_segment(g.rows, tiles.place(min(tile + gridDim.x, tiles.tiles - 1)).e);
        const bool sum_here = DB && p.k0 == 0 && wn == 0;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < MH; ++i) {
                sums[h][i] = 0.0f;
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[h][i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            }
        for (int step = 0; step < steps; ++step) {
            read_a(0, buf);
            read_b(0, buf);
            reads_done();
            if (sum_here) add_rows(h0);
            quarter(h0, h0);
            read_b(1, buf);
            reads_done();
            quarter(h0, h1);
            read_a(1, buf);
            load_b(buf);
            reads_done();
            if (sum_here) add_rows(h1);
            quarter(h1, h1);
            load_a(buf);
            // The next step's loads have landed: newer ones are those of this step, and in
            // a tile's first the stores of the tile before.
            if (step == 0 && tile != blockIdx.x)
                loads_done<2 * kLoads + STORES>();
            else
                loads_done<2 * kLoads>();
            quarter(h1, h0);
            buf ^= 1;
        }
        store(p);
    }
    if (!late) meet();
    loads_done<0>();  // none may land in the next workgroup's LDS
}

constexpr int kCus = 256;

}  // namespace

int64_t grouped_grad_w_tiles(int E, int N, int K) {
    return (int64_t)E * ((N + kTile - 1) / kTile) * ((K + kTile - 1) / kTile);
}

hipError_t launch_grouped_grad_w(const GroupedGradArgs& g, hipStream_t stream) {
    const int n_tiles = (g.N + kTile - 1) / kTile, k_tiles = (g.K + kTile - 1) / kTile;
    const GradTiles t = {k_tiles, n_tiles * k_tiles, (uint32_t)grouped_grad_w_tiles(g.rows.E, g.N, g.K)};
    const uint32_t grid = t.tiles < kCus ? t.tiles : kCus;
    if (g.wide && g.db)
        grad_w_kernel<true, true><<<grid, kGroupedThreads, 0, stream>>>(g, t);
    else if (g.wide)
        grad_w_kernel<true, false><<<grid, kGroupedThreads, 0, stream>>>(g, t);
    else if (g.db)
        grad_w_kernel<false, true><<<grid, kGroupedThreads, 0, stream>>>(g, t);
    else
        grad_w_kernel<false, false><<<grid, kGroupedThreads, 0, stream>>>(g, t);
    return hipGetLastError();
}

}  // namespace moe
