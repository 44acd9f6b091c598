// moe_grouped_linear_grad_w on gfx950: dw_e = dy_e^T x_e and db_e = the column
// sums of dy_e, the sum running over an expert's rows.
//
// Both operands lie with the sum across their rows (grouped.h, "columns"); rows past
// the segment's end read as zeros.  An expert has a few hundred rows, so a tile is a
// handful of steps and its stores: bound by the bytes of dw, and by what a workgroup
// does before its first and behind its last product.  So a workgroup of four waves
// takes tile after tile of 128 by 256: its loads, two steps ahead, run on into the next
// tile while a tile's stores drain; and a CU has two such workgroups, so that one's
// stores and waits fall into the other's products.  (One of eight waves by turns, as in
// grouped.h, on 256 by 256: 423 us for 128 experts' 1536 x 2048 of 256 rows, for the loads
// behind a tile's stores cannot be waited for without them; here GRAD_US.)  db is summed from
// the fragments of dy, in the first column tiles.  Every expert's gradient is written,
// zeros for one without rows; a tile is one workgroup's, so the sums run in one order.
#include "grouped.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kTileN = 128, kTileK = 256;  // of dw's rows and columns
constexpr int MT = 4, NT = 8;              // 16s of a wave, of four, two by two
constexpr int kStep = 32;                  // rows of a step
using AOperand = ColumnsOperand<kTileN * 2, kStep, 4>;
using BOperand = ColumnsOperand<kTileK * 2, kStep, 4>;
using AFragment = ColumnsFragment<kTileN * 2, kStep>;
using BFragment = ColumnsFragment<kTileK * 2, kStep>;
constexpr int kStage = AOperand::LDS_BYTES + BOperand::LDS_BYTES;
constexpr int kStages = 3;
constexpr int kLoads = AOperand::LOADS + BOperand::LOADS;
static_assert(2 * kStages * kStage <= kLdsBytes, "two workgroups a CU");

// The tiles of a workgroup: the `i`-th is number blockIdx + i * workgroups, expert by
// expert, row tile by row tile, so that each XCD has a share of every expert whatever
// their rows.
struct GradTiles {
    int k_tiles, per_expert;
    uint32_t tiles, run;  // run: tiles of an XCD, 0: dealt out one by one
    struct Place {
        int e, n0, k0;
    };
    __device__ __forceinline__ uint32_t first() const {
        return run == 0 ? blockIdx.x : blockIdx.x % 8 * run + blockIdx.x / 8;
    }
    __device__ __forceinline__ uint32_t step() const { return run == 0 ? gridDim.x : gridDim.x / 8; }
    __device__ __forceinline__ uint32_t end() const { return run == 0 ? tiles : min((blockIdx.x % 8 + 1) * run, tiles); }
    __device__ __forceinline__ Place place(uint32_t u) const {
        const int at = (int)(u % (uint32_t)per_expert);
        return {(int)(u / (uint32_t)per_expert), at / k_tiles * kTileN, at % k_tiles * kTileK};
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
__device__ __forceinline__ int steps_of(const Segment& s) { return max((s.n + kStep - 1) / kStep, 1); }

template <bool WIDE, bool DB>
__global__ __launch_bounds__(kThreads, 2) void grad_w_kernel(GroupedGradArgs g, GradTiles tiles) {
    __shared__ __align__(16) uint8_t lds[kStages * kStage];
    const int lane = (int)(threadIdx.x % kWave), wave = (int)uniform(threadIdx.x / kWave);
    const int wm = wave / 2, wn = wave % 2;
    const uint32_t lda = (uint32_t)g.N * 2, ldb = (uint32_t)g.K * 2;

    // The stream of loads: its tile, that tile's rows, and those of the next.
    const uint32_t first = tiles.first(), stride = tiles.step(), end = tiles.end();
    if (first >= end) return;
    uint32_t load_tile = first;
    Segment load_rows = as_segment(g.rows, raw_segment(g.rows, tiles.place(load_tile).e));
    int load_step = 0, load_steps = steps_of(load_rows);
    RawSegment ahead = raw_segment(g.rows, tiles.place(min(load_tile + stride, end - 1)).e);
    AOperand a;
    BOperand b;
    const auto set = [&] {
        const GradTiles::Place at = tiles.place(load_tile);
        const int64_t n = load_tile < end ? load_rows.n : 0;
        a.set(reinterpret_cast<const uint8_t*>(g.dy) + (int64_t)load_rows.first * lda + at.n0 * 2,
              n * lda - at.n0 * 2, lda);
        b.set(reinterpret_cast<const uint8_t*>(g.x) + (int64_t)load_rows.first * ldb + at.k0 * 2,
              n * ldb - at.k0 * 2, ldb);
    };
    set();
    BufferWords a_buf, b_buf;  // of the step that is loaded
    const auto advance = [&] {
        if (load_step == load_steps) {  // on to the next tile; behind the last one zeros
            load_tile += stride;
            load_rows = as_segment(g.rows, ahead);
            load_step = 0;
            load_steps = steps_of(load_rows);
            ahead = raw_segment(g.rows, tiles.place(min(load_tile + stride, end - 1)).e);
            set();
        }
        a_buf = a.buffer(load_step);
        b_buf = b.buffer(load_step++);
    };
    const auto load_one = [&](auto index, int buf) {
        constexpr int j = decltype(index)::value;
        if constexpr (j < AOperand::LOADS)
            a.load_one<j>(a_buf, lds + buf * kStage);
        else
            b.load_one<j - AOperand::LOADS>(b_buf, lds + buf * kStage + AOperand::LDS_BYTES);
    };

    f32x4 acc[MT][NT];
    float sums[MT];
    // Stores of a tile: always STORES a lane, those of rows and columns past dw's end
    // through an offset past its buffer's, so that the waits can count them.
    constexpr int STORES = MT * NT / 2 * (WIDE ? 2 : 1);
    const auto store = [&](const GradTiles::Place& p) {
        constexpr int EL = WIDE ? 4 : 2;
        const int rows = min(g.N - p.n0, kTileN);
        const __amdgpu_buffer_rsrc_t out =
            grouped_buffer(static_cast<uint8_t*>(g.dw) + ((int64_t)p.e * g.N + p.n0) * g.K * EL, (int64_t)rows * g.K * EL);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int n = (wm * MT + i) * 16 + lane % 16;
#pragma unroll
            for (int j = 0; j < NT; j += 2) {
                const int k = p.k0 + (wn * NT + j) * 16 + pair_column();
                const uint32_t to = n < rows && k < g.K ? ((uint32_t)n * (uint32_t)g.K + (uint32_t)k) * EL : kPastEnd;
                float v[8];
                pair_values(acc[i][j], acc[i][j + 1], v);
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
                    const float s = __builtin_bit_cast(float, across_rows(__builtin_bit_cast(uint32_t, sums[i])));
                    if (lane < 16 && n < rows) g.db[(int64_t)p.e * g.N + p.n0 + n] = s;
                }
            }
        }
    };

    const uint32_t a_at = AFragment::at(), b_at = AOperand::LDS_BYTES + BFragment::at();
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        advance();
        unrolled<kLoads>([&](auto j) { load_one(j, s); });
    }
    int buf = 0;
    uint32_t tile = first;
    RawSegment next = raw_segment(g.rows, tiles.place(tile).e);
    for (; tile < end; tile += stride) {
        const GradTiles::Place p = tiles.place(tile);
        const int steps = steps_of(as_segment(g.rows, next));
        next = raw_segment(g.rows, tiles.place(min(tile + stride, end - 1)).e);
        const bool sum_here = DB && p.k0 == 0 && wn == 0;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            sums[i] = 0.0f;
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        for (int step = 0; step < steps; ++step) {
            // This step's loads have landed: newer ones are the next step's, and in a tile's
            // first two the stores of the tile before.
            if (step < 2 && tile != first)
                loads_done<kLoads + STORES>();
            else
                loads_done<kLoads>();
            reads_done();
            meet();
            advance();
            const uint8_t* q = lds + buf * kStage;
            AFragment av[MT];
            BFragment bv[NT];
#pragma unroll
            for (int i = 0; i < MT; ++i) av[i].read(q, a_at ^ (wm * MT + i) * 32);
#pragma unroll
            for (int j = 0; j < NT; ++j) bv[j].read(q, b_at ^ (wn * NT + j) * 32);
            // Loads one by one among the products: all at once they hold the wave up until
            // the CU has taken them.
            unrolled<NT>([&](auto index) {
                constexpr int j = decltype(index)::value;
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bv[j].template half<0>(),
                                                                        av[i].template half<0>(), acc[i][j], 0, 0, 0);
                if constexpr (j < kLoads) load_one(index, buf == 0 ? 2 : buf - 1);
                __builtin_amdgcn_sched_barrier(0);
            });
            if (sum_here) {
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    float f[8];
                    unpack8(__builtin_bit_cast(u32x4, av[i].template half<0>()), f);
                    sums[i] += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
                }
            }
            buf = buf == 2 ? 0 : buf + 1;
        }
        store(p);
    }
    loads_done<0>();  // none may land in the next workgroup's LDS
}

constexpr int kCus = 256;

}  // namespace

int64_t grouped_grad_w_tiles(int E, int N, int K) {
    return (int64_t)E * ((N + kTileN - 1) / kTileN) * ((K + kTileK - 1) / kTileK);
}

hipError_t launch_grouped_grad_w(const GroupedGradArgs& g, hipStream_t stream) {
    const int n_tiles = (g.N + kTileN - 1) / kTileN, k_tiles = (g.K + kTileK - 1) / kTileK;
    const uint32_t tiles = (uint32_t)grouped_grad_w_tiles(g.rows.E, g.N, g.K);
    const GradTiles t = {k_tiles, n_tiles * k_tiles, tiles, 0};
    const uint32_t grid = tiles < 2 * kCus ? (tiles + 7) / 8 * 8 : 2 * kCus;
    if (g.wide && g.db)
        grad_w_kernel<true, true><<<grid, kThreads, 0, stream>>>(g, t);
    else if (g.wide)
        grad_w_kernel<true, false><<<grid, kThreads, 0, stream>>>(g, t);
    else if (g.db)
        grad_w_kernel<false, true><<<grid, kThreads, 0, stream>>>(g, t);
    else
        grad_w_kernel<false, false><<<grid, kThreads, 0, stream>>>(g, t);
    return hipGetLastError();
}

}  // namespace moe
