// moe_grouped_linear_grad_w on gfx950: dw_e = dy_e^T x_e and db_e = the column
// sums of dy_e, the sum running over an expert's rows.
//
// Both operands lie with the sum across their rows (grouped.h, "columns").  Rows
// past the segment's end read as zeros.  db comes from the same tiles: a product
// with a row of ones, in the first column tile's workgroups.  Every expert's
// gradient is written, zeros for one without rows; a tile is one workgroup's, so
// the sums run in one order.
#include "grouped.h"

namespace moe {
namespace {

constexpr int MT = 4, NT = 2;
constexpr int kTileN = 32 * MT, kTileK = 64 * NT;  // of dw's rows (N) and columns (K)
constexpr int AJ = MT / 2;
constexpr int kABytes = ColumnsOperand<AJ>::LDS_BYTES;
constexpr int kStage = kABytes + ColumnsOperand<NT>::LDS_BYTES;
constexpr int kStages = 2;

template <bool WIDE, bool DB>
__global__ __launch_bounds__(kGroupedThreads, 4) void grad_w_kernel(GroupedGradArgs g, int n_tiles, int k_tiles,
                                                                    uint32_t tiles) {
    __shared__ __align__(16) uint8_t lds[kStages * kStage];
    const uint32_t run = (tiles + 7) / 8;  // each XCD a run of neighbouring tiles
    const uint32_t u = blockIdx.x % 8 * run + blockIdx.x / 8;
    if (u >= tiles) return;
    const int per_expert = n_tiles * k_tiles;
    const int e = (int)(u / (uint32_t)per_expert);
    const int at = (int)(u % (uint32_t)per_expert);
    const int n0 = at / k_tiles * kTileN, k0 = at % k_tiles * kTileK;
    const Segment seg = segment(g.rows, e);
    const int lane = (int)(threadIdx.x % kWave), wave = (int)uniform(threadIdx.x / kWave);
    const int wm = wave / 4, wn = wave % 4;
    const uint32_t lda = (uint32_t)g.N * 2, ldb = (uint32_t)g.K * 2;
    const int steps = (seg.n + 63) / 64;

    ColumnsOperand<AJ> a;
    a.set(reinterpret_cast<const uint8_t*>(g.dy) + (int64_t)seg.first * lda + n0 * 2, (int64_t)seg.n * lda - n0 * 2,
          lda);
    ColumnsOperand<NT> b;
    b.set(reinterpret_cast<const uint8_t*>(g.x) + (int64_t)seg.first * ldb + k0 * 2, (int64_t)seg.n * ldb - k0 * 2,
          ldb);
    const auto load = [&](int step, int buf) {
        a.load(step, lds + buf * kStage);
        b.load(step, lds + buf * kStage + kABytes);
    };

    f32x4 acc[MT][NT], sums[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        sums[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    const bool sum_here = DB && k0 == 0 && wn == 0;
    constexpr int AW = ColumnsOperand<AJ>::W, BW = ColumnsOperand<NT>::W;
    const uint32_t a_at = ColumnsFragment<AW>::at(), b_at = kABytes + ColumnsFragment<BW>::at();

    if (steps > 0) load(0, 0);
    for (int step = 0; step < steps; ++step) {
        loads_done<0>();
        reads_done();
        meet();
        if (step + 1 < steps) load(step + 1, (step + 1) % 2);
        const uint8_t* p = lds + step % 2 * kStage;
        ColumnsFragment<AW> av[MT];
        ColumnsFragment<BW> bv[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) bv[j].read(p, b_at ^ (wn * NT + j) * 32);
#pragma unroll
        for (int i = 0; i < MT; ++i) av[i].read(p, a_at ^ (wm * MT + i) * 32);
        const auto half = [&](auto h) {
            constexpr int H = decltype(h)::value;
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bv[j].template half<H>(),
                                                                        av[i].template half<H>(), acc[i][j], 0, 0, 0);
            if (sum_here) {
                const s16x8 ones = {0x3F80, 0x3F80, 0x3F80, 0x3F80, 0x3F80, 0x3F80, 0x3F80, 0x3F80};
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    sums[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, ones),
                                                                      av[i].template half<H>(), sums[i], 0, 0, 0);
            }
        };
        half(std::integral_constant<int, 0>{});
        half(std::integral_constant<int, 1>{});
    }

    const int pc = pair_column();
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int n = n0 + (wm * MT + i) * 16 + lane % 16;
        if (sum_here && n < g.N && lane < 16) g.db[(int64_t)e * g.N + n] = sums[i][0];
#pragma unroll
        for (int j = 0; j < NT; j += 2) {
            float v[8];
            pair_values(acc[i][j], acc[i][j + 1], v);
            const int k = k0 + (wn * NT + j) * 16 + pc;
            if (n < g.N && k < g.K) {
                const int64_t o = ((int64_t)e * g.N + n) * g.K + k;
                if constexpr (WIDE) {
                    f32x4* d = reinterpret_cast<f32x4*>(static_cast<float*>(g.dw) + o);
                    d[0] = f32x4{v[0], v[1], v[2], v[3]};
                    d[1] = f32x4{v[4], v[5], v[6], v[7]};
                } else {
                    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(g.dw) + o) = pack8(v);
                }
            }
        }
    }
}

}  // namespace

int64_t grouped_grad_w_tiles(int E, int N, int K) {
    return (int64_t)E * ((N + kTileN - 1) / kTileN) * ((K + kTileK - 1) / kTileK);
}

hipError_t launch_grouped_grad_w(const GroupedGradArgs& g, hipStream_t stream) {
    const int n_tiles = (g.N + kTileN - 1) / kTileN, k_tiles = (g.K + kTileK - 1) / kTileK;
    const uint32_t tiles = (uint32_t)grouped_grad_w_tiles(g.rows.E, g.N, g.K);
    const uint32_t grid = (tiles + 7) / 8 * 8;
    if (g.wide && g.db)
        grad_w_kernel<true, true><<<grid, kGroupedThreads, 0, stream>>>(g, n_tiles, k_tiles, tiles);
    else if (g.wide)
        grad_w_kernel<true, false><<<grid, kGroupedThreads, 0, stream>>>(g, n_tiles, k_tiles, tiles);
    else if (g.db)
        grad_w_kernel<false, true><<<grid, kGroupedThreads, 0, stream>>>(g, n_tiles, k_tiles, tiles);
    else
        grad_w_kernel<false, false><<<grid, kGroupedThreads, 0, stream>>>(g, n_tiles, k_tiles, tiles);
    return hipGetLastError();
}

}  // namespace moe
