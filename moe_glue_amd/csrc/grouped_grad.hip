// moe_grouped_linear_grad_w on gfx950: dw_e = dy_e^T x_e and db_e = the column
// sums of dy_e, the sum running over an expert's rows.
//
// Both operands lie with the sum across their rows (grouped.h, "columns"); rows past
// the segment's end read as zeros.  An expert has a few hundred rows, so a tile is a
// handful of steps and its stores: bound by the bytes of dw, and by what a workgroup
// does before its first and behind its last product.  So a CU has two workgroups of
// four waves, a tile of 128 by 256 each: one's first loads and its stores fall into the
// other's products, and nothing waits for a store.  (Workgroups that stay and take tile
// after tile, their loads running on into the next: 397 us for 128 experts' 1536 x 2048 of
// 256 rows, since loads behind a tile's stores cannot be waited for without them; here
// 367.)  db is summed from the fragments of dy, in the first column tiles.  Every
// expert's gradient is written, zeros for one without rows; a tile is one workgroup's, so
// the sums run in one order.
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

template <bool WIDE, bool DB>
__global__ __launch_bounds__(kThreads, 2) void grad_w_kernel(GroupedGradArgs g, int k_tiles, int per_expert) {
    __shared__ __align__(16) uint8_t lds[kStages * kStage];
    const int lane = (int)(threadIdx.x % kWave), wave = (int)uniform(threadIdx.x / kWave);
    const int wm = wave / 2, wn = wave % 2;
    // Tiles expert by expert, row by row: each XCD has a share of every expert, so that
    // none waits for the one that has most rows (64 experts, skewed: 833 us with whole
    // experts on an XCD, and no less for 128 even ones).
    const int e = (int)(blockIdx.x / (uint32_t)per_expert), at = (int)(blockIdx.x % (uint32_t)per_expert);
    const int n0 = at / k_tiles * kTileN, k0 = at % k_tiles * kTileK;
    const Segment seg = segment(g.rows, e);
    const uint32_t lda = (uint32_t)g.N * 2, ldb = (uint32_t)g.K * 2;
    const int steps = (seg.n + kStep - 1) / kStep;
    AOperand a;
    a.set(reinterpret_cast<const uint8_t*>(g.dy) + (int64_t)seg.first * lda + n0 * 2, (int64_t)seg.n * lda - n0 * 2,
          lda);
    BOperand b;
    b.set(reinterpret_cast<const uint8_t*>(g.x) + (int64_t)seg.first * ldb + k0 * 2, (int64_t)seg.n * ldb - k0 * 2,
          ldb);

    f32x4 acc[MT][NT];
    float sums[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        sums[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    const bool sum_here = DB && k0 == 0 && wn == 0;
    const uint32_t a_at = AFragment::at(), b_at = AOperand::LDS_BYTES + BFragment::at();

#pragma unroll
    for (int s = 0; s < 2; ++s) {
        if (s < steps) {
            a.load(s, lds + s * kStage);
            b.load(s, lds + s * kStage + AOperand::LDS_BYTES);
        }
    }
    int buf = 0;
    for (int step = 0; step < steps; ++step) {
        if (step + 1 < steps)
            loads_done<kLoads>();  // but the next step's
        else
            loads_done<0>();
        reads_done();
        meet();
        const uint8_t* q = lds + buf * kStage;
        AFragment av[MT];
        BFragment bv[NT];
#pragma unroll
        for (int i = 0; i < MT; ++i) av[i].read(q, a_at ^ (wm * MT + i) * 32);
#pragma unroll
        for (int j = 0; j < NT; ++j) bv[j].read(q, b_at ^ (wn * NT + j) * 32);
        // The step after next, load by load among the products: all at once they hold the
        // wave up until the CU has taken them.
        const bool more = step + 2 < steps;
        const BufferWords a_buf = a.buffer(step + 2), b_buf = b.buffer(step + 2);
        uint8_t* const to = lds + (buf == 0 ? 2 : buf - 1) * kStage;
        unrolled<NT>([&](auto index) {
            constexpr int j = decltype(index)::value;
#pragma unroll
            for (int i = 0; i < MT; ++i)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bv[j].template half<0>(),
                                                                    av[i].template half<0>(), acc[i][j], 0, 0, 0);
            if constexpr (j < AOperand::LOADS) {
                if (more) a.load_one<j>(a_buf, to);
            } else if constexpr (j < kLoads) {
                if (more) b.load_one<j - AOperand::LOADS>(b_buf, to + AOperand::LDS_BYTES);
            }
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

#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int n = n0 + (wm * MT + i) * 16 + lane % 16;
        if (sum_here) {  // a lane has summed its quarter of the rows
            const float s = __builtin_bit_cast(float, across_rows(__builtin_bit_cast(uint32_t, sums[i])));
            if (lane < 16 && n < g.N) g.db[(int64_t)e * g.N + n] = s;
        }
#pragma unroll
        for (int j = 0; j < NT; j += 2) {
            const int k = k0 + (wn * NT + j) * 16 + pair_column();
            float v[8];
            pair_values(acc[i][j], acc[i][j + 1], v);
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
    const int k_tiles = (g.K + kTileK - 1) / kTileK, per_expert = (g.N + kTileN - 1) / kTileN * k_tiles;
    const uint32_t grid = (uint32_t)g.rows.E * (uint32_t)per_expert;
    if (g.wide && g.db)
        grad_w_kernel<true, true><<<grid, kThreads, 0, stream>>>(g, k_tiles, per_expert);
    else if (g.wide)
        grad_w_kernel<true, false><<<grid, kThreads, 0, stream>>>(g, k_tiles, per_expert);
    else if (g.db)
        grad_w_kernel<false, true><<<grid, kThreads, 0, stream>>>(g, k_tiles, per_expert);
    else
        grad_w_kernel<false, false><<<grid, kThreads, 0, stream>>>(g, k_tiles, per_expert);
    return hipGetLastError();
}

}  // namespace moe
