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
// 355 in the same run, and 359 in a trace of 60 passes.)  Within a wave nothing overlaps: matrix
// cores are busy 28 % of a busy CU's cycles, LDS 21 %.  db is summed from the fragments of dy,
// in the first column tiles.  Every expert's gradient is written, zeros for one without rows;
// a tile is one workgroup's, so the sums run in one order.
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

// A piece of an expert, of `of`; the slots of the partial sums are numbered over the
// experts that have several pieces, and slot is the expert's first.
struct Piece {
    int e, at;  // e = -1: none
    int of, slot;
};
// Every expert's first piece has a workgroup a tile of its own; these are the others:
// number u of them, as find_tile() finds its tile.
__device__ __forceinline__ Piece find_piece(const GroupedRows& g, int piece, int u) {
    const int lane = (int)(threadIdx.x % kWave);
    int before = 0, slots = 0;
    for (int e0 = 0; e0 < g.E; e0 += kWave) {
        const int here = e0 + lane < g.E ? pieces_of(segment(g, e0 + lane).n, piece) : 1;
        const int upto = before + wave_inclusive_sum(here - 1);
        const int slots_upto = slots + wave_inclusive_sum(here > 1 ? here : 0);
        const int last = __builtin_amdgcn_readlane(upto, kWave - 1);
        if (u < last) {
            const int which = __builtin_ctzll(__ballot(upto > u));
            const int of = __builtin_amdgcn_readlane(here, which);
            return {e0 + which, u - (__builtin_amdgcn_readlane(upto, which) - (of - 1)) + 1, of,
                    __builtin_amdgcn_readlane(slots_upto, which) - of};
        }
        before = last;
        slots = __builtin_amdgcn_readlane(slots_upto, kWave - 1);
    }
    return {-1, 0, 0, 0};
}
// The first slot of expert e.
__device__ __forceinline__ int slot_of(const GroupedRows& g, int piece, int e) {
    int slots = 0;
    for (int e0 = 0; e0 < e; e0 += kWave) {
        const int at = e0 + (int)(threadIdx.x % kWave);
        const int here = at < e ? pieces_of(segment(g, at).n, piece) : 1;
        slots += __builtin_amdgcn_readlane(wave_inclusive_sum(here > 1 ? here : 0), kWave - 1);
    }
    return slots;
}

template <bool WIDE, bool DB, bool PIECES>
__global__ __launch_bounds__(kThreads, 2) void grad_w_kernel(GroupedGradArgs g, int k_tiles, int per_expert) {
    __shared__ __align__(16) uint8_t lds[kStages * kStage];
    const int lane = (int)(threadIdx.x % kWave), wave = (int)uniform(threadIdx.x / kWave);
    const int wm = wave / 2, wn = wave % 2;
    // Tiles expert by expert (piece by piece), row by row: each XCD has a share of every
    // expert, so that none waits for the one that has most rows (64 experts, skewed: 833
    // us with whole experts on an XCD, and no less for 128 even ones).
    Piece p = {(int)(blockIdx.x / (uint32_t)per_expert), 0, 1, 0};
    if constexpr (PIECES) {
        if (p.e >= g.rows.E) {
            p = find_piece(g.rows, g.piece, p.e - g.rows.E);
        } else {
            p.of = pieces_of(segment(g.rows, p.e).n, g.piece);
            if (p.of > 1) p.slot = slot_of(g.rows, g.piece, p.e);
        }
        if (p.e < 0 || (p.of > 1 && p.slot + p.of > g.slots)) return;  // (the latter if segments overlap)
    }
    const int e = p.e, at = (int)(blockIdx.x % (uint32_t)per_expert);
    const int n0 = at / k_tiles * kTileN, k0 = at % k_tiles * kTileK;
    Segment seg = segment(g.rows, e);
    if constexpr (PIECES) {
        seg.first += p.at * g.piece;
        seg.n = min(seg.n - p.at * g.piece, g.piece);
    }
    const uint32_t lda = (uint32_t)g.N * 2, ldb = (uint32_t)g.K * 2;
    const int steps = (int)(((uint32_t)seg.n + kStep - 1) / kStep);
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

    const bool partial = PIECES && p.of > 1;
    float* const sums_out = partial ? g.partial_db + (int64_t)(p.slot + p.at) * g.N : DB ? g.db + (int64_t)e * g.N : nullptr;
    const int64_t first = (int64_t)(partial ? p.slot + p.at : e) * g.N * g.K;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int n = n0 + (wm * MT + i) * 16 + lane % 16;
        if (sum_here) {  // a lane has summed its quarter of the rows
            const float s = __builtin_bit_cast(float, across_rows(__builtin_bit_cast(uint32_t, sums[i])));
            if (lane < 16 && n < g.N) sums_out[n] = s;
        }
        const int row = n0 + (wm * MT + i) * 16 + line_row();
#pragma unroll
        for (int j = 0; j < NT; j += 2) {
            const int k = k0 + (wn * NT + j) * 16 + line_column();
            float v[8];
            pair_values(acc[i][j], acc[i][j + 1], v);
            const bool inside = row < g.N && k < g.K;
            const int64_t o = first + (int64_t)row * g.K + k;
            if (WIDE || partial) {
                to_lines(v);
                f32x4* d = reinterpret_cast<f32x4*>((partial ? g.partial : static_cast<float*>(g.dw)) + o);
                if (inside) {
                    d[0] = f32x4{v[0], v[1], v[2], v[3]};
                    d[1] = f32x4{v[4], v[5], v[6], v[7]};
                }
            } else {
                const u32x4 b = to_lines(pack8(v));
                if (inside) store(static_cast<uint16_t*>(g.dw) + o, b);
            }
        }
    }
}

// The partial sums of the experts that have several: workgroup row y is the y-th of
// them, x a share of its N K values and of its N sums.
template <bool WIDE, bool DB>
__global__ __launch_bounds__(kThreads) void join_kernel(GroupedGradArgs g, uint32_t vectors) {
    // the blockIdx.y-th expert with several pieces, and its slot
    const int lane = (int)(threadIdx.x % kWave);
    int e = -1, of = 0, slot = 0, seen = 0, slots = 0;
    for (int e0 = 0; e0 < g.rows.E; e0 += kWave) {
        const int here = e0 + lane < g.rows.E ? pieces_of(segment(g.rows, e0 + lane).n, g.piece) : 0;
        const int several = here > 1 ? here : 0;
        const int upto = seen + wave_inclusive_sum(several > 0 ? 1 : 0), slots_upto = slots + wave_inclusive_sum(several);
        const uint64_t which = __ballot(several > 0 && upto == (int)blockIdx.y + 1);
        if (which != 0) {
            const int w = __builtin_ctzll(which);
            e = e0 + w;
            of = __builtin_amdgcn_readlane(several, w);
            slot = __builtin_amdgcn_readlane(slots_upto - several, w);
        }
        seen = __builtin_amdgcn_readlane(upto, kWave - 1);
        slots = __builtin_amdgcn_readlane(slots_upto, kWave - 1);
    }
    if (e < 0 || slot + of > g.slots) return;
    const int64_t size = (int64_t)g.N * g.K;
    for (uint32_t i = blockIdx.x * kThreads + threadIdx.x; i < vectors; i += gridDim.x * kThreads) {
        float v[8] = {};
        for (int q = 0; q < of; ++q) {
            const f32x4* s = reinterpret_cast<const f32x4*>(g.partial + (slot + q) * size) + (size_t)i * 2;
            const f32x4 a = s[0], b = s[1];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] += a[j];
                v[4 + j] += b[j];
            }
        }
        if constexpr (WIDE) {
            f32x4* d = reinterpret_cast<f32x4*>(static_cast<float*>(g.dw) + e * size) + (size_t)i * 2;
            d[0] = f32x4{v[0], v[1], v[2], v[3]};
            d[1] = f32x4{v[4], v[5], v[6], v[7]};
        } else {
            reinterpret_cast<u32x4*>(static_cast<uint16_t*>(g.dw) + e * size)[i] = pack8(v);
        }
    }
    if constexpr (DB) {
        for (int n = (int)(blockIdx.x * kThreads + threadIdx.x); n < g.N; n += (int)(gridDim.x * kThreads)) {
            float v = 0.0f;
            for (int q = 0; q < of; ++q) v += g.partial_db[(int64_t)(slot + q) * g.N + n];
            g.db[(int64_t)e * g.N + n] = v;
        }
    }
}

template <bool WIDE, bool DB>
hipError_t launch(const GroupedGradArgs& g, hipStream_t stream) {
    const int k_tiles = (g.K + kTileK - 1) / kTileK, per_expert = (g.N + kTileN - 1) / kTileN * k_tiles;
    if (g.piece == 0) {
        grad_w_kernel<WIDE, DB, false>
            <<<(uint32_t)g.rows.E * (uint32_t)per_expert, kThreads, 0, stream>>>(g, k_tiles, per_expert);
        return hipGetLastError();
    }
    const int pieces = g.rows.R / g.piece + g.rows.E;
    grad_w_kernel<WIDE, DB, true>
        <<<(uint32_t)pieces * (uint32_t)per_expert, kThreads, 0, stream>>>(g, k_tiles, per_expert);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const uint32_t vectors = (uint32_t)((int64_t)g.N * g.K / 8);
    const uint32_t experts = (uint32_t)(g.rows.R / g.piece < g.rows.E ? g.rows.R / g.piece : g.rows.E);
    const uint32_t blocks = (vectors + kThreads - 1) / kThreads;
    join_kernel<WIDE, DB><<<dim3(blocks < 256 ? blocks : 256, experts), kThreads, 0, stream>>>(g, vectors);
    return hipGetLastError();
}

// Rows of a piece: those whose steps are as many as one of the workgroups that run at a
// time would have if all tiles' steps were spread evenly, 1024 at least: below that
// joining costs more than it gives.  0: whole experts, where none can have more rows, or
// an expert has kTilesMax tiles or more.  Below that pieces win (whole and in pieces, us: 34
// skewed experts of 31239 rows, 784 x 328 in fp32 369 and 79; one of 3059 rows, 224 x 4232, with
// dx, 79 and 47).  From there on it goes by what the rule does not look at, the number of experts
// and how uneven they are:
//   128 even experts, 32768 rows, 1536 x 2048 (96 tiles): 348 and 366, since nothing is cut and the
//     search and the join are paid; one expert, 8192 rows, 2048 x 7168 (448 tiles): 238 and 248;
//   one expert, 32768 rows: 1024 x 2048 (64 tiles) 624 and 167, 1536 x 2048 629 and 240; 8192 rows,
//     4096 x 1408 in fp32 (192 tiles) 163 and 135; 4096 rows, 2048 x 2048 (128 tiles) 82 and 62;
//   8 experts, 32768 rows, 1536 x 2048: even 209 and 206, skewed 392 and 265; 128 skewed ones 602
//     and 449; 64 skewed ones, 6138 rows, 4096 x 1408 in fp32 366 and 357.
// So few or uneven experts of many rows lose by the whole ones, up to fourfold.
constexpr int kSlots = 512, kPieceMin = 1024, kTilesMax = 64;
int piece_rows(const GroupedRows& g, int N, int K) {
    const int64_t per_expert = (int64_t)((N + kTileN - 1) / kTileN) * ((K + kTileK - 1) / kTileK);
    if (per_expert >= kTilesMax) return 0;
    int64_t rows = (g.R * per_expert + kSlots - 1) / kSlots;
    rows = ((rows < kPieceMin ? kPieceMin : rows) + kStep - 1) / kStep * kStep;
    return rows >= g.R ? 0 : (int)rows;
}
// Partial sums: experts with several pieces have more than a piece's rows each, and at
// most twice as many pieces as whole ones.
int64_t slots_of(const GroupedRows& g, int piece) { return piece == 0 ? 0 : 2 * (int64_t)(g.R / piece); }

}  // namespace

int64_t grouped_grad_w_tiles(const GroupedRows& g, int N, int K) {
    const int64_t per_expert = (int64_t)((N + kTileN - 1) / kTileN) * ((K + kTileK - 1) / kTileK);
    if (g.R < 0 || g.E < 1) return 0;
    const int piece = piece_rows(g, N, K);
    return (g.E + (piece > 0 ? g.R / piece : 0)) * per_expert;
}

size_t grouped_grad_w_workspace_bytes(const GroupedRows& g, int N, int K) {
    return (size_t)slots_of(g, piece_rows(g, N, K)) * N * (K + 1) * sizeof(float);
}

hipError_t launch_grouped_grad_w(GroupedGradArgs g, void* workspace, hipStream_t stream) {
    g.piece = piece_rows(g.rows, g.N, g.K);
    g.slots = (int)slots_of(g.rows, g.piece);
    g.partial = static_cast<float*>(workspace);
    g.partial_db = g.partial + (int64_t)g.slots * g.N * g.K;
    if (g.wide) return g.db ? launch<true, true>(g, stream) : launch<true, false>(g, stream);
    return g.db ? launch<false, true>(g, stream) : launch<false, false>(g, stream);
}

}  // namespace moe
