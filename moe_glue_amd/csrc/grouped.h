// Products of rows in expert order with their experts' weights, and their
// gradients: the tile that the kernels of grouped_linear.hip and
// grouped_grad.hip share.
//
// A workgroup of eight waves computes D = A B^T over a tile of 32 MT rows (m) by
// 64 NT columns (n), fp32, with v_mfma_f32_16x16x32_bf16 (or the block-scaled
// 16x16x128 on MXFP8).  Steps of 128 bytes of a row (64 bf16 or 128 E4M3) of both
// operands go from memory to LDS without registers (buffer_load_dwordx4 .. lds,
// 16 bytes a lane), through a ring of as many stages as LDS holds: loads of a
// stage are in flight while the stages before it are multiplied, with one barrier
// a step.  An operand lies in memory with the summed index along its rows
// ("rows": x, dy for dx, the weights of the forward product) or across them
// ("columns": the weights for dx, both operands of the weight gradient).
//
//   rows     LDS rows of 128 bytes; lane l of a fragment reads 16-byte pieces
//            l / 16 and 4 + l / 16 of row l % 16: k 8 (l / 16) .. + 7 of each half
//            for bf16, and for MXFP8 the two halves of a 16x16x128 operand.
//            Piece c of row r is stored at c ^ (r / 2 % 8), so the 16 rows that a
//            read touches fall into different banks.
//   columns  LDS rows of one k each; ds_read_b64_tr_b16 hands lane l 4 k of
//            column l % 16.  16 columns (32 bytes) of row k are stored at unit
//            u ^ (k % 4 + k / 8 % 2 * 4): the 8 rows that half a wave touches fall
//            into different banks.
//
// The operands are swapped in the matrix instruction (n is its row), so that a
// lane's four accumulators are neighbouring columns of one row of D; swapping
// 16-lane rows between two tiles makes them eight: 16-byte stores in bf16.
#pragma once

#include "device_common.h"
#include "kernels.h"

namespace moe {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

#define MOE_LDS __attribute__((address_space(3)))

constexpr int kGroupedThreads = 512;
constexpr int kLdsBytes = 160 * 1024;
constexpr int kStepBytes = 128;             // of a row, per step
constexpr uint32_t kPastEnd = 0x80000000u;  // an offset past the end of every buffer

// ---------------------------------------------------------------- segments
// Rows of expert e: [first, first + n), inside [0, R) whatever the arrays hold.
struct Segment {
    int first, n;
};
__device__ __forceinline__ Segment segment(const GroupedRows& g, int e) {
    if (g.offsets == nullptr) return {0, g.R};
    const int first = min(max(g.offsets[e], 0), g.R);
    const int n = g.counts != nullptr ? g.counts[e] : min(max(g.offsets[e + 1], 0), g.R) - first;
    return {first, min(max(n, 0), g.R - first)};
}

// Row tiles of an expert with n rows: up to kSplitTiles tiles share the rows
// evenly (in 32s), more are full but for the last.
constexpr int kSplitTiles = 4;
__host__ __device__ __forceinline__ int row_tiles(int n) { return (n + kGroupedRows - 1) / kGroupedRows; }
__host__ __device__ __forceinline__ int tile_rows(int n) {
    const int t = row_tiles(n);
    return t > kSplitTiles || t == 0 ? kGroupedRows : ((n + t - 1) / t + 31) / 32 * 32;
}

struct Tile {
    int e;      // expert, -1: none
    int first;  // first row
    int rows;
    int last_rows;  // rows of a whole tile of this expert (what the tile is laid out for)
    int col;    // column tile
};

// The tile of this workgroup.  Tiles are numbered expert by expert; in an expert,
// groups of kTogether row tiles by column tile by row tile.  Each XCD (workgroups
// b with equal b % 8) takes one run of them, so that the weights that row tiles
// share, and the rows that column tiles share, meet in its L2.  Every wave does
// this on its own: a lane sums the tiles of up to 8 experts, the wave's prefix
// sums find the one that holds the tile.
constexpr int kTogether = 8;
__device__ __forceinline__ Tile find_tile(const GroupedRows& g, int col_tiles) {
    const int lane = (int)(threadIdx.x % kWave);
    const int per = (g.E + kWave - 1) / kWave;
    int mine = 0;
    for (int i = 0; i < per; ++i) {
        const int e = lane * per + i;
        if (e < g.E) mine += row_tiles(segment(g, e).n);
    }
    const int upto = wave_inclusive_sum(mine);
    const int total = __builtin_amdgcn_readlane(upto, kWave - 1) * col_tiles;
    const int run = (total + 7) / 8;
    const int u = (int)(blockIdx.x % 8) * run + (int)(blockIdx.x / 8);
    Tile t = {-1, 0, 0, 0, 0};
    if ((int)(blockIdx.x / 8) >= run || u >= total) return t;
    const int owner = __builtin_ctzll(__ballot(upto * col_tiles > u));
    int before = __builtin_amdgcn_readlane(upto - mine, owner);
    for (int i = 0; i < per; ++i) {
        const int e = owner * per + i;
        const Segment s = segment(g, e);
        const int tiles = row_tiles(s.n);
        if (u < (before + tiles) * col_tiles) {
            const int v = u - before * col_tiles;
            const int group = v / (kTogether * col_tiles);
            const int in_group = min(kTogether, tiles - group * kTogether);
            const int at = v - group * kTogether * col_tiles;
            const int m = group * kTogether + at % in_group;
            t.e = e;
            t.last_rows = tile_rows(s.n);
            t.first = s.first + m * t.last_rows;
            t.rows = min(t.last_rows, s.n - m * t.last_rows);
            t.col = at / in_group;
            return t;
        }
        before += tiles;
    }
    return t;
}

// ------------------------------------------------------------------- loads
__device__ __forceinline__ __amdgpu_buffer_rsrc_t grouped_buffer(const void* p, int64_t bytes) {
    const int64_t n = bytes < 0 ? 0 : bytes > (int64_t)kPastEnd ? (int64_t)kPastEnd : bytes;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)(uint32_t)n, kRawBufferWord3);
}
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t r, uint32_t lane, uint32_t scalar, uint8_t* lds) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (MOE_LDS void*)lds, 16, (int)lane, (int)scalar, 0, 0);
}

// An operand with the summed index along its rows: `rows` rows of `ld` bytes from
// base on; J * 64 rows of LDS, J loads a wave.  Rows past the last read zeros, as
// do bytes past a row's end.
template <int J>
struct RowsOperand {
    static constexpr int LDS_BYTES = J * 64 * kStepBytes;
    __amdgpu_buffer_rsrc_t buf;
    uint32_t at[J];
    uint32_t piece, ld;
    __device__ __forceinline__ void set(const uint8_t* base, int64_t bytes, uint32_t ld_, uint32_t first_row,
                                        uint32_t row_step) {
        const uint32_t lane = threadIdx.x % kWave, wave = uniform(threadIdx.x / kWave);
        buf = grouped_buffer(base, bytes);
        ld = ld_;
        const uint32_t row = wave * 8 + lane / 8;  // of LDS, modulo 64
        piece = (lane % 8 ^ (row / 2 % 8)) * 16;
#pragma unroll
        for (int j = 0; j < J; ++j) at[j] = (first_row + lane / 8 + j * row_step) * ld + piece;
    }
    __device__ __forceinline__ void load(int step, uint8_t* lds) const {
        const uint32_t wave = uniform(threadIdx.x / kWave);
        const uint32_t k = (uint32_t)step * kStepBytes;
        const bool past = k + piece >= ld;
#pragma unroll
        for (int j = 0; j < J; ++j) load_to_lds(buf, past ? kPastEnd : at[j], k, lds + (j * 8 + wave) * 1024);
    }
};

// An operand with the summed index across its rows: rows [0, sum) of `ld` bytes
// from base on (base: the first column of the tile), W bytes of each; J loads a
// wave of 64 rows.
template <int J>
struct ColumnsOperand {
    static constexpr int W = J * 128;  // 64 rows * W = J * 8 KiB
    static constexpr int LDS_BYTES = 64 * W;
    const uint8_t* base;
    int64_t bytes;  // from base to the end of the last row
    uint32_t at[J];
    uint32_t ld;
    __device__ __forceinline__ void set(const uint8_t* base_, int64_t bytes_, uint32_t ld_) {
        constexpr uint32_t ROWS = 1024 / W, PIECES = W / 16;
        const uint32_t lane = threadIdx.x % kWave, wave = uniform(threadIdx.x / kWave);
        base = base_;
        bytes = bytes_;
        ld = ld_;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const uint32_t row = (j * 8 + wave) * ROWS + lane / PIECES;
            const uint32_t key = row % 4 + row / 8 % 2 * 4;
            const uint32_t piece = lane % PIECES;
            at[j] = row * ld + ((piece / 2 ^ key) * 2 + piece % 2) * 16;
        }
    }
    __device__ __forceinline__ void load(int step, uint8_t* lds) const {
        const uint32_t wave = uniform(threadIdx.x / kWave);
        const int64_t from = (int64_t)step * 64 * ld;
        const __amdgpu_buffer_rsrc_t buf = grouped_buffer(base + from, bytes - from);
#pragma unroll
        for (int j = 0; j < J; ++j) load_to_lds(buf, at[j], 0, lds + (j * 8 + wave) * 1024);
    }
};

// --------------------------------------------------------------- fragments
// 16 bytes of row r, piece c (0..7) of a rows operand in LDS.
__device__ __forceinline__ uint32_t rows_at(uint32_t row, uint32_t piece) {
    return row * kStepBytes + ((piece ^ (row / 2 % 8)) * 16);
}
// A lane's place in a columns operand of W bytes a row, less its unit of 16
// columns: add the step half's 32 W, then xor unit * 32.
template <int W>
__device__ __forceinline__ uint32_t columns_at() {
    const uint32_t lane = threadIdx.x % kWave;
    const uint32_t row = lane / 16 * 8 + lane % 16 / 4;
    const uint32_t key = row % 4 + row / 8 % 2 * 4;
    return row * W + key * 32 + lane % 4 * 8;
}
template <int W>
__device__ __forceinline__ bf16x8 columns_fragment(const uint8_t* lds, uint32_t at) {
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_LDS s16x4*)(lds + at));
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_LDS s16x4*)(lds + at + 4 * W));
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    return __builtin_bit_cast(bf16x8, s16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]});
}

// Waits until at most N of this wave's loads are in flight and its LDS reads are
// done, then for the other waves.
template <int N>
__device__ __forceinline__ void wait_and_meet() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Eight neighbouring columns of one row of D, of the tile pair (a, b): see
// pair_column() for which.  Quarter q of a row of 16 lanes holds columns 4 q .. of
// both tiles; the swap of odd rows of a with even rows of b gives lanes of even
// q tile a and of odd q tile b.
__device__ __forceinline__ void pair_values(const f32x4& a, const f32x4& b, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float ai = a[i], bi = b[i];  // (a bit cast of a vector's element takes element 0)
        const auto p = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, ai),
                                                        __builtin_bit_cast(uint32_t, bi), false, false);
        const uint32_t lo = p[0], hi = p[1];
        v[i] = __builtin_bit_cast(float, lo);
        v[4 + i] = __builtin_bit_cast(float, hi);
    }
}
__device__ __forceinline__ int pair_column() {
    const int q = (int)(threadIdx.x % kWave) / 16;
    return q % 2 * 16 + q / 2 * 8;
}

}  // namespace moe
