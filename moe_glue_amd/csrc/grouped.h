// Products of rows in expert order with their experts' weights, and their
// gradients: what the kernels of grouped_linear.hip, grouped_few.hip and
// grouped_grad.hip share, and the tile of the first.
//
// A workgroup of eight waves, two by four, computes D = A B^T over a tile of 64 MH
// rows (m) by 256 columns (n) in fp32, with v_mfma_f32_16x16x32_bf16 (or the
// block-scaled 16x16x128 on MXFP8).  Steps of 128 bytes of a row (64 bf16 or 128
// E4M3) of both operands go from memory to LDS without registers
// (buffer_load_dwordx4 .. lds, 16 bytes a lane), two to four steps ahead.  An
// operand lies in memory with the summed index along its rows ("rows": x, dy for dx,
// the weights of the forward product) or across them ("columns": the weights for dx,
// both operands of the weight gradient).
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

#include <type_traits>

#include "device_common.h"
#include "kernels.h"

namespace moe {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

#define MOE_LDS __attribute__((address_space(3)))

constexpr int kGroupedThreads = 512;
constexpr int kLdsBytes = 160 * 1024;
constexpr int kStepBytes = 128;             // of a row, per step
// An offset past the end of every buffer.  (The range check takes lane's and scalar's offsets
// together and does not wrap: a scalar offset beyond a short buffer reads zeros too.  Measured.)
constexpr uint32_t kPastEnd = 0x80000000u;

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

// Row tiles of an expert with n rows, each of up to `whole` (a multiple of 64): n
// in units of 64 rows, dealt out evenly.
__host__ __device__ __forceinline__ int row_tiles(int n, int whole) { return (n + whole - 1) / whole; }

// Pieces of an expert's n rows, of up to `piece`; none has one too.  (n may be any int32: a
// weight gradient's rows have no other limit.)
__host__ __device__ __forceinline__ int pieces_of(int n, int piece) { return n > 0 ? (n - 1) / piece + 1 : 1; }

struct Tile {
    int e;      // expert
    int first;  // first row
    int rows;   // 0: no tile
    int col;    // column tile
};

// The tile of this workgroup.  Tiles are numbered expert by expert; in an expert,
// groups of kTogether row tiles by column tile by row tile.  The XCDs (workgroups b with
// equal b % 8) take kRun tiles each by turns, so that
// the weights that row tiles share, and the rows that column tiles share, meet in its
// L2, and an expert with many rows is not one XCD's alone (64 experts under skewed
// routing, MXFP8: 187 us with an eighth of all tiles at a stretch, 171 so).  Every wave
// looks for itself: a lane sums the tiles of up to 8 experts and the wave's prefix sums
// find the lane that holds the tile; then, past 64 experts, the lane's own the same way.
constexpr int kTogether = 8, kRun = 8;
__device__ __forceinline__ Tile find_tile(const GroupedRows& g, int col_tiles, int whole) {
    const int lane = (int)(threadIdx.x % kWave);
    const int per = (g.E + kWave - 1) / kWave;
    int mine = 0;
    Segment s = {0, 0};
    for (int i = 0; i < per; ++i) {
        const int e = lane * per + i;
        if (e < g.E) {
            s = segment(g, e);
            mine += row_tiles(s.n, whole);
        }
    }
    const int upto = wave_inclusive_sum(mine);
    const int total = __builtin_amdgcn_readlane(upto, kWave - 1) * col_tiles;
    const uint32_t run = min((uint32_t)(total + 7) / 8, (uint32_t)kRun);
    if (total == 0) return {0, 0, 0, 0};
    const int u = (int)(blockIdx.x / 8 / run * (8 * run) + blockIdx.x % 8 * run + blockIdx.x / 8 % run);
    if (u >= total) return {0, 0, 0, 0};
    const int owner = __builtin_ctzll(__ballot(upto * col_tiles > u));
    const int before = __builtin_amdgcn_readlane(upto - mine, owner);
    int which = owner, here = mine, until = upto;
    if (per > 1) {
        s = {0, 0};
        if (lane < per && owner * per + lane < g.E) s = segment(g, owner * per + lane);
        here = row_tiles(s.n, whole);
        until = before + wave_inclusive_sum(here);
        which = __builtin_ctzll(__ballot(until * col_tiles > u));
    }
    const int n = __builtin_amdgcn_readlane(s.n, which), tiles = __builtin_amdgcn_readlane(here, which);
    const int v = u - __builtin_amdgcn_readlane(until - here, which) * col_tiles;
    const int group = v / (kTogether * col_tiles);
    const int in_group = min(kTogether, tiles - group * kTogether);
    const int at = v - group * kTogether * col_tiles;
    const int m = group * kTogether + at % in_group;
    const int units = (n + 63) / 64, each = units / tiles, more = units % tiles;
    const int first = (m * each + min(m, more)) * 64;
    return {per > 1 ? owner * per + which : owner, __builtin_amdgcn_readlane(s.first, which) + first,
            min((each + (m < more ? 1 : 0)) * 64, n - first), at / in_group};
}

template <int N, class F>
__device__ __forceinline__ void unrolled(F&& f) {
    if constexpr (N > 0) {
        unrolled<N - 1>(f);
        f(std::integral_constant<int, N - 1>{});
    }
}

// ------------------------------------------------------------------- loads
__device__ __forceinline__ int grouped_bytes(int64_t bytes) {
    return (int)(uint32_t)(bytes < 0 ? 0 : bytes > (int64_t)kPastEnd ? (int64_t)kPastEnd : bytes);
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t grouped_buffer(const void* p, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, grouped_bytes(bytes), kRawBufferWord3);
}
typedef __attribute__((ext_vector_type(4))) int BufferWords;
__device__ __forceinline__ BufferWords buffer_words(const void* p, int64_t bytes) {
    const uint64_t at = reinterpret_cast<uint64_t>(p);
    return {(int)(uint32_t)at, (int)((uint32_t)(at >> 32) & 0xFFFFu), grouped_bytes(bytes), kRawBufferWord3};
}
// 16 bytes (or a dword) a lane from byte lane + scalar of a buffer to LDS, the wave's one
// behind the other.  In assembly, for behind the builtin the compiler takes a transposing
// LDS read for one of what is in flight, whatever buffer it goes to, and waits for all
// loads before it (dx of 32768 rows, 128 experts, 1536 x 2048: 336 us, 298 without).  There is
// no register to write; waiting is the caller's (loads_done).  M0 holds the LDS address,
// and the wait state is the one it asks for before a load to LDS.  (M0 is reserved: the compiler
// keeps nothing in it, and takes no clobber of it.)  A scalar register that a
// vector instruction wrote may be read by a load five wait states later at the earliest, which
// the compiler does not see to here: the buffers come from scalar arithmetic on values read
// from lanes long before, and tests/test_grouped_listing.py follows every path to every load.
// (All five in the assembly: 1023 x 2816 x 4096 40.6 us, then 43.2; 8192 x 7168 x 2048 222 and 227.)
__device__ __forceinline__ void load_to_lds(const BufferWords& r, uint32_t lane, uint32_t scalar, uint8_t* lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(
                     (uint32_t)(uintptr_t)(MOE_LDS uint8_t*)lds),
                 "v"(lane), "s"(r), "s"(scalar)
                 : "memory");
}
__device__ __forceinline__ void load_dword_to_lds(const BufferWords& r, uint32_t lane, uint8_t* lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(
                     (uint32_t)(uintptr_t)(MOE_LDS uint8_t*)lds),
                 "v"(lane), "s"(r)
                 : "memory");
}

// An operand with the summed index along its rows, of `ld` bytes each; load j of a
// wave brings eight of 64 LDS rows.  Rows past the end of their buffer and bytes past
// a row's end read zeros.
template <int J>
struct RowsOperand {
    uint32_t at[J];
    uint32_t piece, ld;
    __device__ __forceinline__ void set(uint32_t ld_) {
        const uint32_t lane = threadIdx.x % kWave, wave = uniform(threadIdx.x / kWave);
        ld = ld_;
        const uint32_t row = wave * 8 + lane / 8;
        piece = (lane % 8 ^ (row / 2 % 8)) * 16;
#pragma unroll
        for (int j = 0; j < J; ++j) at[j] = (row + j * 64) * ld + piece;
    }
    // Loads FROM .. TO - 1 of a step, the first of them to LDS row 0.  Steps in order:
    // from the one that holds a row's end on, lanes past it stay turned away.
    template <int FROM, int TO>
    __device__ __forceinline__ void load(const BufferWords& buf, int step, uint8_t* lds) {
        const uint32_t wave = uniform(threadIdx.x / kWave);
        const uint32_t k = (uint32_t)step * kStepBytes;
        if (k + kStepBytes > ld) {
            const bool past = k + piece >= ld;
#pragma unroll
            for (int j = FROM; j < TO; ++j) at[j] = past ? kPastEnd : at[j];
        }
#pragma unroll
        for (int j = FROM; j < TO; ++j) load_to_lds(buf, at[j], k, lds + ((j - FROM) * 8 + wave) * 1024);
    }
};

// An operand with the summed index across its rows, of `ld` bytes each, in `bytes`
// bytes from base (the first column of the tile) on: K rows a step, W bytes of each,
// by a workgroup of WAVES waves.  Rows past the end read zeros.
template <int W, int K, int WAVES>
struct ColumnsOperand {
    static constexpr int LDS_BYTES = K * W;
    static constexpr int LOADS = LDS_BYTES / (WAVES * 1024);  // of a wave, per step
    const uint8_t* base;
    int64_t bytes;
    uint32_t at[LOADS];
    uint32_t ld;
    __device__ __forceinline__ void set(const uint8_t* base_, int64_t bytes_, uint32_t ld_) {
        constexpr uint32_t ROWS = 1024 / W, PIECES = W / 16;
        const uint32_t lane = threadIdx.x % kWave, wave = uniform(threadIdx.x / kWave);
        base = base_;
        bytes = bytes_;
        ld = ld_;
#pragma unroll
        for (int j = 0; j < LOADS; ++j) {
            const uint32_t row = (j * WAVES + wave) * ROWS + lane / PIECES;
            const uint32_t key = row % 4 + row / 8 % 2 * 4;
            const uint32_t piece = lane % PIECES;
            at[j] = row * ld + ((piece / 2 ^ key) * 2 + piece % 2) * 16;
        }
    }
    __device__ __forceinline__ BufferWords buffer(int step) const {
        const int64_t from = (int64_t)step * K * ld;
        return buffer_words(base + from, bytes - from);
    }
    template <int J>  // load J of a step
    __device__ __forceinline__ void load_one(const BufferWords& buf, uint8_t* lds) const {
        load_to_lds(buf, at[J], 0, lds + (J * WAVES + uniform(threadIdx.x / kWave)) * 1024);
    }
    __device__ __forceinline__ void load(int step, uint8_t* lds) const {
        const BufferWords buf = buffer(step);
        unrolled<LOADS>([&](auto j) { load_one<decltype(j)::value>(buf, lds); });
    }
};

// --------------------------------------------------------------- fragments
// 16 rows (columns of D) by a step's k, in a lane's registers.
struct RowsFragment {
    i32x4 lo, hi;
    // The lane's place for the 16 rows from row 0 on; 16 rows further is 2048 bytes on.
    static __device__ __forceinline__ uint32_t at() {
        const uint32_t lane = threadIdx.x % kWave, row = lane % 16;
        return row * kStepBytes + (lane / 16 ^ row / 2) * 16;
    }
    __device__ __forceinline__ void read(const uint8_t* p, uint32_t at) {
        lo = *reinterpret_cast<const i32x4*>(p + at);
        hi = *reinterpret_cast<const i32x4*>(p + (at ^ 64));
    }
    template <int H>
    __device__ __forceinline__ bf16x8 half() const {
        return __builtin_bit_cast(bf16x8, H == 0 ? lo : hi);
    }
    __device__ __forceinline__ i32x8 whole() const { return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7); }
};
template <int W, int K>  // bytes of an LDS row, rows of a step: 32 or 64
struct ColumnsFragment {
    s16x4 v[K / 16];
    // The lane's place for unit 0: xor the unit's 32 bytes in.
    static __device__ __forceinline__ uint32_t at() {
        const uint32_t lane = threadIdx.x % kWave;
        const uint32_t row = lane / 16 * 8 + lane % 16 / 4;
        return row * W + (row % 4 + row / 8 % 2 * 4) * 32 + lane % 4 * 8;
    }
    __device__ __forceinline__ void read(const uint8_t* p, uint32_t at) {
#pragma unroll
        for (int i = 0; i < K / 16; ++i)  // k 0..3, 4..7 of the lane's eight, of every 32
            v[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_LDS s16x4*)(p + at + (i / 2 * 32 + i % 2 * 4) * W));
    }
    template <int H>
    __device__ __forceinline__ bf16x8 half() const {
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(v[2 * H], v[2 * H + 1], 0, 1, 2, 3, 4, 5, 6, 7));
    }
};

// ------------------------------------------------------------------- steps
__device__ __forceinline__ void meet() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}
// This wave's LDS reads, and what it wrote to LDS itself (MXFP8 scale bytes), are done.
__device__ __forceinline__ void reads_done() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
// At most N of this wave's loads in flight.
template <int N>
__device__ __forceinline__ void loads_done() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// The steps of a tile.  A step is four quarters: the halves of the wave's rows by the
// halves of its columns,
//   0: rows 0, columns 0   1: rows 0, columns 1   2: rows 1, columns 1   3: rows 1, columns 0
// each of them a part that fills registers from LDS (and asks for the step after next)
// and a part of matrix instructions, with a barrier behind either.  The second four
// waves start one barrier late: on each SIMD one wave multiplies while the other reads.
//   read_a(h, buffer), read_b(h, buffer)   half h of a step to registers
//   multiply(ha, hb)
//   load(q, step, buffer)                  what quarter q = 1, 2, 3 asks for
// There are two buffers, and a part of one is asked for again as soon as both halves of
// the waves have read it: rows 0 and columns 0 in quarter 1, columns 1 in quarter 2,
// rows 1 in quarter 3, L1, L2 and L3 loads of a wave.  So everything is asked for a step
// and a half before it is read, and each wait leaves the loads of a step and more in
// flight.  LEFT0: how many of quarter 3's loads (or 2's and 3's) the first quarter does
// not need; LEFT1: the second; the third needs all.
template <int L1, int L2, int L3, int LEFT0, int LEFT1, class ReadA, class ReadB, class Multiply, class Load>
__device__ __forceinline__ void run_steps(int steps, const ReadA& read_a, const ReadB& read_b,
                                          const Multiply& multiply, const Load& load) {
    constexpr std::integral_constant<int, 0> q0{};
    constexpr std::integral_constant<int, 1> q1{};
    constexpr std::integral_constant<int, 2> q2{};
    constexpr std::integral_constant<int, 3> q3{};
    constexpr int STEP = L1 + L2 + L3;
    const bool late = uniform(threadIdx.x / kWave) >= 4;
    if (steps == 0) return;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        load(q1, s, s);
        load(q2, s, s);
        load(q3, s, s);
    }
    loads_done<LEFT0 + STEP>();
    reads_done();  // scale bytes that this wave wrote and others read
    meet();
    if (late) meet();
    const auto quarter = [&](auto ha, auto hb) {
        meet();
        __builtin_amdgcn_s_setprio(1);
        multiply(ha, hb);
        __builtin_amdgcn_s_setprio(0);
        meet();
    };
    for (int step = 0; step < steps; ++step) {
        const int buf = step % 2;
        read_a(q0, buf);
        read_b(q0, buf);
        loads_done<LEFT1 + STEP>();
        reads_done();
        quarter(q0, q0);
        read_b(q1, buf);
        load(q1, step + 2, buf);
        loads_done<STEP + L1>();
        reads_done();
        quarter(q0, q1);
        read_a(q1, buf);
        load(q2, step + 2, buf);
        reads_done();
        quarter(q1, q1);
        load(q3, step + 2, buf);
        loads_done<LEFT0 + STEP>();
        quarter(q1, q0);
    }
    if (!late) meet();
    loads_done<0>();  // none may land in the next workgroup's LDS
}

// The steps of a tile of few rows, whose quarters would be a few instructions between
// barriers: STAGES buffers by turns, one barrier a step, all waves abreast.  load(step,
// buffer) issues the LOADS loads of a wave of a step, also behind the last (zeros then).
template <int STAGES, int LOADS, class Compute, class Load>
__device__ __forceinline__ void run_short_steps(int steps, const Compute& compute, const Load& load) {
    if (steps == 0) return;
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) load(s, s);
    int buf = 0;
    for (int step = 0; step < steps; ++step) {
        loads_done<(STAGES - 2) * LOADS>();
        reads_done();  // of the step before, whose buffer is the one that is loaded now
        meet();
        load(step + STAGES - 1, buf == 0 ? STAGES - 1 : buf - 1);
        compute(buf);
        buf = buf + 1 == STAGES ? 0 : buf + 1;
    }
    loads_done<0>();  // none may land in the next workgroup's LDS
}

// The sum of a value over the four 16-lane rows, in every lane.
__device__ __forceinline__ uint32_t across_rows(uint32_t v) {
    const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = apply<Op::FAdd>(p[0], p[1]);
    const auto q = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return apply<Op::FAdd>(q[0], q[1]);
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

// The 16 rows by 4 pieces of a wave's pair_values(), a piece a lane, as memory wants
// them: lane l has piece l % 4 of row l / 4 (line_row(), line_column()), so that the four
// lanes of a quad stay inside a line.  Left where they are, with neighbouring lanes in different
// rows, each store or load of a wave holds the CU's address path for 64 clocks, not 16
// (weight gradients of 128 experts, 1536 x 2048: 367 us, 355 so in the same run; fp32, skewed: 376
// and 362.  fp32's two stores of a lane leave every other 16 bytes of a line to each other.)
__device__ __forceinline__ int line_row() { return (int)(threadIdx.x % kWave) / 4; }
__device__ __forceinline__ int line_column() { return (int)(threadIdx.x % 4) * 8; }
__device__ __forceinline__ uint32_t from_lane(uint32_t v, int lane) {
    return (uint32_t)__builtin_amdgcn_ds_bpermute(lane * 4, (int)v);
}
__device__ __forceinline__ int line_source() {
    const int lane = (int)(threadIdx.x % kWave);
    return (lane % 2 * 2 + lane % 4 / 2) * 16 + lane / 4;
}
__device__ __forceinline__ u32x4 to_lines(const u32x4& v) {
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = from_lane(v[i], line_source());
    return r;
}
__device__ __forceinline__ void to_lines(float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = __builtin_bit_cast(float, from_lane(__builtin_bit_cast(uint32_t, v[i]), line_source()));
}
// And back.
__device__ __forceinline__ u32x4 from_lines(const u32x4& v) {
    const int lane = (int)(threadIdx.x % kWave), q = lane / 16;
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = from_lane(v[i], lane % 16 * 4 + q % 2 * 2 + q / 2);
    return r;
}

// ---------------------------------------------------------------- epilogue
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
__device__ __forceinline__ void store(uint16_t* p, const u32x4& v) { *reinterpret_cast<u32x4*>(p) = v; }

constexpr int kCus = 256;
// Workgroups for so many tiles: whole turns of find_tile's.
inline uint32_t grouped_grid(int64_t tiles) { return (uint32_t)((tiles + 8 * kRun - 1) / (8 * kRun) * (8 * kRun)); }

}  // namespace moe
