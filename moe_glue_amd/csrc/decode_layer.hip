// moe_decode_layer, moe_decode_layer_mxfp4 on gfx950: the whole
// Mixture-of-Experts layer for T <= 64 tokens in two launches.
//
//   1  top-k routing; act[p, :] = bf16(silu(g) u), (g | u) = Wgu[e] x[t]
//   2  y[p, :] = Wd[e] act[p, :];  out[t, :] = bf16(sum_j w[t,j] y[p(t,j), :])
//
// p numbers the (expert, token) pairs by expert, then token.  Bound by the
// stream of the picked experts' weights, each read once for every entry (16 or 8 of
// an expert's tokens): a few tokens per expert are far too little arithmetic to
// matter, so every kernel is built round loads in flight, with the products on the
// matrix cores (mfma_rows.h).
//
// Launch 1.  No workgroup waits for another, so each recomputes the routing in
// LDS (as the one-launch dispatch does; about 4 us) and then walks its share of
// the row quads: 4 gate rows and their 4 up rows of an expert, whose products with
// one token a lane holds together for the SwiGLU.  In whole rounds of the grid a
// wave has all of K to itself, and no barrier; what is left over, all there is
// with one token, is split along K between the waves and meets in LDS.  act is
// rounded to bf16, the operand type of the second product.  Workgroup 0 writes the
// ids, the weights and the tables that launch 2 reads.
//
// Launch 2.  A workgroup owns a few output columns for every token, so the sum
// over experts needs no atomics and no third launch.  Its waves deal the entries,
// and split K when there are few.  fp32 y meets in LDS and is summed over j in
// order, so the same call always gives the same bits.
//
// Measured (us, launch 1 + launch 2, medians of 27 dispatches under rocprofv3's
// kernel trace, of several runs; the weights read at the rate of a large streaming
// read, 6.7 TB/s, in brackets): one token, 128 experts of 2048 x 768, bf16, 13.6 to
// 14.5 + 6.8 to 7.3 (11.3 together), MXFP4 11.2 + 7.9 (3.0); 32 tokens, bf16, 119 to
// 120 + 60 (155), MXFP4 43 + 35 (42); 8 tokens, some 42 of 64 experts of 7168 x 2048,
// bf16, 366 + 180 (550); of 256 such experts, MXFP4, one token 29.6 + 21.1 (28), 16
// tokens 234 to 239 + 128 to 132 (285); 61 tokens, skewed, 64 experts of 4096 x 1408,
// MXFP4, 87 to 90 + 52 to 53 (47; here the columns' loads and the products count too).
#include "kernels.h"
#include "mfma_rows.h"
#include "route_common.h"

namespace moe {
namespace {

using namespace route_detail;

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / kWave;
constexpr int kMaxTokens = kDecodeLayerMaxTokens;
static_assert(kMaxTokens <= 64, "one bitmap word per expert");
constexpr int kMaxSlots = kMaxTokens * kKMax;

// The work is dealt in entries: an active expert with up to kEntryTokens of its
// tokens (an expert with more has several, next to each other), so that entries
// cost about the same however the router's choices are spread.
template <class W>
constexpr int kEntryTokens = 16;
template <>
constexpr int kEntryTokens<Mxfp4Weights> = 8;  // by registers, see mfma_rows.h
constexpr int kMaxEntries = kEMax + kMaxSlots / 8;
// Weights are streamed past the caches (decode workload 132 -> 120 and 65 -> 60
// us, DeepSeek-V3-shaped MXFP4 247 -> 234 and 134 -> 129), except under entries
// as wide as they come: the expert may have another, which reads them again
// (skewed MXFP4 98 -> 86 and 55 -> 52).
template <class W, int NT>
constexpr int kWeightCache = NT * 4 < kEntryTokens<W> ? kCacheNt : 0;

// Front of the workspace, written by launch 1 for launch 2.
struct Tables {
    int32_t n;                       // entries
    int32_t expert[kMaxEntries];     // in ascending order
    int32_t first[kMaxEntries + 1];  // first p of each; first[n] = number of pairs
    int32_t dest[kMaxSlots];         // p of slot t*k + j
};
static_assert(sizeof(Tables) <= kDecodeLayerTableBytes, "tables outgrow their part of the workspace");

__device__ __forceinline__ float silu_mul(float g, float u) {
    // g / (1 + e^-g) * u; for g << 0 the exponential is inf and the quotient -0
    const float e = __builtin_amdgcn_exp2f(-g * 1.4426950408889634f);
    return g * __builtin_amdgcn_rcpf(1.0f + e) * u;
}

// Row quads (4 gate rows and their 4 up rows) that a wave multiplies together
// where it has K to itself: with MXFP4 a column's loads cost as much as four
// row tiles', so two quads share them.
template <class W>
constexpr int kWaveQuads = 1;
template <>
constexpr int kWaveQuads<Mxfp4Weights> = 2;
// Steps of loads in flight for a task of RT row and NT column tiles.
template <class W, int RT, int NT>
constexpr int kInFlight = NT <= 2 ? 4 : 2;
template <int RT, int NT>
constexpr int kInFlight<Mxfp4Weights, RT, NT> = NT == 1 ? 4 : 2;

// Where a task's rows and tokens are: row quad `quad` (4 gate rows and their 4
// up rows) of expert e; of its tokens, the set bits of mask, m from number c0
// on; and their rows p0, p0 + 1, .. of act.
struct GateUpTask {
    uint32_t e, quad, p0;
    int c0, m;
    unsigned long long mask;
};

// g, u: the products of QT row quads with the task's tokens over the steps
// [s0, s1), row l / 16 and column l % 16 / 4 of each tile in lane l.
template <class W, int QT, int NT>
__device__ __forceinline__ void gate_up_product(const GateUpTask& t, __amdgpu_buffer_rsrc_t x, int H, const uint8_t* w,
                                                const uint8_t* sc, int I, int s0, int s1, float (&g)[QT][NT],
                                                float (&u)[QT][NT]) {
    const int lane = (int)(threadIdx.x % kWave);
    const size_t first = (size_t)t.e * 2 * I + t.quad * 4;
    const uint32_t row_bytes = W::bytes_of((uint32_t)H), row_scales = W::row_scales(H);
    const uint8_t* gate = w + uniform_offset(first * row_bytes);
    const uint8_t* gate_scales = sc + uniform_offset(first * row_scales);
    // tile 2 q: the gate rows of quad q, tile 2 q + 1: its up rows
    RowTiles<2 * QT> rows;
    uint32_t col[1][NT];
    f32x4 acc[2 * QT][NT];
#pragma unroll
    for (int r = 0; r < 2 * QT; ++r) {
        rows.at[r] = (uint32_t)(r / 2 * 4) * row_bytes;
        rows.scales[r] = gate_scales + ((size_t)(r % 2) * I + r / 2 * 4) * row_scales;
        rows.last[r] = 3;
#pragma unroll
        for (int c = 0; c < NT; ++c) acc[r][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
#pragma unroll
    for (int c = 0; c < NT; ++c) {
        const int column = c * 4 + lane % 16 / 4;
        col[0][c] = column < t.m ? (uint32_t)select_bit(t.mask, t.c0 + column) * (uint32_t)H * 2 : kNowhere;
    }
    multiply_rows<W, 2 * QT, NT, kInFlight<W, 2 * QT, NT>, kWeightCache<W, NT>, 1>(
        buffer_of(gate, (size_t)(4 * QT) * row_bytes),
        buffer_of(gate + (size_t)I * row_bytes, (size_t)(4 * QT) * row_bytes), rows, x, col, H, s0, s1, acc);
#pragma unroll
    for (int q = 0; q < QT; ++q)
#pragma unroll
        for (int c = 0; c < NT; ++c) {
            g[q][c] = diagonal_sum(acc[2 * q][c]);
            u[q][c] = diagonal_sum(acc[2 * q + 1][c]);
        }
}

__device__ __forceinline__ uint16_t swiglu_bf16(float g, float u) {
    return (uint16_t)(pack_bf16x2(silu_mul(g, u), 0.0f) & 0xFFFFu);
}

// All of K by one wave: the outputs go straight to act.
template <class W, int QT, int NT>
__device__ __forceinline__ void gate_up_whole(const GateUpTask& t, __amdgpu_buffer_rsrc_t x, int H, const uint8_t* w,
                                              const uint8_t* sc, int I, uint16_t* __restrict__ act) {
    float g[QT][NT], u[QT][NT];
    gate_up_product<W, QT, NT>(t, x, H, w, sc, I, 0, steps_of<W>(H), g, u);
    const int lane = (int)(threadIdx.x % kWave);
#pragma unroll
    for (int q = 0; q < QT; ++q)
#pragma unroll
        for (int c = 0; c < NT; ++c) {
            const int column = c * 4 + lane % 16 / 4;
            if (lane % 4 == (q * NT + c) % 4 && column < t.m)
                act[(size_t)(t.p0 + column) * I + (t.quad + q) * 4 + lane / 16] = swiglu_bf16(g[q][c], u[q][c]);
        }
}

// A part of K: the partial sums go to LDS, [column tile][gate, up][16].
constexpr int kPartSums = 4 * 2 * 16;

template <class W, int NT>
__device__ __forceinline__ void gate_up_part(const GateUpTask& t, __amdgpu_buffer_rsrc_t x, int H, const uint8_t* w,
                                             const uint8_t* sc, int I, int s0, int s1, float* sums) {
    float g[1][NT], u[1][NT];
    gate_up_product<W, 1, NT>(t, x, H, w, sc, I, s0, s1, g, u);
    const int lane = (int)(threadIdx.x % kWave);
    const int at = lane / 16 * 4 + lane % 16 / 4;
#pragma unroll
    for (int c = 0; c < NT; ++c) {
        if (lane % 4 == 0) sums[c * 32 + at] = g[0][c];
        if (lane % 4 == 1) sums[c * 32 + 16 + at] = u[0][c];
    }
}

template <class W, int G, int V>
__global__ __launch_bounds__(kThreads, 2) void decode_gate_up_kernel(
    const float* __restrict__ logits, const float* __restrict__ bias, int T, int E, int k,
    const uint16_t* __restrict__ x, int H, const uint8_t* __restrict__ w, const uint8_t* __restrict__ sc, int I,
    int32_t* __restrict__ topk_ids, float* __restrict__ topk_weights, Tables* __restrict__ tables,
    uint16_t* __restrict__ act) {
    constexpr int TOK_PER_PASS = kThreads / G;
    __shared__ int32_t s_ids[kMaxSlots];
    __shared__ unsigned long long s_mask[kEMax];  // bit t: token t picked the expert
    __shared__ int32_t s_entry[kMaxEntries];  // expert, and number of the entry among its own from bit 16 on
    __shared__ int32_t s_first[kMaxEntries + 1];
    __shared__ int32_t s_off[kEMax];  // first p by expert
    __shared__ int32_t s_n;
    __shared__ float s_sums[kWaves][kPartSums];

    const int lane = (int)(threadIdx.x % kWave);
    const int wave = wave_index();
    const bool writer = blockIdx.x == 0;
    for (int e = (int)threadIdx.x; e < E; e += kThreads) s_mask[e] = 0ull;
    __syncthreads();
    const int grp = (int)threadIdx.x / G, gl = (int)threadIdx.x % G;
    for (int t0 = 0; t0 < T; t0 += TOK_PER_PASS) {
        if (t0 + wave * (kWave / G) >= T) continue;  // wave-uniform: the lane exchange stays whole-wave
        const int t = t0 + grp;
        topk_token<G, V>(logits, bias, T, E, k, t, t, gl, writer ? topk_ids : nullptr, topk_weights, s_ids);
        if (t < T)
            for (int r = gl; r < k; r += G) atomicOr(&s_mask[s_ids[t * k + r]], 1ull << t);
    }
    __syncthreads();
    constexpr int TOKENS = kEntryTokens<W>;
    if (wave == 0) {  // the entries, and the first p of each
        int n = 0, run = 0;
        for (int e0 = 0; e0 < E; e0 += kWave) {
            const int e = e0 + lane;
            const int cnt = e < E ? __popcll(s_mask[e]) : 0;
            const int own = (cnt + TOKENS - 1) / TOKENS;
            const int incl = wave_inclusive_sum(cnt | own << 16);  // both counts stay below 2^16
            const int p0 = run + (incl & 0xFFFF) - cnt, at = n + (incl >> 16) - own;
            if (cnt > 0) s_off[e] = p0;
            for (int i = 0; i < own; ++i) {
                s_entry[at + i] = e | i << 16;
                s_first[at + i] = p0 + i * TOKENS;
            }
            const int total = __builtin_amdgcn_readlane(incl, kWave - 1);
            n += total >> 16;
            run += total & 0xFFFF;
        }
        if (lane == 0) {
            s_n = n;
            s_first[n] = run;
        }
    }
    __syncthreads();
    const int n = s_n;
    if (writer) {
        if (threadIdx.x == 0) tables->n = n;
        for (int a = (int)threadIdx.x; a <= n; a += kThreads) {
            if (a < n) tables->expert[a] = s_entry[a] & 0xFFFF;
            tables->first[a] = s_first[a];
        }
        for (int s = (int)threadIdx.x; s < T * k; s += kThreads) {
            const int e = s_ids[s];
            tables->dest[s] = s_off[e] + __popcll(s_mask[e] & ((1ull << (s / k)) - 1ull));
        }
    }
    const uint32_t per = (uint32_t)I / 4;  // row quads of an expert
    const uint32_t all = uniform((uint32_t)n) * per;
    const __amdgpu_buffer_rsrc_t xb = buffer_of(x, (size_t)T * H * 2);
    const auto task_of = [&](uint32_t at) {
        GateUpTask t;
        const uint32_t a = at / per;
        const uint32_t entry = uniform((uint32_t)s_entry[a]);
        t.quad = at - a * per;
        t.e = entry & 0xFFFFu;
        t.c0 = (int)(entry >> 16) * TOKENS;
        t.p0 = uniform((uint32_t)s_first[a]);
        t.m = (int)uniform((uint32_t)s_first[a + 1]) - (int)t.p0;
        t.mask = s_mask[t.e];
        return t;
    };
    // whole rounds of the grid, QT quads a wave (I / 4 is a multiple of QT: a
    // wave's quads are one expert's).  Neighbouring workgroups take neighbouring
    // rows, so that the rows of an expert with many tokens, which take longer,
    // are spread over all of them.
    constexpr uint32_t QT = kWaveQuads<W>;
    const uint32_t round = gridDim.x * kWaves * QT;
    const uint32_t whole = all / round * round;
    for (uint32_t at = (blockIdx.x * kWaves + (uint32_t)wave) * QT; at < whole; at += round) {
        const GateUpTask t = task_of(at);
        if (t.m <= 4)
            gate_up_whole<W, QT, 1>(t, xb, H, w, sc, I, act);
        else if (t.m <= 8 || TOKENS == 8)
            gate_up_whole<W, QT, 2>(t, xb, H, w, sc, I, act);
        else if constexpr (TOKENS == 16)
            gate_up_whole<W, QT, 4>(t, xb, H, w, sc, I, act);
    }
    // this workgroup's share of the quads that are left, eight or fewer at a
    // time: `parts` waves split the K of each, and meet in LDS
    const int steps = steps_of<W>(H);
    const uint32_t begin = whole + (uint32_t)((uint64_t)(all - whole) * blockIdx.x / gridDim.x);
    const uint32_t left = whole + (uint32_t)((uint64_t)(all - whole) * (blockIdx.x + 1) / gridDim.x) - begin;
    for (uint32_t done = 0; done < left; done += kWaves) {
        const uint32_t now = min(left - done, (uint32_t)kWaves);
        int parts = kWaves;
        while (parts * now > kWaves) parts /= 2;
        const uint32_t mine = done + (uint32_t)(wave / parts);
        const int part = wave % parts;
        const bool busy = mine < done + now;  // uniform
        GateUpTask t{};
        if (busy) {
            t = task_of(begin + mine);
            const int s0 = steps * part / parts, s1 = steps * (part + 1) / parts;
            if (t.m <= 4)
                gate_up_part<W, 1>(t, xb, H, w, sc, I, s0, s1, s_sums[wave]);
            else if (t.m <= 8 || TOKENS == 8)
                gate_up_part<W, 2>(t, xb, H, w, sc, I, s0, s1, s_sums[wave]);
            else if constexpr (TOKENS == 16)
                gate_up_part<W, 4>(t, xb, H, w, sc, I, s0, s1, s_sums[wave]);
        }
        __syncthreads();
        const int column = lane / 16 * 4 + lane % 4;
        if (busy && part == 0 && column < t.m) {
            const int at = lane / 16 * 32 + lane % 16;
            float g = 0.0f, u = 0.0f;
            for (int k = 0; k < parts; ++k) {
                g += s_sums[wave + k][at];
                u += s_sums[wave + k][at + 16];
            }
            act[(size_t)(t.p0 + column) * I + t.quad * 4 + lane % 16 / 4] = swiglu_bf16(g, u);
        }
        __syncthreads();
    }
}

// Steps of loads in flight for RT row and NT column tiles.
template <class W, int RT, int NT>
constexpr int kDownInFlight = NT == 1 ? 8 : NT == 2 ? 4 : 2;
template <int RT, int NT>
constexpr int kDownInFlight<Mxfp4Weights, RT, NT> = NT == 1 || RT == 4 ? 4 : 2;

constexpr int kMaxY = kMaxSlots;  // y entries of a workgroup: pairs times K parts

// K parts of an entry's rows: enough that the eight waves have two tasks each,
// as long as y holds them.  One part always fits: there are at most kMaxSlots
// pairs.
__device__ __forceinline__ int k_parts(int n, int pairs) {
    int parts = 8;
    while (parts > 1 && (n * parts > 16 || pairs * parts > kMaxY)) parts /= 2;
    return parts;
}

// What a task of launch 2 multiplies: the rows of w_down from w on by the act
// rows p0 to end - 1.
struct DownTask {
    const uint8_t* w;
    const uint8_t* scales;
    int p0, end;
};

// G tasks side by side (G = 1, or 2 with the same s0 and s1), RT row tiles each.
template <class W, int RT, int NT, int G>
__device__ __forceinline__ void down_columns(const DownTask (&t)[G], __amdgpu_buffer_rsrc_t act, int I, int s0,
                                             int s1, float* y) {
    const int lane = (int)(threadIdx.x % kWave);
    const uint32_t row_bytes = W::bytes_of((uint32_t)I), row_scales = W::row_scales(I);
    RowTiles<RT * G> rows;  // tile r * G + g: row tile r of task g
    uint32_t col[G][NT];
    f32x4 acc[RT * G][NT];
#pragma unroll
    for (int r = 0; r < RT * G; ++r) {
        rows.at[r] = (uint32_t)(r / G * 4) * row_bytes;
        rows.scales[r] = t[r % G].scales + (size_t)(r / G * 4) * row_scales;
        rows.last[r] = 3;
#pragma unroll
        for (int c = 0; c < NT; ++c) acc[r][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int c = 0; c < NT; ++c) {
            const int p = t[g].p0 + c * 4 + lane % 16 / 4;
            col[g][c] = p < t[g].end ? (uint32_t)p * (uint32_t)I * 2 : kNowhere;
        }
    const size_t bytes = (size_t)(4 * RT) * row_bytes;
    multiply_rows<W, RT * G, NT, kDownInFlight<W, RT, NT * G>, kWeightCache<W, NT>, G>(
        buffer_of(t[0].w, bytes), buffer_of(t[G - 1].w, bytes), rows, act, col, I, s0, s1, acc);
#pragma unroll
    for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int r = 0; r < RT * G; ++r) {
            const int p = t[r % G].p0 + c * 4 + lane % 16 / 4;
            const float v = diagonal_sum(acc[r][c]);
            if (lane % 4 == r % 4 && p < t[r % G].end) y[p * (4 * RT) + r / G * 4 + lane / 16] = v;
        }
}

// RT tiles of 4 output columns a workgroup; H is a multiple of 4 RT.
template <class W, int RT, bool PAIRS>
__global__ __launch_bounds__(kThreads) void decode_down_kernel(int T, int k, const uint8_t* __restrict__ w,
                                                               const uint8_t* __restrict__ sc, int H, int I,
                                                               const Tables* __restrict__ tables,
                                                               const uint16_t* __restrict__ act,
                                                               const float* __restrict__ topk_weights,
                                                               uint16_t* __restrict__ out) {
    constexpr int ROWS = 4 * RT;
    __shared__ float s_y[kMaxY * ROWS];  // [part][p][row]
    __shared__ float s_w[kMaxSlots];
    __shared__ int32_t s_dest[kMaxSlots];
    const int wave = wave_index();
    const int h0 = (int)blockIdx.x * ROWS;
    const int n = tables->n;
    const int pairs = tables->first[n];
    for (int s = (int)threadIdx.x; s < T * k; s += kThreads) {
        s_w[s] = topk_weights[s];
        s_dest[s] = tables->dest[s];
    }
    const int parts = k_parts(n, pairs);
    const int steps = steps_of<W>(I);
    const __amdgpu_buffer_rsrc_t actb = buffer_of(act, (size_t)pairs * I * 2);
    const auto task_of = [&](int a) {
        const size_t row = (size_t)tables->expert[a] * H + h0;
        return DownTask{w + uniform_offset(row * W::bytes_of((uint32_t)I)),
                        sc + uniform_offset(row * W::row_scales(I)), tables->first[a], tables->first[a + 1]};
    };
    for (int task = wave; task < n * parts; task += kWaves) {
        const int a = task / parts, part = task - a * parts;
        const DownTask t[1] = {task_of(a)};
        // two small entries at a time: a wave with short rows would wait out the
        // memory's latency after every few loads (MXFP4, 32 tokens, 2048 x 768 38.0
        // -> 34.2 us, 1024 x 2048 45 -> 40; not for bf16 rows, 60 -> 63 us)
        if (PAIRS && parts == 1 && task + kWaves < n && t[0].end - t[0].p0 <= 4) {
            const DownTask two[2] = {t[0], task_of(task + kWaves)};
            if (two[1].end - two[1].p0 <= 4) {
                down_columns<W, RT, 1, 2>(two, actb, I, 0, steps, s_y);
                task += kWaves;
                continue;
            }
        }
        const int m = t[0].end - t[0].p0;
        const int s0 = steps * part / parts, s1 = steps * (part + 1) / parts;
        float* y = s_y + part * pairs * ROWS;
        if (m <= 4)
            down_columns<W, RT, 1, 1>(t, actb, I, s0, s1, y);
        else if (m <= 8 || kEntryTokens<W> == 8)
            down_columns<W, RT, 2, 1>(t, actb, I, s0, s1, y);
        else if constexpr (kEntryTokens<W> == 16)
            down_columns<W, RT, 4, 1>(t, actb, I, s0, s1, y);
    }
    __syncthreads();
    for (int i = (int)threadIdx.x; i < T * ROWS; i += kThreads) {
        const int t = i / ROWS, h = i % ROWS;
        float sum = 0.0f;
        for (int j = 0; j < k; ++j) {
            const int s = t * k + j;
            float y = 0.0f;
            for (int part = 0; part < parts; ++part) y += s_y[(part * pairs + s_dest[s]) * ROWS + h];
            sum = fmaf(s_w[s], y, sum);
        }
        out[(size_t)t * H + h0 + h] = (uint16_t)(pack_bf16x2(sum, 0.0f) & 0xFFFFu);
    }
}

// From this width on MXFP4's launch 2 takes 16 columns a workgroup instead of 4:
// four row tiles share a column's loads, which cost more than theirs.  Below, too
// few workgroups would be left.  One against the other (us): H = 2048 53 / 38,
// 1024 74 / 45, 3584 33 / 39, 4096 55 / 67, 7168 130 / 146 (the last three against
// 8 columns).  With bf16 weights 8 columns against 4 changes nothing either way.
constexpr int kWideDown = 3584;

// One workgroup per CU, its 8 waves with up to 256 registers each.  Two of half
// the registers: decode workload 120 -> 135 us, DeepSeek-V3-shaped MXFP4, which
// then spills, 234 -> 316 us.
constexpr int kMaxGrid = 256;

template <class W, int G, int V>
hipError_t launch_gv(const DecodeLayerArgs& a, hipStream_t stream) {
    Tables* tables = static_cast<Tables*>(a.workspace);
    uint16_t* act = reinterpret_cast<uint16_t*>(static_cast<char*>(a.workspace) + kDecodeLayerTableBytes);
    const uint16_t* x = static_cast<const uint16_t*>(a.x);
    const int64_t quads = (int64_t)(a.E < a.T * a.k ? a.E : a.T * a.k) * (a.I / 4);  // at most
    const int grid = (int)(quads < kMaxGrid ? quads : kMaxGrid);
    decode_gate_up_kernel<W, G, V><<<grid, kThreads, 0, stream>>>(
        a.logits, a.bias, a.T, a.E, a.k, x, a.H, static_cast<const uint8_t*>(a.w_gate_up), a.s_gate_up, a.I,
        a.topk_ids, a.topk_weights, tables, act);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const auto down = [&](auto tiles, auto pairs) {
        constexpr int RT = decltype(tiles)::value;
        decode_down_kernel<W, RT, decltype(pairs)::value><<<a.H / (4 * RT), kThreads, 0, stream>>>(
            a.T, a.k, static_cast<const uint8_t*>(a.w_down), a.s_down, a.H, a.I, tables, act, a.topk_weights,
            static_cast<uint16_t*>(a.out));
        return hipGetLastError();
    };
    if constexpr (std::is_same_v<W, Bf16Weights>)
        return down(std::integral_constant<int, 1>{}, std::false_type{});
    else if (a.H >= kWideDown)
        return down(std::integral_constant<int, 4>{}, std::false_type{});
    else
        return down(std::integral_constant<int, 1>{}, std::true_type{});
}

template <class W>
hipError_t launch_w(const DecodeLayerArgs& a, hipStream_t stream) {
    switch (route_lanes_per_token(a.E) * 16 + route_keys_per_lane(a.E)) {
        case 1 * 16 + 4: return launch_gv<W, 1, 4>(a, stream);
        case 2 * 16 + 4: return launch_gv<W, 2, 4>(a, stream);
        case 4 * 16 + 4: return launch_gv<W, 4, 4>(a, stream);
        case 8 * 16 + 4: return launch_gv<W, 8, 4>(a, stream);
        case 8 * 16 + 8: return launch_gv<W, 8, 8>(a, stream);
        case 16 * 16 + 8: return launch_gv<W, 16, 8>(a, stream);
        case 32 * 16 + 8: return launch_gv<W, 32, 8>(a, stream);
        default: return launch_gv<W, 64, 8>(a, stream);
    }
}

}  // namespace

hipError_t launch_decode_layer(const DecodeLayerArgs& a, hipStream_t stream) {
    return a.s_gate_up != nullptr ? launch_w<Mxfp4Weights>(a, stream) : launch_w<Bf16Weights>(a, stream);
}

}  // namespace moe
