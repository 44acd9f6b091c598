// moe_decode_layer, moe_decode_layer_mxfp4 on gfx950: the whole
// Mixture-of-Experts layer for T <= 64 tokens in two launches.
//
//   1  top-k routing; act[p, :] = bf16(silu(g) u), (g | u) = Wgu[e] x[t]
//   2  y[p, :] = Wd[e] act[p, :];  out[t, :] = bf16(sum_j w[t,j] y[p(t,j), :])
//
// p numbers the (expert, token) pairs by expert, then token.  Bound by the
// stream of the picked experts' weights, each read once: a few tokens per
// expert are far too little arithmetic to matter, so every kernel is built
// round loads in flight, with the products on the matrix cores (mfma_rows.h).
//
// Launch 1.  No workgroup waits for another, so each recomputes the routing in
// LDS (as the one-launch dispatch does) and then walks its share of the items
// (expert, 16 gate rows and their 16 up rows).  The eight waves of a workgroup
// split K, so even one token's few experts keep the whole chip loading; their
// partial sums meet in LDS, where gate and up of one output lie side by side
// for the SwiGLU.  act is rounded to bf16 there, the operand type of the second
// product.  Workgroup 0 writes the ids, the weights and the tables that launch
// 2 reads.
//
// Launch 2.  A workgroup owns a few output columns (4 rows of w_down, 8 with
// MXFP4) for every token, so the sum over experts needs no atomics and no third
// launch.  Its waves deal the active experts, and split K when there are few.
// fp32 y meets in LDS and is summed over j in order, so the same call always
// gives the same bits.
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

// Front of the workspace, written by launch 1 for launch 2.
struct Tables {
    int32_t n;                  // active experts
    int32_t expert[kEMax];      // in ascending order
    int32_t first[kEMax + 1];   // first p of each; first[n] = number of pairs
    int32_t dest[kMaxSlots];    // p of slot t*k + j
};
static_assert(sizeof(Tables) <= kDecodeLayerTableBytes, "tables outgrow their part of the workspace");

__device__ __forceinline__ float silu_mul(float g, float u) {
    // g / (1 + e^-g) * u; for g << 0 the exponential is inf and the quotient -0
    const float e = __builtin_amdgcn_exp2f(-g * 1.4426950408889634f);
    return g * __builtin_amdgcn_rcpf(1.0f + e) * u;
}

// Row tiles of an item: 16 gate rows, then their 16 up rows, 4 to a tile.
constexpr int kItemTiles = 8;

// One wave's sums of an item: [row tile][row of the tile * 4 + column].
template <int NT>
using ItemSums = float[NT][kItemTiles][16];

// Columns c0 .. c0 + 4 NT - 1 of an item.  `flip` alternates between the two
// halves of `sums`, so one barrier an item is enough: a wave that writes the
// half used two items ago has passed the barrier after it was read.
template <class W, int NT>
__device__ __forceinline__ void gate_up_item(const uint8_t* x, int H, const uint8_t* w, const uint8_t* sc, int I,
                                             uint32_t e, uint32_t i0, unsigned long long mask, int m, int c0,
                                             uint32_t p0, uint16_t* __restrict__ act, ItemSums<NT>* sums) {
    const int lane = (int)(threadIdx.x % kWave);
    const int wave = wave_index();
    const size_t first = (size_t)e * 2 * I + i0;
    const WeightBase gate{w + uniform_offset(first * W::row_bytes(H)), sc + uniform_offset(first * W::row_scales(H))};
    const WeightBase up{gate.w + (size_t)I * W::row_bytes(H), gate.scales + (size_t)I * W::row_scales(H)};
    WeightBase base[kItemTiles];
    uint32_t row[kItemTiles], col[NT];
#pragma unroll
    for (int r = 0; r < kItemTiles; ++r) {
        base[r] = r < kItemTiles / 2 ? gate : up;
        row[r] = min((uint32_t)(r % (kItemTiles / 2) * 4 + lane % 16 / 4), (uint32_t)I - 1 - i0);
    }
#pragma unroll
    for (int c = 0; c < NT; ++c)
        col[c] = (uint32_t)select_bit(mask, min(c0 + c * 4 + lane % 16 / 4, m - 1)) * (uint32_t)H * 2;
    f32x4 acc[kItemTiles][NT];
#pragma unroll
    for (int r = 0; r < kItemTiles; ++r)
#pragma unroll
        for (int c = 0; c < NT; ++c) acc[r][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int steps = (H + kStep - 1) / kStep;
    multiply_rows<W, kItemTiles, NT, (NT == 1 ? 2 : 1)>(base, row, x, col, H, steps * wave / kWaves, steps * (wave + 1) / kWaves, acc);
#pragma unroll
    for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int r = 0; r < kItemTiles; ++r) {
            const float v = diagonal_sum(acc[r][c]);
            if (lane % 4 == r % 4) sums[wave][c][r][lane / 16 * 4 + lane % 16 / 4] = v;
        }
    __syncthreads();
    for (int o = (int)threadIdx.x; o < NT * 64; o += kThreads) {
        const int c = o / 64, r = o / 16 % 4, at = o % 16;
        float g = 0.0f, u = 0.0f;
#pragma unroll
        for (int k = 0; k < kWaves; ++k) {
            g += sums[k][c][r][at];
            u += sums[k][c][r + kItemTiles / 2][at];
        }
        const int column = c0 + c * 4 + at % 4;
        const uint32_t i = i0 + r * 4 + at / 4;
        if (column < m && i < (uint32_t)I)
            act[(size_t)(p0 + column) * I + i] = (uint16_t)(pack_bf16x2(silu_mul(g, u), 0.0f) & 0xFFFFu);
    }
}

template <class W, int G, int V>
__global__ __launch_bounds__(kThreads, 4) void decode_gate_up_kernel(
    const float* __restrict__ logits, const float* __restrict__ bias, int T, int E, int k,
    const uint16_t* __restrict__ x, int H, const uint8_t* __restrict__ w, const uint8_t* __restrict__ sc, int I,
    int32_t* __restrict__ topk_ids, float* __restrict__ topk_weights, Tables* __restrict__ tables,
    uint16_t* __restrict__ act) {
    constexpr int TOK_PER_PASS = kThreads / G;
    __shared__ int32_t s_ids[kMaxSlots];
    __shared__ unsigned long long s_mask[kEMax];  // bit t: token t picked the expert
    __shared__ int32_t s_expert[kEMax];
    __shared__ int32_t s_first[kEMax + 1];
    __shared__ int32_t s_off[kEMax];  // first p by expert
    __shared__ int32_t s_n;
    __shared__ float s_sums[2][kWaves * 2 * kItemTiles * 16];  // two halves for up to 2 column tiles

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
    if (wave == 0) {  // the active experts, and the first p of each
        int n = 0, run = 0;
        for (int e0 = 0; e0 < E; e0 += kWave) {
            const int e = e0 + lane;
            const int cnt = e < E ? __popcll(s_mask[e]) : 0;
            const unsigned long long some = __ballot(cnt > 0);
            const int incl = wave_inclusive_sum(cnt);
            const int at = n + __popcll(some & ((1ull << lane) - 1ull));
            if (cnt > 0) {
                s_expert[at] = e;
                s_first[at] = run + incl - cnt;
                s_off[e] = run + incl - cnt;
            }
            n += __popcll(some);
            run += __builtin_amdgcn_readlane(incl, kWave - 1);
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
            if (a < n) tables->expert[a] = s_expert[a];
            tables->first[a] = s_first[a];
        }
        for (int s = (int)threadIdx.x; s < T * k; s += kThreads) {
            const int e = s_ids[s];
            tables->dest[s] = s_off[e] + __popcll(s_mask[e] & ((1ull << (s / k)) - 1ull));
        }
    }
    const int tiles = (I + 15) / 16;
    int half = 0;
    for (int it = (int)blockIdx.x; it < n * tiles; it += (int)gridDim.x) {
        const int a = it / tiles;
        const uint32_t e = uniform((uint32_t)s_expert[a]);
        const unsigned long long mask = s_mask[e];
        const int m = (int)uniform((uint32_t)__popcll(mask));
        const uint32_t i0 = (uint32_t)(it - a * tiles) * 16;
        const uint32_t p0 = uniform((uint32_t)s_first[a]);
        const uint8_t* xb = reinterpret_cast<const uint8_t*>(x);
        for (int c0 = 0; c0 < m; c0 += 8) {
            if (m - c0 <= 4)
                gate_up_item<W, 1>(xb, H, w, sc, I, e, i0, mask, m, c0, p0, act,
                                   reinterpret_cast<ItemSums<1>*>(s_sums[half]));
            else
                gate_up_item<W, 2>(xb, H, w, sc, I, e, i0, mask, m, c0, p0, act,
                                   reinterpret_cast<ItemSums<2>*>(s_sums[half]));
            half ^= 1;
        }
    }
}

// Output columns of a workgroup of launch 2, in tiles of 4 rows of w_down.
template <class W>
constexpr int kDownTiles = 1;
template <>
constexpr int kDownTiles<Mxfp4Weights> = 2;

constexpr int kMaxY = kMaxSlots;  // y entries of a workgroup: pairs times K parts

// K parts of an expert's rows: enough that the eight waves have two tasks each,
// as long as y holds them.  One part always fits: there are at most kMaxSlots
// pairs.
__device__ __forceinline__ int k_parts(int n, int pairs) {
    int parts = 8;
    while (parts > 1 && (n * parts > 16 || pairs * parts > kMaxY)) parts /= 2;
    return parts;
}

template <class W, int NT>
__device__ __forceinline__ void down_columns(const WeightBase& rows, int left, const uint8_t* act, int I, int p0,
                                             int end, int s0, int s1, float* y) {
    constexpr int RT = kDownTiles<W>;
    const int lane = (int)(threadIdx.x % kWave);
    WeightBase base[RT];
    uint32_t row[RT], col[NT];
    f32x4 acc[RT][NT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        base[r] = rows;
        row[r] = (uint32_t)min(r * 4 + lane % 16 / 4, left - 1);
#pragma unroll
        for (int c = 0; c < NT; ++c) acc[r][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
#pragma unroll
    for (int c = 0; c < NT; ++c) col[c] = (uint32_t)min(p0 + c * 4 + lane % 16 / 4, end - 1) * (uint32_t)I * 2;
    multiply_rows<W, RT, NT, 4>(base, row, act, col, I, s0, s1, acc);
#pragma unroll
    for (int c = 0; c < NT; ++c) {
        const int p = p0 + c * 4 + lane % 16 / 4;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const float v = diagonal_sum(acc[r][c]);
            if (lane % 4 == r && p < end) y[p * (4 * RT) + r * 4 + lane / 16] = v;
        }
    }
}

template <class W>
__global__ __launch_bounds__(kThreads) void decode_down_kernel(int T, int k, const uint8_t* __restrict__ w,
                                                               const uint8_t* __restrict__ sc, int H, int I,
                                                               const Tables* __restrict__ tables,
                                                               const uint16_t* __restrict__ act,
                                                               const float* __restrict__ topk_weights,
                                                               uint16_t* __restrict__ out) {
    constexpr int ROWS = 4 * kDownTiles<W>;
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
    const int steps = (I + kStep - 1) / kStep;
    const uint8_t* actb = reinterpret_cast<const uint8_t*>(act);
    for (int task = wave; task < n * parts; task += kWaves) {
        const int a = task / parts, part = task - a * parts;
        const size_t row = (size_t)tables->expert[a] * H + h0;
        const WeightBase rows{w + uniform_offset(row * W::row_bytes(I)), sc + uniform_offset(row * W::row_scales(I))};
        const int begin = tables->first[a], end = tables->first[a + 1];
        const int s0 = steps * part / parts, s1 = steps * (part + 1) / parts;
        float* y = s_y + part * pairs * ROWS;
        for (int p0 = begin; p0 < end; p0 += 8) {
            if (end - p0 <= 4)
                down_columns<W, 1>(rows, H - h0, actb, I, p0, end, s0, s1, y);
            else
                down_columns<W, 2>(rows, H - h0, actb, I, p0, end, s0, s1, y);
        }
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
        if (h0 + h < H) out[(size_t)t * H + h0 + h] = (uint16_t)(pack_bf16x2(sum, 0.0f) & 0xFFFFu);
    }
}

constexpr int kMaxGrid = 512;  // two workgroups per CU

template <class W, int G, int V>
hipError_t launch_gv(const DecodeLayerArgs& a, hipStream_t stream) {
    Tables* tables = static_cast<Tables*>(a.workspace);
    uint16_t* act = reinterpret_cast<uint16_t*>(static_cast<char*>(a.workspace) + kDecodeLayerTableBytes);
    const uint16_t* x = static_cast<const uint16_t*>(a.x);
    const int64_t most = (int64_t)(a.E < a.T * a.k ? a.E : a.T * a.k) * ((a.I + 15) / 16);
    const int grid = (int)(most < kMaxGrid ? most : kMaxGrid);
    decode_gate_up_kernel<W, G, V><<<grid, kThreads, 0, stream>>>(
        a.logits, a.bias, a.T, a.E, a.k, x, a.H, static_cast<const uint8_t*>(a.w_gate_up), a.s_gate_up, a.I,
        a.topk_ids, a.topk_weights, tables, act);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    decode_down_kernel<W><<<(a.H + 4 * kDownTiles<W> - 1) / (4 * kDownTiles<W>), kThreads, 0, stream>>>(
        a.T, a.k, static_cast<const uint8_t*>(a.w_down), a.s_down, a.H, a.I, tables, act, a.topk_weights,
        static_cast<uint16_t*>(a.out));
    return hipGetLastError();
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
