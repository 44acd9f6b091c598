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
// Launch 2.  A workgroup owns 4 output columns, for every token, so the sum
// over experts needs no atomics and no third launch.  Four rows are a quarter
// of an MFMA tile: a tile takes the 4 rows of 4 experts, whose tokens are
// consecutive p, and the lane that holds column p and the quarter of its own
// expert has the 4 outputs; the other quarters are products nobody asked for.
// The waves of a workgroup deal these units, and split K when there are few.
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

template <class W>
__device__ __forceinline__ WeightRow weight_row(const uint8_t* w, const uint8_t* scales, size_t row, int K) {
    return {w + row * W::row_bytes(K), scales + row * W::row_scales(K)};
}

// Partial sums of one 16x16 tile pair: [wave][gate or up][lane].
struct GateUpShared {
    f32x4 part[kWaves][2][kWave];
};

template <class W, int NT>
__device__ __forceinline__ void gate_up_item(const uint16_t* __restrict__ x, int H, const uint8_t* __restrict__ w,
                                             const uint8_t* __restrict__ sc, int I, int e, int i0,
                                             unsigned long long mask, int m, int c0, size_t p0,
                                             uint16_t* __restrict__ act, GateUpShared& sh) {
    const int lane = (int)(threadIdx.x % kWave);
    const int wave = (int)(threadIdx.x / kWave);
    const size_t gate = (size_t)e * 2 * I + min(i0 + lane % 16, I - 1);
    const WeightRow rows[2] = {weight_row<W>(w, sc, gate, H), weight_row<W>(w, sc, gate + I, H)};
    const uint16_t* cols[NT];
#pragma unroll
    for (int c = 0; c < NT; ++c) {
        const int t = select_bit(mask, min(c0 + c * 16 + lane % 16, m - 1));
        cols[c] = x + (size_t)t * H;
    }
    f32x4 acc[2][NT];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int c = 0; c < NT; ++c) acc[r][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int steps = (H + W::STEP - 1) / W::STEP;
    multiply_rows<W, 2, NT>(rows, cols, H, steps * wave / kWaves, steps * (wave + 1) / kWaves, acc);
#pragma unroll
    for (int c = 0; c < NT; ++c) {
        __syncthreads();  // the last tile's sums are read
        sh.part[wave][0][lane] = acc[0][c];
        sh.part[wave][1][lane] = acc[1][c];
        __syncthreads();
        if (threadIdx.x < 256) {
            const int l = (int)threadIdx.x / 4, v = (int)threadIdx.x % 4;
            float g = 0.0f, u = 0.0f;
#pragma unroll
            for (int k = 0; k < kWaves; ++k) {
                g += sh.part[k][0][l][v];
                u += sh.part[k][1][l][v];
            }
            const int col = c0 + c * 16 + l % 16, i = i0 + l / 16 * 4 + v;
            if (col < m && i < I)
                act[(p0 + col) * I + i] = (uint16_t)(pack_bf16x2(silu_mul(g, u), 0.0f) & 0xFFFFu);
        }
    }
}

template <class W, int G, int V>
__global__ __launch_bounds__(kThreads) void decode_gate_up_kernel(
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
    __shared__ GateUpShared sh;

    const int lane = (int)(threadIdx.x % kWave);
    const int wave = (int)(threadIdx.x / kWave);
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
    for (int it = (int)blockIdx.x; it < n * tiles; it += (int)gridDim.x) {
        const int a = it / tiles;
        const int e = s_expert[a];
        const unsigned long long mask = s_mask[e];
        const int m = __popcll(mask);
        const int i0 = (it - a * tiles) * 16;
        const size_t p0 = (size_t)s_first[a];
        for (int c0 = 0; c0 < m; c0 += 32) {
            if (m - c0 <= 16)
                gate_up_item<W, 1>(x, H, w, sc, I, e, i0, mask, m, c0, p0, act, sh);
            else
                gate_up_item<W, 2>(x, H, w, sc, I, e, i0, mask, m, c0, p0, act, sh);
        }
    }
}

// Most y entries of a workgroup: pairs times K parts (see parts()).
constexpr int kMaxY = 3072;

// K parts of a unit (4 experts) by the number of units: enough that the eight
// waves all have work.  Up to 4 experts hold at most 256 pairs, 12 at most
// 768, and more at most 1024 (k is at most the number of active experts).
__device__ __forceinline__ int k_parts(int units) { return units >= 8 ? 1 : units >= 4 ? 2 : units >= 2 ? 4 : 8; }

template <class W, int NT>
__device__ __forceinline__ void down_columns(const WeightRow (&rows)[1], const uint16_t* __restrict__ act, int I,
                                             int p0, int lo, int hi, int end, int s0, int s1, f32x4* y) {
    const int lane = (int)(threadIdx.x % kWave);
    const uint16_t* cols[NT];
#pragma unroll
    for (int c = 0; c < NT; ++c) cols[c] = act + (size_t)min(p0 + c * 16 + lane % 16, end - 1) * I;
    f32x4 acc[1][NT];
#pragma unroll
    for (int c = 0; c < NT; ++c) acc[0][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    multiply_rows<W, 1, NT>(rows, cols, I, s0, s1, acc);
#pragma unroll
    for (int c = 0; c < NT; ++c) {
        const int p = p0 + c * 16 + lane % 16;
        if (p >= lo && p < hi) y[p] = acc[0][c];  // this lane's quarter is the column's expert
    }
}

template <class W>
__global__ __launch_bounds__(kThreads) void decode_down_kernel(int T, int k, const uint8_t* __restrict__ w,
                                                               const uint8_t* __restrict__ sc, int H, int I,
                                                               const Tables* __restrict__ tables,
                                                               const uint16_t* __restrict__ act,
                                                               const float* __restrict__ topk_weights,
                                                               uint16_t* __restrict__ out) {
    __shared__ f32x4 s_y[kMaxY];
    __shared__ float s_w[kMaxSlots];
    __shared__ int32_t s_dest[kMaxSlots];
    const int lane = (int)(threadIdx.x % kWave);
    const int wave = (int)(threadIdx.x / kWave);
    const int h0 = (int)blockIdx.x * 4;
    const int n = tables->n;
    const int pairs = tables->first[n];
    for (int s = (int)threadIdx.x; s < T * k; s += kThreads) {
        s_w[s] = topk_weights[s];
        s_dest[s] = tables->dest[s];
    }
    const int units = (n + 3) / 4;
    const int parts = k_parts(units);
    const int steps = (I + W::STEP - 1) / W::STEP;
    for (int task = wave; task < units * parts; task += kWaves) {
        const int u = task / parts, part = task - u * parts;
        const int mine = min(4 * u + lane % 16 / 4, n - 1);  // the expert of the lane's weight row
        const size_t row = (size_t)tables->expert[mine] * H + min(h0 + lane % 4, H - 1);
        const WeightRow rows[1] = {weight_row<W>(w, sc, row, I)};
        const int quarter = 4 * u + lane / 16;  // the expert of the lane's accumulators
        const int lo = tables->first[min(quarter, n)], hi = tables->first[min(quarter + 1, n)];
        const int begin = tables->first[4 * u], end = tables->first[min(4 * u + 4, n)];
        const int s0 = steps * part / parts, s1 = steps * (part + 1) / parts;
        f32x4* y = s_y + part * pairs;
        for (int p0 = begin; p0 < end; p0 += 32) {
            if (end - p0 <= 16)
                down_columns<W, 1>(rows, act, I, p0, lo, hi, end, s0, s1, y);
            else
                down_columns<W, 2>(rows, act, I, p0, lo, hi, end, s0, s1, y);
        }
    }
    __syncthreads();
    for (int i = (int)threadIdx.x; i < T * 4; i += kThreads) {
        const int t = i / 4, h = i % 4;
        float sum = 0.0f;
        for (int j = 0; j < k; ++j) {
            const int s = t * k + j;
            float y = 0.0f;
            for (int part = 0; part < parts; ++part) y += s_y[part * pairs + s_dest[s]][h];
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
    decode_down_kernel<W><<<(a.H + 3) / 4, kThreads, 0, stream>>>(
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
