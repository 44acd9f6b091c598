// Gradients of the streaming steps on gfx950: SwiGLU, combine, expand (dispatch)
// and the routing's softmax over the selected keys.  All are bound by their bytes.
#include "device_common.h"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kKMax = 16;

// ------------------------------------------------------------------ SwiGLU
// act = g s u with s = 1 / (1 + e^-g):
//   du = dact g s,   dg = dact u s (1 + g (1 - s))
// with 1 - s = e^-g s formed as s(-g), so that it keeps its digits for large g.
// One 16-byte vector of each of gate, up and dact a lane, as moe_swiglu.  32768 x 768
// with act: 48.6 us, 6.2 TB/s of HBM's 6.7.
constexpr int kSwigluThreads = 64;

template <bool ACT>
__global__ __launch_bounds__(kSwigluThreads) void swiglu_backward_kernel(const u32x4* h, const u32x4* dact,
                                                                         uint32_t n, uint32_t I8, FastDiv div_i8,
                                                                         u32x4* dh, u32x4* act) {
    const uint32_t i = blockIdx.x * kSwigluThreads + threadIdx.x;
    if (i >= n) return;
    const uint32_t r = fastdiv(i, div_i8);
    const size_t at = (size_t)r * (2 * I8) + (i - r * I8);
    float g[8], u[8], d[8], dg[8], du[8], a[8];
    const u32x4 gv = load_stream(h + at), uv = load_stream(h + at + I8), dv = load_stream(dact + i);
    unpack8(gv, g);
    unpack8(uv, u);
    unpack8(dv, d);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        // e^-|g| <= 1: neither form overflows
        const float e = __builtin_amdgcn_exp2f(-__builtin_fabsf(g[q]) * 1.4426950408889634f);
        const float small = __builtin_amdgcn_rcpf(1.0f + e);      // s(|g|)
        const float s = g[q] >= 0.0f ? small : e * small;         // s(g)
        const float rest = g[q] >= 0.0f ? e * small : small;      // 1 - s(g)
        const float silu = g[q] * s;
        dg[q] = d[q] * u[q] * (s + silu * rest);
        du[q] = d[q] * silu;
        if constexpr (ACT) a[q] = silu * u[q];
    }
    store_stream(dh + at, pack8(dg));
    store_stream(dh + at + I8, pack8(du));
    if constexpr (ACT) store_stream(act + i, pack8(a));
}

// ----------------------------------------------------------------- combine
// out[t] = sum_j w[t, j] y[dest]: dy[dest] = bf16(w dout[t]), dw[t, j] = <dout[t],
// y[dest]>.  A workgroup takes one token: each lane holds its 16-byte vectors of
// dout, reads the k rows' and writes the k gradients'; the k sums meet through
// lane-group reductions and LDS.  8192 x 7168, k = 8: 400 us, 4.9 TB/s, of as many bytes
// written as read, in rows all over y (a stream of that mix in order: 6.6; rows taken in the order
// of y would need the inverse map, which moe_route gives and this call does not take); 64 to 896 lanes a token, other store
// hints and rows asked for ahead all took 400 to 417.  (Rows of up to 512 columns take
// one wave: 8192 x 128, k = 8 10.0 us, 14.9 with four; 8192 x 512 26.2 and 28.3.)
template <int THREADS, int KC>
__global__ __launch_bounds__(THREADS) void combine_backward_kernel(const u32x4* __restrict__ dout,
                                                                   const u32x4* y, const float* __restrict__ w,
                                                                   const int32_t* __restrict__ dest_of_src,
                                                                   uint32_t H8, int k, u32x4* dy,
                                                                   float* __restrict__ dw) {
    constexpr int WAVES = THREADS / kWave;
    __shared__ float s_sum[KC][WAVES];
    const uint32_t t = blockIdx.x;
    const int32_t* dt = dest_of_src + (size_t)t * k;
    const float* wt = w + (size_t)t * k;
    float sum[KC];
#pragma unroll
    for (int j = 0; j < KC; ++j) sum[j] = 0.0f;
    for (uint32_t c = threadIdx.x; c < H8; c += THREADS) {
        const u32x4 dv = load_stream(dout + (size_t)t * H8 + c);
        u32x4 yv[KC];
#pragma unroll
        for (int j = 0; j < KC; ++j)
            if (j < k) yv[j] = load_stream(y + (size_t)dt[j] * H8 + c);
        float d[8];
        unpack8(dv, d);
#pragma unroll
        for (int j = 0; j < KC; ++j) {
            if (j < k) {
                float v[8], o[8];
                unpack8(yv[j], v);
                const float wj = wt[j];
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    sum[j] = __builtin_fmaf(d[q], v[q], sum[j]);
                    o[q] = wj * d[q];
                }
                store_stream(dy + (size_t)dt[j] * H8 + c, pack8(o));
            }
        }
    }
#pragma unroll
    for (int j = 0; j < KC; ++j) {
        const float v = __builtin_bit_cast(float, group_reduce<64, Op::FAdd>(__builtin_bit_cast(uint32_t, sum[j])));
        if (threadIdx.x % kWave == 0) s_sum[j][threadIdx.x / kWave] = v;
    }
    __syncthreads();
    if ((int)threadIdx.x < k) {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < WAVES; ++i) v += s_sum[threadIdx.x][i];
        dw[(size_t)t * k + threadIdx.x] = v;
    }
}

// ------------------------------------------------------------------ expand
// x_expanded[dest] = x[t]: dx[t] = bf16(residual[t] + sum_j dx_expanded[dest]),
// fp32 in j order.  One 16-byte vector of one token's row a lane, its k loads in
// flight at once, as combine.  8192 x 7168, k = 8 with residual: 195 us, 6.0 TB/s.
constexpr int kExpandThreads = 64;

template <int KC>
__global__ __launch_bounds__(kExpandThreads) void expand_backward_kernel(const u32x4* __restrict__ dxe,
                                                                         const int32_t* __restrict__ dest_of_src,
                                                                         const u32x4* residual, uint32_t n,
                                                                         uint32_t H8, FastDiv div_h8, int k,
                                                                         u32x4* dx) {
    const uint32_t i = blockIdx.x * kExpandThreads + threadIdx.x;
    if (i >= n) return;
    const uint32_t t = fastdiv(i, div_h8), c = i - t * H8;
    const int32_t* dt = dest_of_src + (size_t)t * k;
    u32x4 v[KC];
#pragma unroll
    for (int j = 0; j < KC; ++j)
        if (j < k) v[j] = load_stream(dxe + (size_t)dt[j] * H8 + c);
    float acc[8] = {};
    if (residual != nullptr) unpack8(load_stream(residual + i), acc);
#pragma unroll
    for (int j = 0; j < KC; ++j) {
        if (j < k) {
            float f[8];
            unpack8(v[j], f);
#pragma unroll
            for (int q = 0; q < 8; ++q) acc[q] += f[q];
        }
    }
    store_stream(dx + i, pack8(acc));
}

// ------------------------------------------------------------------- route
// w = softmax over the k selected keys: ds_j = w_j (dw_j - sum_i w_i dw_i), the
// gradient of the logit of expert topk_ids[t, j]; every other logit's is 0.  A
// wave takes a row of dlogits: lane j < k holds slot j, and each lane writes the
// experts e = lane + 64 i, adding up its own among the slots.  8192 x 256: 6.9 us, most of it
// latency.
constexpr int kRouteThreads = 256;

__global__ __launch_bounds__(kRouteThreads) void route_backward_kernel(const int32_t* __restrict__ topk_ids,
                                                                       const float* __restrict__ w,
                                                                       const float* __restrict__ dw, int T, int E,
                                                                       int k, float* __restrict__ dlogits) {
    const int lane = (int)(threadIdx.x % kWave);
    const int64_t t = (int64_t)blockIdx.x * (kRouteThreads / kWave) + uniform(threadIdx.x / kWave);
    if (t >= T) return;
    float wj = 0.0f, dj = 0.0f;
    int id = -1;
    if (lane < k) {
        wj = w[t * k + lane];
        dj = dw[t * k + lane];
        id = topk_ids[t * k + lane];
    }
    const float mean = __builtin_bit_cast(float, group_reduce<64, Op::FAdd>(__builtin_bit_cast(uint32_t, wj * dj)));
    const float ds = wj * (dj - mean);
    for (int e0 = 0; e0 < E; e0 += kWave) {
        float v = 0.0f;
        for (int j = 0; j < k; ++j) {
            const int ij = __builtin_amdgcn_readlane(id, j);
            const float sj = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, ds), j));
            if (ij == e0 + lane) v += sj;
        }
        if (e0 + lane < E) dlogits[t * E + e0 + lane] = v;
    }
}

// dbias[e] = sum_t dlogits[t, e]: a workgroup takes 16 experts, 64 lanes of tokens
// by 16 experts; the sums meet in LDS in one order.  E / 16 workgroups walk all tokens, so it is
// latency: with the logits' launch 13 us for 1023 tokens, 27 for 8192 x 256 (8.4 without it), 88
// and 160 for 65536 x 8 and x 256 (8.5 and 33).
constexpr int kBiasThreads = 1024, kBiasExperts = 16, kBiasRows = kBiasThreads / kBiasExperts;

__global__ __launch_bounds__(kBiasThreads) void route_bias_kernel(const float* __restrict__ dlogits, int T, int E,
                                                                  float* __restrict__ dbias) {
    __shared__ float s_sum[kBiasRows][kBiasExperts];
    const int e = (int)blockIdx.x * kBiasExperts + (int)(threadIdx.x % kBiasExperts);
    const int r = (int)(threadIdx.x / kBiasExperts);
    float sum[4] = {};
    if (e < E) {
        int64_t t = r;
        for (; t + 3 * kBiasRows < T; t += 4 * kBiasRows)
#pragma unroll
            for (int q = 0; q < 4; ++q) sum[q] += dlogits[(t + q * kBiasRows) * E + e];
        for (; t < T; t += kBiasRows) sum[0] += dlogits[t * E + e];
    }
    s_sum[r][threadIdx.x % kBiasExperts] = (sum[0] + sum[1]) + (sum[2] + sum[3]);
    for (int half = kBiasRows / 2; half > 0; half /= 2) {
        __syncthreads();
        if (r < half) s_sum[r][threadIdx.x % kBiasExperts] += s_sum[r + half][threadIdx.x % kBiasExperts];
    }
    if (r == 0 && e < E) dbias[e] = s_sum[0][threadIdx.x];
}

// A launch holds fewer than 2^32 lanes: kSliceTokens tokens of up to 256.
constexpr int64_t kSliceTokens = 1 << 22;

template <int THREADS>
hipError_t combine_threads(const void* dout, const void* y, const float* w, const int32_t* dest, int T, int H, int k,
                           void* dy, float* dw, hipStream_t stream) {
    const auto* yv = static_cast<const u32x4*>(y);
    auto* o = static_cast<u32x4*>(dy);
    const uint32_t H8 = (uint32_t)H / 8;
    for (int64_t t = 0; t < T; t += kSliceTokens) {
        const uint32_t n = (uint32_t)(T - t < kSliceTokens ? T - t : kSliceTokens);
        const auto* d = static_cast<const u32x4*>(dout) + t * H8;
        if (k <= 8)
            combine_backward_kernel<THREADS, 8><<<n, THREADS, 0, stream>>>(d, yv, w + t * k, dest + t * k, H8, k, o,
                                                                           dw + t * k);
        else
            combine_backward_kernel<THREADS, kKMax><<<n, THREADS, 0, stream>>>(d, yv, w + t * k, dest + t * k, H8, k,
                                                                               o, dw + t * k);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_swiglu_backward(const void* h, const void* dact, int R, int I, void* dh, void* act,
                                  hipStream_t stream) {
    const uint32_t I8 = (uint32_t)I / 8, n = (uint32_t)R * I8;
    const uint32_t blocks = (n + kSwigluThreads - 1) / kSwigluThreads;
    const auto* hv = static_cast<const u32x4*>(h);
    const auto* dv = static_cast<const u32x4*>(dact);
    auto* o = static_cast<u32x4*>(dh);
    if (act != nullptr)
        swiglu_backward_kernel<true><<<blocks, kSwigluThreads, 0, stream>>>(hv, dv, n, I8, make_fastdiv(I8), o,
                                                                            static_cast<u32x4*>(act));
    else
        swiglu_backward_kernel<false><<<blocks, kSwigluThreads, 0, stream>>>(hv, dv, n, I8, make_fastdiv(I8), o,
                                                                             nullptr);
    return hipGetLastError();
}

hipError_t launch_combine_backward(const void* dout, const void* y, const float* topk_weights,
                                   const int32_t* dest_of_src, int T, int H, int k, void* dy, float* dweights,
                                   hipStream_t stream) {
    if (H <= 8 * 64) return combine_threads<64>(dout, y, topk_weights, dest_of_src, T, H, k, dy, dweights, stream);
    return combine_threads<256>(dout, y, topk_weights, dest_of_src, T, H, k, dy, dweights, stream);
}

hipError_t launch_expand_backward(const void* dx_expanded, const int32_t* dest_of_src, const void* residual, int T,
                                  int H, int k, void* dx, hipStream_t stream) {
    const uint32_t H8 = (uint32_t)H / 8, n = (uint32_t)T * H8;
    const uint32_t blocks = (n + kExpandThreads - 1) / kExpandThreads;
    const auto* v = static_cast<const u32x4*>(dx_expanded);
    const auto* r = static_cast<const u32x4*>(residual);
    auto* o = static_cast<u32x4*>(dx);
    if (k <= 8)
        expand_backward_kernel<8><<<blocks, kExpandThreads, 0, stream>>>(v, dest_of_src, r, n, H8, make_fastdiv(H8), k,
                                                                         o);
    else
        expand_backward_kernel<kKMax><<<blocks, kExpandThreads, 0, stream>>>(v, dest_of_src, r, n, H8,
                                                                             make_fastdiv(H8), k, o);
    return hipGetLastError();
}

hipError_t launch_route_backward(const int32_t* topk_ids, const float* topk_weights, const float* dweights, int T,
                                 int E, int k, float* dlogits, float* dbias, hipStream_t stream) {
    const uint32_t rows = kRouteThreads / kWave;
    for (int64_t t = 0; t < T; t += kSliceTokens) {
        const int n = (int)(T - t < kSliceTokens ? T - t : kSliceTokens);
        route_backward_kernel<<<((uint32_t)n + rows - 1) / rows, kRouteThreads, 0, stream>>>(
            topk_ids + t * k, topk_weights + t * k, dweights + t * k, n, E, k, dlogits + t * E);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (dbias != nullptr)
        route_bias_kernel<<<(E + kBiasExperts - 1) / kBiasExperts, kBiasThreads, 0, stream>>>(dlogits, T, E, dbias);
    return hipGetLastError();
}

}  // namespace moe
