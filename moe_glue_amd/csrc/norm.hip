// moe_rmsnorm, moe_rmsnorm_fp8, moe_rmsnorm_mxfp8 on gfx950: the residual's
// addition, the root-mean-square norm and the output's format in one pass.
//
//   s = x + r              (fp32; residual_out = bf16(s))
//   n = s / sqrt(mean(s^2) + eps) * w        (fp32)
//   out = bf16(n), or E4M3 codes of n with fp32 or E8M0 block scales
//
// Bound by HBM: about 6 operations for 6 to 8 bytes (8192 x 7168 with residual
// and MXFP8 out moves 412 MB in 69 us, 6.0 TB/s).  A row stays in
// registers from its load to its store, so x and r are read once.  One
// workgroup takes one row with WPR waves of NV 16-byte vectors a lane; the
// sum of squares crosses lanes by DPP and waves by LDS, in an order that
// depends on H alone, so a row's result does not depend on its batch.
// The sum of squares and the root are formed in fp64, which has the range for
// any fp32 square, and so are the products of a vector whose s / rms falls below
// fp32's normals (the look for one costs 0.1 us at one row, 0.2 of 69 at 8192 x
// 7168); n is then right to three fp32 steps.  An MXFP8 scale is a power of two,
// decided by which power the block's maximum reaches, so a maximum that near to
// one is looked at again in fp64: decided in fp32 about one block in six million
// took the neighbouring scale.  (All products in fp64: 72.4 us instead of 70.0 at
// 8192 x 7168.)  n is rounded once in every format: codes are not taken of a bf16
// row.
#include "fp8_common.h"
#include "kernels.h"

namespace moe {
namespace {

enum NormMode { kNormBf16 = 0, kNormFp8 = 1, kNormMx = 2 };

constexpr uint32_t kInfBits = 0x7F800000u;
// fp32 steps that n may be off by, 2.5 at most (two products and the factor's own
// rounding), with room to spare.
constexpr uint32_t kNear = 8;

// Sum over the 64 lanes of a wave, in every lane.
template <int CTRL>
__device__ __forceinline__ double add_dpp(double v) {
    const u32x2 w = __builtin_bit_cast(u32x2, v);
    return v + __builtin_bit_cast(double, u32x2{dpp<CTRL>(w[0]), dpp<CTRL>(w[1])});
}
__device__ __forceinline__ double wave_sum(double v) {
    v = add_dpp<kQuadXor1>(v);
    v = add_dpp<kQuadXor2>(v);
    v = add_dpp<kRowHalfMirror>(v);
    v = add_dpp<kRowMirror>(v);
    u32x2 w = __builtin_bit_cast(u32x2, v);
    auto lo = __builtin_amdgcn_permlane16_swap(w[0], w[0], false, false);
    auto hi = __builtin_amdgcn_permlane16_swap(w[1], w[1], false, false);
    v = __builtin_bit_cast(double, u32x2{lo[0], hi[0]}) + __builtin_bit_cast(double, u32x2{lo[1], hi[1]});
    w = __builtin_bit_cast(u32x2, v);
    lo = __builtin_amdgcn_permlane32_swap(w[0], w[0], false, false);
    hi = __builtin_amdgcn_permlane32_swap(w[1], w[1], false, false);
    return __builtin_bit_cast(double, u32x2{lo[0], hi[0]}) + __builtin_bit_cast(double, u32x2{lo[1], hi[1]});
}

template <int WPR>
__device__ __forceinline__ double row_sum(double v, double* s_part) {
    v = wave_sum(v);
    if constexpr (WPR > 1) {
        if (threadIdx.x % kWave == 0) s_part[threadIdx.x / kWave] = v;
        __syncthreads();
        v = 0.0;
#pragma unroll
        for (int w = 0; w < WPR; ++w) v += s_part[w];
    }
    return v;
}

// s * rstd * w in fp64, for the few vectors that need it.  The compiler shall not
// know s and w: it would keep all of the row sum's conversions in registers until
// here (8192 x 7168 MXFP8 76 us instead of 70) and convert every weight.
__device__ __forceinline__ double product64(float s, double rstd, float w) {
    asm("" : "+v"(s), "+v"(w));
    return (double)s * rstd * (double)w;
}

template <int WPR, int NV, int MODE>
__global__ __launch_bounds__(kWave* WPR) void rmsnorm_kernel(const u32x4* __restrict__ x, const u32x4* r,
                                                             const u32x4* __restrict__ w, uint32_t n8, double width,
                                                             float eps, u32x4* r_out, u32x4* out,
                                                             u32x2* __restrict__ codes, void* __restrict__ scales,
                                                             int gl) {
    constexpr int THREADS = kWave * WPR;
    __shared__ double s_part[WPR];
    const size_t base = (size_t)blockIdx.x * n8;
    u32x4 xv[NV], rv[NV], wv[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const uint32_t c = threadIdx.x + i * THREADS;
        xv[i] = u32x4{0u, 0u, 0u, 0u};
        rv[i] = u32x4{0u, 0u, 0u, 0u};
        if (c < n8) xv[i] = load_stream(x + base + c);
    }
    if (r != nullptr)  // uniform
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const uint32_t c = threadIdx.x + i * THREADS;
            if (c < n8) rv[i] = load_stream(r + base + c);
        }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const uint32_t c = threadIdx.x + i * THREADS;
        wv[i] = u32x4{0u, 0u, 0u, 0u};
        if (c < n8) wv[i] = w[c];
    }
    float s[NV][8];
    double sq = 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        unpack8(xv[i], s[i]);
        if (r != nullptr) {
            float f[8];
            unpack8(rv[i], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[i][e] += f[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sq = fma((double)s[i][e], (double)s[i][e], sq);
    }
    if (r_out != nullptr)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const uint32_t c = threadIdx.x + i * THREADS;
            if (c < n8) store_stream(r_out + base + c, pack8(s[i]));
        }
    const double rstd = 1.0 / sqrt(row_sum<WPR>(sq, s_part) / width + (double)eps);
    // where fp32 would hold 1 / rms as a subnormal, both factors move by 2^80
    const bool huge = rstd < 0x1p-100;
    const float pre = huge ? 0x1p-80f : 1.0f;
    const float scaled = (float)(huge ? rstd * 0x1p80 : rstd);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const uint32_t c = threadIdx.x + i * THREADS;
        float f[8], n[8];
        unpack8(wv[i], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) n[e] = s[i][e] * pre * scaled;
        // a quotient below fp32's normals has lost bits that a large weight would
        // bring back: then, and where it is 0, the vector's products in fp64
        float least = fabsf(n[0]);
#pragma unroll
        for (int e = 1; e < 8; ++e) least = fminf(least, fabsf(n[e]));
        if (__builtin_expect(least < 0x1p-126f, 0)) {
#pragma unroll
            for (int e = 0; e < 8; ++e) n[e] = (float)product64(s[i][e], rstd, f[e]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) n[e] *= f[e];
        }
        if (out != nullptr && c < n8) store_stream(out + base + c, pack8(n));
        if constexpr (MODE != kNormBf16) {
            // a scale group is gl consecutive lanes; H is a multiple of it, so
            // a group lies whole inside or whole past the row
            const uint32_t amax = group_abs_max(abs_max_bits8(n), gl);
            BlockScale b = block_scale(amax, MODE == kNormMx);
            if constexpr (MODE == kNormMx) {
                // a maximum within fp32's error of a power of two: whether it reaches
                // it decides the scale, so look again with products in fp64, which
                // neither pass its range nor fall below it.  A finite maximum below
                // 2^128 does not reach it.
                const bool near = (amax + kNear) % 0x800000u < 2 * kNear && amax + kNear < kInfBits;
                if (__any(near)) {
                    // short of it by less than the row sum's and the products' own
                    // errors, 2^-44 of it, is on it: rows of one magnitude land there
                    const uint32_t edge = (amax + kNear) & 0xFF800000u;
                    const double reach = (double)__builtin_bit_cast(float, edge) * (1.0 - 0x1p-44);
                    uint32_t reaches = 0;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (fabs(product64(s[i][e], rstd, f[e])) >= reach) reaches = 1;
                    reaches = group_abs_max(reaches, gl);
                    if (near) b = block_scale(reaches ? edge : edge - 1, true);
                }
            }
            u32x2 q = quantize8_e4m3(n, b.inv, b.pre);
            if (amax >= kInfBits) {  // a NaN or an infinity in the group: NaN scale, NaN codes
                b.scale = __builtin_nanf("");
                b.byte = 0xFF;
                q = u32x2{0x7F7F7F7Fu, 0x7F7F7F7Fu};
            }
            if (c < n8) {
                __builtin_nontemporal_store(q, codes + base + c);
                if (threadIdx.x % (uint32_t)gl == 0)
                    store_block_scale(scales, (base + c) / (uint32_t)gl, b, MODE == kNormMx);
            }
        }
    }
}

template <int WPR, int NV>
hipError_t launch_shape(const NormArgs& a, hipStream_t stream) {
    const uint32_t n8 = (uint32_t)a.H / 8;
    const auto go = [&](auto kernel) {
        for (int i = 0; i < norm_launches(a.T); ++i) {
            const NormLaunch part = norm_launch(a.T, i);
            const size_t at = (size_t)part.first * n8;
            const auto rows = [at](const void* p) {
                return p == nullptr ? nullptr : static_cast<const u32x4*>(p) + at;
            };
            const auto out_rows = [at](void* p) { return p == nullptr ? nullptr : static_cast<u32x4*>(p) + at; };
            u32x2* codes = a.codes == nullptr ? nullptr : static_cast<u32x2*>(a.codes) + at;
            void* scales = a.codes == nullptr ? nullptr
                                              : static_cast<char*>(a.scales) +
                                                    at / (size_t)(a.group / 8) * (a.mx ? 1 : sizeof(float));
            kernel<<<part.rows, kWave * WPR, 0, stream>>>(
                rows(a.x), rows(a.residual), static_cast<const u32x4*>(a.weight), n8, (double)a.H, a.eps,
                out_rows(a.residual_out), out_rows(a.out), codes, scales, a.group / 8);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        return hipSuccess;
    };
    if (a.codes == nullptr) return go(rmsnorm_kernel<WPR, NV, kNormBf16>);
    return a.mx ? go(rmsnorm_kernel<WPR, NV, kNormMx>) : go(rmsnorm_kernel<WPR, NV, kNormFp8>);
}

}  // namespace

hipError_t launch_rmsnorm(const NormArgs& a, hipStream_t stream) {
    // Two vectors a lane, as many waves as that takes (medians): at 4096 x 2048 bf16
    // 13.2 us (one vector and twice the waves 13.4, four and half 13.1), 1023 x 4096
    // FP8 9.1 (9.9, 9.9), 8192 x 7168 MXFP8 69.2 (77.2, 70.4); one row of 2048 2.1
    // (1.9, 2.5).  Rows past 8192 columns take sixteen waves.
    const int waves = (a.H / 8 + 2 * kWave - 1) / (2 * kWave);
    switch (waves) {
        case 1: return launch_shape<1, 2>(a, stream);
        case 2: return launch_shape<2, 2>(a, stream);
        case 3: return launch_shape<3, 2>(a, stream);
        case 4: return launch_shape<4, 2>(a, stream);
        case 5: return launch_shape<5, 2>(a, stream);
        case 6: return launch_shape<6, 2>(a, stream);
        case 7: return launch_shape<7, 2>(a, stream);
        case 8: return launch_shape<8, 2>(a, stream);
        default: break;
    }
    if (waves <= 16) return launch_shape<16, 2>(a, stream);
    static_assert(16 * 8 * kWave * 8 == MOE_NORM_H_MAX, "the widest row: 16 waves of 8 vectors a lane");
    return launch_shape<16, 8>(a, stream);
}

}  // namespace moe
