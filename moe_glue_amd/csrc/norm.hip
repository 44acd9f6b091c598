// moe_rmsnorm, moe_rmsnorm_fp8, moe_rmsnorm_mxfp8 on gfx950: the residual's
// addition, the root-mean-square norm and the output's format in one pass.
//
//   s = x + r              (fp32; residual_out = bf16(s))
//   n = s / sqrt(mean(s^2) + eps) * w        (fp32)
//   out = bf16(n), or E4M3 codes of n with fp32 or E8M0 block scales
//
// Bound by HBM: about 6 operations for 6 to 8 bytes (8192 x 7168 with residual
// and MXFP8 out moves 412 MB in 68 us, 6.0 TB/s).  A row stays in
// registers from its load to its store, so x and r are read once.  One
// workgroup takes one row with WPR waves of NV 16-byte vectors a lane; the
// sum of squares crosses lanes by DPP and waves by LDS, in an order that
// depends on H alone, so a row's result does not depend on its batch.
// n is rounded once, straight from fp32, in every format (codes are not
// taken of a bf16 row).
#include "fp8_common.h"
#include "kernels.h"

namespace moe {
namespace {

enum NormMode { kNormBf16 = 0, kNormFp8 = 1, kNormMx = 2 };

constexpr uint32_t kInfBits = 0x7F800000u;

template <int WPR>
__device__ __forceinline__ float row_sum(float v, float* s_part) {
    v = __builtin_bit_cast(float, group_reduce<kWave, Op::FAdd>(__builtin_bit_cast(uint32_t, v)));
    if constexpr (WPR > 1) {
        if (threadIdx.x % kWave == 0) s_part[threadIdx.x / kWave] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int w = 0; w < WPR; ++w) v += s_part[w];
    }
    return v;
}

template <int WPR, int NV, int MODE>
__global__ __launch_bounds__(kWave* WPR) void rmsnorm_kernel(const u32x4* __restrict__ x, const u32x4* r,
                                                             const u32x4* __restrict__ w, uint32_t n8, float width,
                                                             float eps, u32x4* r_out, u32x4* out,
                                                             u32x2* __restrict__ codes, void* __restrict__ scales,
                                                             int gl) {
    constexpr int THREADS = kWave * WPR;
    __shared__ float s_part[2][WPR];
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
    float sq = 0.0f;
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
        for (int e = 0; e < 8; ++e) sq = fmaf(s[i][e], s[i][e], sq);
    }
    if (r_out != nullptr)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const uint32_t c = threadIdx.x + i * THREADS;
            if (c < n8) store_stream(r_out + base + c, pack8(s[i]));
        }
    float sum = row_sum<WPR>(sq, s_part[0]);
    if (!(sum < __builtin_inff())) {
        // squares beyond fp32 (|s| from 2^64): once more on s * 2^-80, whose
        // squares cannot overflow (an infinite or NaN s still does: NaN)
        sq = 0.0f;
        eps *= 0x1p-80f * 0x1p-80f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s[i][e] *= 0x1p-80f;
                sq = fmaf(s[i][e], s[i][e], sq);
            }
        sum = row_sum<WPR>(sq, s_part[1]);
    }
    const float rstd = 1.0f / sqrtf(sum / width + eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const uint32_t c = threadIdx.x + i * THREADS;
        float f[8], n[8];
        unpack8(wv[i], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) n[e] = s[i][e] * rstd * f[e];
        if (out != nullptr && c < n8) store_stream(out + base + c, pack8(n));
        if constexpr (MODE != kNormBf16) {
            // a scale group is gl consecutive lanes; H is a multiple of it, so
            // a group lies whole inside or whole past the row
            const uint32_t amax = group_abs_max(abs_max_bits8(n), gl);
            BlockScale b = block_scale(amax, MODE == kNormMx);
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
        kernel<<<a.T, kWave * WPR, 0, stream>>>(
            static_cast<const u32x4*>(a.x), static_cast<const u32x4*>(a.residual),
            static_cast<const u32x4*>(a.weight), n8, (float)a.H, a.eps, static_cast<u32x4*>(a.residual_out),
            static_cast<u32x4*>(a.out), static_cast<u32x2*>(a.codes), a.scales, a.group / 8);
        return hipGetLastError();
    };
    if (a.codes == nullptr) return go(rmsnorm_kernel<WPR, NV, kNormBf16>);
    return a.mx ? go(rmsnorm_kernel<WPR, NV, kNormMx>) : go(rmsnorm_kernel<WPR, NV, kNormFp8>);
}

}  // namespace

hipError_t launch_rmsnorm(const NormArgs& a, hipStream_t stream) {
    // Two vectors a lane, as many waves as that takes: at 4096 x 2048 bf16 12.8 us
    // (one vector and twice the waves 13.5, four and half 12.8), 1023 x 4096 FP8
    // 8.3 (9.1, 9.0), 8192 x 7168 MXFP8 68.1 (four waves of four 69.7, fourteen of
    // one 71.8); one row of 2048 1.9 (1.7, 2.2).  Rows past 8192 columns take
    // sixteen waves.
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
    return launch_shape<16, 8>(a, stream);
}

}  // namespace moe
