// Products of a few tokens with streamed weight rows, shared by the few-token
// layer (decode_layer.hip) and the MXFP4 linear (linear.hip).
//
// D = A B by v_mfma_f32_16x16x32_bf16: A holds 16 weight rows, B 16 tokens
// (columns).  Lane l has row (and column) l % 16 and the k quarter q = l / 16;
// its 4 accumulators are rows 4q .. 4q+3 of column l % 16.  A dot product does
// not mind the order of its terms, so a lane may take any 8 k per instruction
// as long as A and B agree: weights are always loaded 16 bytes a lane, straight
// from memory to registers in the layout that they have there.
//
//   bf16   a step is 32 k: lane q takes k = 32 s + 8 q .. +7, one MFMA
//   MXFP4  a step is 128 k: 16 bytes are the 32 codes of one scale block,
//          k = 128 s + 32 q .. +31, and four MFMAs take 8 of them each.
//          E2M1 times 2^e has a 2-bit significand, so the widening to bf16
//          (v_cvt_scalef32_pk_bf16_fp4, scale included) is exact.
//
// With few tokens most of a tile's columns repeat the last token; the matrix
// cores have that to spare, the weights' stream is what bounds these kernels.
#pragma once

#include <type_traits>

#include "device_common.h"

namespace moe {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// A lane's weight row: its first byte, and its scales.
struct WeightRow {
    const uint8_t* w;
    const uint8_t* scales;
};

struct Bf16Weights {
    static constexpr int STEP = 32;   // k per step
    static constexpr int SUB = 1;     // MFMAs per step
    static constexpr int BATCH = 8;   // steps whose loads are issued together
    struct Frag {
        u32x4 v;
    };
    static __device__ __forceinline__ size_t row_bytes(int K) { return (size_t)K * 2; }
    static __device__ __forceinline__ size_t row_scales(int) { return 0; }
    static __device__ __forceinline__ Frag load(const WeightRow& r, uint32_t k) {
        return {*reinterpret_cast<const u32x4*>(r.w + (size_t)k * 2)};
    }
    static __device__ __forceinline__ void clear(Frag& f) { f.v = u32x4{0u, 0u, 0u, 0u}; }
    template <int M>
    static __device__ __forceinline__ bf16x8 sub(const Frag& f) {
        return __builtin_bit_cast(bf16x8, f.v);
    }
};

struct Mxfp4Weights {
    static constexpr int STEP = 128;
    static constexpr int SUB = 4;
    static constexpr int BATCH = 2;
    struct Frag {
        u32x4 v;
        uint32_t scale;  // E8M0 byte
    };
    static __device__ __forceinline__ size_t row_bytes(int K) { return (size_t)K / 2; }
    static __device__ __forceinline__ size_t row_scales(int K) { return (size_t)K / 32; }
    static __device__ __forceinline__ Frag load(const WeightRow& r, uint32_t k) {
        return {*reinterpret_cast<const u32x4*>(r.w + k / 2), (uint32_t)r.scales[k / 32]};
    }
    static __device__ __forceinline__ void clear(Frag& f) {
        f.v = u32x4{0u, 0u, 0u, 0u};
        f.scale = 127u;
    }
    // 2^(b - 127) as fp32: exponent field b; b = 0 is a subnormal, 255 is NaN
    static __device__ __forceinline__ float scale_value(uint32_t b) {
        const uint32_t u = b == 0u ? 0x00400000u : b == 255u ? 0x7FC00000u : b << 23;
        return __builtin_bit_cast(float, u);
    }
    template <int M>
    static __device__ __forceinline__ bf16x8 sub(const Frag& f) {
        const float s = scale_value(f.scale);
        const uint32_t c = f.v[M];
        const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0);
        const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1);
        const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2);
        const bf16x2 e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3);
        return bf16x8{a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
    }
};

// acc[r][c] += rows r (16 each) times columns c (16 each) over the steps
// [s0, s1) of K.  col[c]: the lane's column, its first bf16.  Steps past the
// range repeat the last one's loads (the addresses stay inside the row) and
// are not multiplied; in a step that K ends inside, lanes past K hold zeros.
template <class W, int RT, int NT>
__device__ __forceinline__ void multiply_rows(const WeightRow (&row)[RT], const uint16_t* const (&col)[NT], int K,
                                              int s0, int s1, f32x4 (&acc)[RT][NT]) {
    constexpr int PIECE = W::STEP / 4;  // k of a lane in a step
    const uint32_t q = (threadIdx.x % kWave) / 16;
    const uint32_t last = (uint32_t)K - PIECE;
    for (int s = s0; s < s1; s += W::BATCH) {
        typename W::Frag a[W::BATCH][RT];
        u32x4 b[W::BATCH][NT][W::SUB];
#pragma unroll
        for (int u = 0; u < W::BATCH; ++u) {
            const uint32_t k = min((uint32_t)min(s + u, s1 - 1) * W::STEP + q * PIECE, last);
#pragma unroll
            for (int r = 0; r < RT; ++r) a[u][r] = W::load(row[r], k);
        }
#pragma unroll
        for (int u = 0; u < W::BATCH; ++u) {
            const uint32_t k = min((uint32_t)min(s + u, s1 - 1) * W::STEP + q * PIECE, last);
#pragma unroll
            for (int c = 0; c < NT; ++c)
#pragma unroll
                for (int m = 0; m < W::SUB; ++m)
                    b[u][c][m] = *reinterpret_cast<const u32x4*>(col[c] + k + m * 8);
        }
#pragma unroll
        for (int u = 0; u < W::BATCH; ++u) {
            if (s + u >= s1) continue;  // uniform
            if ((s + u + 1) * W::STEP > K && (uint32_t)(s + u) * W::STEP + q * PIECE > last) {
#pragma unroll
                for (int r = 0; r < RT; ++r) W::clear(a[u][r]);
#pragma unroll
                for (int c = 0; c < NT; ++c)
#pragma unroll
                    for (int m = 0; m < W::SUB; ++m) b[u][c][m] = u32x4{0u, 0u, 0u, 0u};
            }
            const auto mul = [&](auto sub_index) {
                constexpr int M = decltype(sub_index)::value;
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const bf16x8 av = W::template sub<M>(a[u][r]);
#pragma unroll
                    for (int c = 0; c < NT; ++c)
                        acc[r][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            av, __builtin_bit_cast(bf16x8, b[u][c][M]), acc[r][c], 0, 0, 0);
                }
            };
            mul(std::integral_constant<int, 0>{});
            if constexpr (W::SUB == 4) {
                mul(std::integral_constant<int, 1>{});
                mul(std::integral_constant<int, 2>{});
                mul(std::integral_constant<int, 3>{});
            }
        }
    }
}

}  // namespace moe
