// Products of a few tokens with streamed weight rows, for the few-token layer
// (decode_layer.hip) and the MXFP4 linear (linear.hip).
//
// v_mfma_f32_16x16x32_bf16 multiplies 16 rows by 16 columns over 32 k: lane l
// holds 8 k of row (of A) and of column (of B) l % 16, which 8 of the 32 by its
// quarter l / 16.  A vector load takes a CU 16 clocks when each four
// neighbouring lanes stay inside one 128-byte line, whatever their width, but 64
// when they all differ (measured, from cache) -- and a weight row per lane makes
// them differ.  So the 16 rows are 4 weight rows times 4 segments of k, and the
// 16 columns 4 tokens times the same segments:
//
//   lane l: row (column) r = l % 16 / 4, segment s = l % 4, quarter q = l / 16
//           k = step + (4 q + s) * P .. + P - 1
//
// Of the products only those of equal segments are wanted: the sum of
// accumulator s over the four lanes s of a quad is token c = l % 16 / 4 times
// row q (diagonal_sum).  Three quarters of the multiplications are thrown away;
// with a few tokens an expert the matrix cores have that to spare.
//
//   bf16   P = 8: a step is 128 k, one MFMA, 256 bytes of each row
//   MXFP4  P = 16: a step is 256 k, two MFMAs, 128 bytes of each row (with 8
//          bytes a lane; 4 cost as many clocks, and with 16 the neighbouring
//          lanes' columns would lie 64 bytes apart).  Two lanes share a scale
//          block of 32 columns.  E2M1 times 2^e has a 2-bit significand, so the
//          widening to bf16 (v_cvt_scalef32_pk_bf16_fp4, scale included) is
//          exact.
#pragma once

#include <type_traits>

#include "device_common.h"

namespace moe {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// A wave-uniform offset that the compiler cannot see to be one.  (Pointers stay
// sums of a kernel argument and such an offset: then loads are global ones with
// a scalar base.)
__device__ __forceinline__ size_t uniform_offset(size_t v) {
    return (size_t)uniform((uint32_t)(v >> 32)) << 32 | uniform((uint32_t)v);
}
__device__ __forceinline__ int wave_index() { return (int)uniform(threadIdx.x / kWave); }

// Weight rows of one matrix part: row i's codes at w + i * row_bytes(K), its
// scales at scales + i * row_scales(K); w and scales are uniform.
struct WeightBase {
    const uint8_t* w;
    const uint8_t* scales;
};

// A lane's part of one row over U steps: load() fills step u's registers (and
// scales() those of SCALE_STEPS steps), values<u, m>() gives the 8 weights of
// its MFMA m.
struct Bf16Weights {
    static constexpr int STEP = 128;
    static constexpr int SUB = 1;          // MFMAs per step
    static constexpr int SCALE_STEPS = 1;  // steps to a scale load (1: no scales)
    template <int U>
    struct Rows {
        u32x4 v[U];
    };
    static __device__ __forceinline__ uint32_t row_bytes(int K) { return (uint32_t)K * 2; }
    static __device__ __forceinline__ uint32_t row_scales(int) { return 0; }
    template <int U>
    static __device__ __forceinline__ void scales(Rows<U>&, int, const WeightBase&, uint32_t, int, int) {}
    template <int U>
    static __device__ __forceinline__ void load(Rows<U>& f, int u, const WeightBase& b, uint32_t row, int K,
                                                uint32_t k) {
        f.v[u] = *reinterpret_cast<const u32x4*>(b.w + (row * row_bytes(K) + k * 2));
    }
    template <int U>
    static __device__ __forceinline__ void clear(Rows<U>& f, int u) {
        f.v[u] = u32x4{0u, 0u, 0u, 0u};
    }
    template <int u, int M, int U>
    static __device__ __forceinline__ bf16x8 values(const Rows<U>& f) {
        return __builtin_bit_cast(bf16x8, f.v[u]);
    }
};

struct Mxfp4Weights {
    static constexpr int STEP = 256;
    static constexpr int SUB = 2;
    static constexpr int SCALE_STEPS = 2;
    template <int U>
    struct Rows {
        u32x2 codes[U];
        uint32_t scale[(U + 1) / 2];  // even lanes: step 2 g's, odd lanes: step 2 g + 1's, as fp32 bits
    };
    static __device__ __forceinline__ uint32_t row_bytes(int K) { return (uint32_t)K / 2; }
    static __device__ __forceinline__ uint32_t row_scales(int K) { return (uint32_t)K / 32; }
    // One byte load for two steps: of the two lanes that share a block in both,
    // each fetches one step's byte, and values() hands it over.  2^(b - 127) has
    // exponent field b; b = 0 is a subnormal, 255 is NaN.
    template <int U>
    static __device__ __forceinline__ void scales(Rows<U>& f, int g, const WeightBase& b, uint32_t row, int K,
                                                  int step) {
        const uint32_t lane = threadIdx.x % kWave;
        const uint32_t at = min((uint32_t)(step + lane % 2) * (STEP / 32) + lane / 16 * 2 + lane % 4 / 2,
                                row_scales(K) - 1);
        const uint32_t v = b.scales[row * row_scales(K) + at];
        f.scale[g] = v == 0u ? 0x00400000u : v == 255u ? 0x7FC00000u : v << 23;
    }
    template <int U>
    static __device__ __forceinline__ void load(Rows<U>& f, int u, const WeightBase& b, uint32_t row, int K,
                                                uint32_t k) {
        f.codes[u] = *reinterpret_cast<const u32x2*>(b.w + (row * row_bytes(K) + k / 2));
    }
    template <int U>
    static __device__ __forceinline__ void clear(Rows<U>& f, int u) {
        f.codes[u] = u32x2{0u, 0u};
    }
    template <int u, int M, int U>
    static __device__ __forceinline__ bf16x8 values(const Rows<U>& f) {
        // quad_perm [0, 0, 2, 2] or [1, 1, 3, 3]
        const float s = __builtin_bit_cast(float, dpp<u % 2 == 0 ? 0xA0 : 0xF5>(f.scale[u / 2]));
        const uint32_t v = f.codes[u][M];
        const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, s, 0);
        const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, s, 1);
        const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, s, 2);
        const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, s, 3);
        return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
    }
};

template <class W>
__device__ __forceinline__ int steps_of(int K) {
    return (K + W::STEP - 1) / W::STEP;
}

template <int N, class F>
__device__ __forceinline__ void unrolled(F&& f) {
    if constexpr (N > 0) {
        unrolled<N - 1>(f);
        f(std::integral_constant<int, N - 1>{});
    }
}

// acc[r][c] += the lane's row of base[r] (row[r], counted from base[r]) times
// its column c (first bf16 at x + col[c], in bytes) over the steps [s0, s1) of
// K, both uniform.  The loads of U steps are in flight: a step's registers are
// loaded again, for the step U later, as soon as it is multiplied.  In a step
// that K ends inside, lanes past K load the row's last piece and hold zeros.
template <class W, int RT, int NT, int U>
__device__ __forceinline__ void multiply_rows(const WeightBase (&base)[RT], const uint32_t (&row)[RT],
                                              const uint8_t* x, const uint32_t (&col)[NT], int K, int s0, int s1,
                                              f32x4 (&acc)[RT][NT]) {
    constexpr int PIECE = W::STEP / 16;
    static_assert(PIECE == 8 * W::SUB && U % W::SCALE_STEPS == 0, "whole pieces, whole scale loads");
    const uint32_t lane = threadIdx.x % kWave;
    const uint32_t piece = (lane / 16 * 4 + lane % 4) * PIECE;
    const uint32_t last = (uint32_t)K - PIECE;
    typename W::template Rows<U> a[RT];
    u32x4 b[U][NT][W::SUB];
    const auto load = [&](auto index, int s) {
        constexpr int u = decltype(index)::value;
        const uint32_t k = min((uint32_t)s * W::STEP + piece, last);
#pragma unroll
        for (int r = 0; r < RT; ++r) W::load(a[r], u, base[r], row[r], K, k);
#pragma unroll
        for (int c = 0; c < NT; ++c)
#pragma unroll
            for (int m = 0; m < W::SUB; ++m)
                b[u][c][m] = *reinterpret_cast<const u32x4*>(x + (col[c] + k * 2 + m * 16));
    };
    const auto scales = [&](int g, int s) {
#pragma unroll
        for (int r = 0; r < RT; ++r) W::scales(a[r], g, base[r], row[r], K, s);
    };
    unrolled<U>([&](auto index) {
        constexpr int u = decltype(index)::value;
        if (s0 + u >= s1) return;
        if constexpr (W::SCALE_STEPS > 1 && u % W::SCALE_STEPS == 0) scales(u / W::SCALE_STEPS, s0 + u);
        load(index, s0 + u);
    });
    for (int s = s0; s < s1; s += U)
        unrolled<U>([&](auto index) {
            constexpr int u = decltype(index)::value;
            if (s + u >= s1) return;
            if ((s + u + 1) * W::STEP > K && (uint32_t)(s + u) * W::STEP + piece > last) {
#pragma unroll
                for (int r = 0; r < RT; ++r) W::clear(a[r], u);
#pragma unroll
                for (int c = 0; c < NT; ++c)
#pragma unroll
                    for (int m = 0; m < W::SUB; ++m) b[u][c][m] = u32x4{0u, 0u, 0u, 0u};
            }
            unrolled<W::SUB>([&](auto sub) {
                constexpr int m = decltype(sub)::value;
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const bf16x8 av = W::template values<u, m>(a[r]);
#pragma unroll
                    for (int c = 0; c < NT; ++c)
                        acc[r][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            av, __builtin_bit_cast(bf16x8, b[u][c][m]), acc[r][c], 0, 0, 0);
                }
            });
            if (s + u + U < s1) load(index, s + u + U);
            if constexpr (W::SCALE_STEPS > 1 && u % W::SCALE_STEPS == W::SCALE_STEPS - 1) {
                constexpr int first = u - (W::SCALE_STEPS - 1);
                if (s + first + U < s1) scales(first / W::SCALE_STEPS, s + first + U);
            }
        });
}

// The product of row l / 16 with column l % 16 / 4, in all four lanes of the
// quad: segment s of both is accumulator s of the quad's lane s.
__device__ __forceinline__ float diagonal_sum(const f32x4& a) {
    const uint32_t s = threadIdx.x % 4;
    const float v = s < 2 ? (s == 0 ? a[0] : a[1]) : (s == 2 ? a[2] : a[3]);
    return __builtin_bit_cast(float, group_reduce<4, Op::FAdd>(__builtin_bit_cast(uint32_t, v)));
}

}  // namespace moe
