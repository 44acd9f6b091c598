// Products of a few tokens with streamed weight rows, for the few-token layer
// (decode_layer.hip) and the MXFP4 linear (linear.hip).
//
// v_mfma_f32_16x16x32_bf16 multiplies 16 rows by 16 columns over 32 k: lane l
// holds 8 k of row (of A) and of column (of B) l % 16, which 8 of the 32 by its
// quarter l / 16.  A weight row per lane would make neighbouring lanes load from
// different rows, and a wave's 16-byte loads then go through the address path
// one lane at a time (64 clocks a KiB instead of 16: measured on a 16 MB matrix
// in cache, 5.4 us against 3.3).  So the 16 rows are 4 weight rows times 4
// segments of k, and the 16 columns 4 tokens times the same segments:
//
//   lane l: row (column) r = l % 16 / 4, segment s = l % 4, quarter q = l / 16
//           k = 128 step + 32 q + 8 s .. + 7
//
// Four neighbouring lanes load 64 consecutive bytes and the 16 lanes of a row
// 256.  Of the products only those of equal segments are wanted: the sum of
// accumulator s over the four lanes of a quad is token c = l % 16 / 4 times row
// q (diagonal_sum).  Three quarters of the multiplications are thrown away; with
// a few tokens an expert the matrix cores have that to spare.
//
// MXFP4: a lane's 8 codes are one dword, and the four lanes of a quarter share
// the scale block of 32 columns.  E2M1 times 2^e has a 2-bit significand, so
// the widening to bf16 (v_cvt_scalef32_pk_bf16_fp4, scale included) is exact.
#pragma once

#include "device_common.h"

namespace moe {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kStep = 128;  // k per step of a wave: 8 for each lane of a row

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

struct Bf16Weights {
    using Frag = u32x4;
    static __device__ __forceinline__ uint32_t row_bytes(int K) { return (uint32_t)K * 2; }
    static __device__ __forceinline__ uint32_t row_scales(int) { return 0; }
    static __device__ __forceinline__ Frag load(const WeightBase& b, uint32_t row, int K, uint32_t k) {
        return *reinterpret_cast<const u32x4*>(b.w + (row * row_bytes(K) + k * 2));
    }
    static __device__ __forceinline__ Frag zero() { return u32x4{0u, 0u, 0u, 0u}; }
    static __device__ __forceinline__ bf16x8 values(const Frag& f) { return __builtin_bit_cast(bf16x8, f); }
};

struct Mxfp4Weights {
    struct Frag {
        uint32_t codes;
        uint32_t scale;  // E8M0 byte
    };
    static __device__ __forceinline__ uint32_t row_bytes(int K) { return (uint32_t)K / 2; }
    static __device__ __forceinline__ uint32_t row_scales(int K) { return (uint32_t)K / 32; }
    static __device__ __forceinline__ Frag load(const WeightBase& b, uint32_t row, int K, uint32_t k) {
        return {*reinterpret_cast<const uint32_t*>(b.w + (row * row_bytes(K) + k / 2)),
                (uint32_t)b.scales[row * row_scales(K) + k / 32]};
    }
    static __device__ __forceinline__ Frag zero() { return {0u, 127u}; }
    // 2^(b - 127) as fp32: exponent field b; b = 0 is a subnormal, 255 is NaN
    static __device__ __forceinline__ float scale_value(uint32_t b) {
        const uint32_t u = b == 0u ? 0x00400000u : b == 255u ? 0x7FC00000u : b << 23;
        return __builtin_bit_cast(float, u);
    }
    static __device__ __forceinline__ bf16x8 values(const Frag& f) {
        const float s = scale_value(f.scale);
        const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(f.codes, s, 0);
        const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(f.codes, s, 1);
        const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(f.codes, s, 2);
        const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(f.codes, s, 3);
        return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
    }
};

// acc[r][c] += the lane's row of base[r] (row[r], counted from base[r]) times
// its column c (first bf16 at x + col[c], in bytes) over the steps [s0, s1) of
// K.  U steps' loads are issued together; steps past the range repeat the last
// one's loads (addresses stay inside the row) and are not multiplied.  In a
// step that K ends inside, lanes past K hold zeros.
template <class W, int RT, int NT, int U>
__device__ __forceinline__ void multiply_rows(const WeightBase (&base)[RT], const uint32_t (&row)[RT],
                                              const uint8_t* x, const uint32_t (&col)[NT], int K, int s0, int s1,
                                              f32x4 (&acc)[RT][NT]) {
    const uint32_t lane = threadIdx.x % kWave;
    const uint32_t piece = lane / 16 * 32 + lane % 4 * 8;
    const uint32_t last = (uint32_t)K - 8;
    for (int s = s0; s < s1; s += U) {
        typename W::Frag a[U][RT];
        u32x4 b[U][NT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t k = min((uint32_t)min(s + u, s1 - 1) * kStep + piece, last);
#pragma unroll
            for (int r = 0; r < RT; ++r) a[u][r] = W::load(base[r], row[r], K, k);
#pragma unroll
            for (int c = 0; c < NT; ++c) b[u][c] = *reinterpret_cast<const u32x4*>(x + (col[c] + k * 2));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s + u >= s1) continue;  // uniform
            if ((s + u + 1) * kStep > K && (uint32_t)(s + u) * kStep + piece > last) {
#pragma unroll
                for (int r = 0; r < RT; ++r) a[u][r] = W::zero();
#pragma unroll
                for (int c = 0; c < NT; ++c) b[u][c] = u32x4{0u, 0u, 0u, 0u};
            }
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const bf16x8 av = W::values(a[u][r]);
#pragma unroll
                for (int c = 0; c < NT; ++c)
                    acc[r][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, __builtin_bit_cast(bf16x8, b[u][c]),
                                                                        acc[r][c], 0, 0, 0);
            }
        }
    }
}

// The product of row l / 16 with column l % 16 / 4, in all four lanes of the
// quad: segment s of both is accumulator s of the quad's lane s.
__device__ __forceinline__ float diagonal_sum(const f32x4& a) {
    const uint32_t s = threadIdx.x % 4;
    const float v = s < 2 ? (s == 0 ? a[0] : a[1]) : (s == 2 ? a[2] : a[3]);
    return __builtin_bit_cast(float, group_reduce<4, Op::FAdd>(__builtin_bit_cast(uint32_t, v)));
}

}  // namespace moe
