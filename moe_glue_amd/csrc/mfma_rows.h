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

constexpr uint32_t kNowhere = 0x80000000u;  // an offset past the end of every buffer

// A wave-uniform offset that the compiler cannot see to be one.  (Pointers stay
// sums of a kernel argument and such an offset: then loads are global ones with
// a scalar base.)
__device__ __forceinline__ size_t uniform_offset(size_t v) {
    return (size_t)uniform((uint32_t)(v >> 32)) << 32 | uniform((uint32_t)v);
}
__device__ __forceinline__ int wave_index() { return (int)uniform(threadIdx.x / kWave); }

// Loads go through buffer resources: a lane's offset stays put, the step's is a
// scalar, and a lane that shall have zeros (a column past the last token, k past
// a row's end) takes an offset past the end, and gets them, instead of a branch.
// That is all the range check is used for: every other offset plus its step lies
// inside, whether or not the check counts the step.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, size_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0,
                                             (int)(uint32_t)(bytes < kNowhere ? bytes : kNowhere), kRawBufferWord3);
}

// A lane's part of one row in a step (Frag), and what its tile's rows carry
// over several steps (Scales).
struct Bf16Weights {
    static constexpr int STEP = 128;
    static constexpr int SUB = 1;          // MFMAs per step
    static constexpr int SCALE_STEPS = 0;  // steps of a scale load (0: no scales)
    using Frag = u32x4;
    struct Scales {};
    static __host__ __device__ __forceinline__ uint32_t bytes_of(uint32_t k) { return k * 2; }
    static __host__ __device__ __forceinline__ uint32_t row_scales(int) { return 0; }
    template <int CACHE>
    static __device__ __forceinline__ Frag load(__amdgpu_buffer_rsrc_t w, uint32_t lane, uint32_t step) {
        return __builtin_bit_cast(Frag, __builtin_amdgcn_raw_buffer_load_b128(w, (int)lane, (int)step, CACHE));
    }
    template <int M>
    static __device__ __forceinline__ bf16x8 values(const Frag& f, float) {
        return __builtin_bit_cast(bf16x8, f);
    }
};

// Scales: a lane fetches the bytes of four blocks, so that the 16 lanes of a row
// fetch 64 bytes, those of 8 steps.  The block of a lane in step j of the 8 is
// byte j * 8 + (4 q + s) / 2, which lane 2 j + q / 2 of the 16 holds: handed over
// through the LDS crossbar (ds_bpermute).  A byte load per lane and step instead
// takes 28 clocks, and finds its line gone from the first cache nearly every
// time.
struct Mxfp4Weights {
    static constexpr int STEP = 256;
    static constexpr int SUB = 2;
    static constexpr int SCALE_STEPS = 8;
    using Frag = u32x2;
    struct Scales {
        uint32_t now, next;
    };
    static __host__ __device__ __forceinline__ uint32_t bytes_of(uint32_t k) { return k / 2; }
    static __host__ __device__ __forceinline__ uint32_t row_scales(int K) { return (uint32_t)K / 32; }
    template <int CACHE>
    static __device__ __forceinline__ Frag load(__amdgpu_buffer_rsrc_t w, uint32_t lane, uint32_t step) {
        return __builtin_bit_cast(Frag, __builtin_amdgcn_raw_buffer_load_b64(w, (int)lane, (int)step, CACHE));
    }
    // The lane's four scale bytes of the 8 steps from `step` on, of the row whose
    // scales begin at p + row, in one dword at any byte address; at a row's end
    // the row's last dword, which shifted() puts right: later, when the load has
    // arrived.  A row shorter than a dword has the one step of first_scales().
    static __device__ __forceinline__ uint32_t scale_at(int step) {
        const uint32_t lane = threadIdx.x % kWave;
        return (uint32_t)step * (STEP / 32) + (lane / 16 * 4 + lane % 4) * 4;
    }
    static __device__ __forceinline__ uint32_t load_scales(const uint8_t* p, uint32_t row, int K, int step) {
        uint32_t v;
        __builtin_memcpy(&v, p + (row + min(scale_at(step), row_scales(K) - 4)), 4);
        return v;
    }
    static __device__ __forceinline__ uint32_t shifted(uint32_t v, int K, int step) {
        const uint32_t at = scale_at(step), n = row_scales(K);
        return n < 4 ? v : v >> ((at - min(at, n - 4)) % 4 * 8);
    }
    static __device__ __forceinline__ uint32_t first_scales(const uint8_t* p, uint32_t row, int K, int step) {
        const uint32_t n = row_scales(K);
        if (n >= 4) return load_scales(p, row, K, step);  // uniform
        return p[row] | p[row + n / 2] << 8 | p[row + n - 1] << 16;  // n = 1, 2, 3: every byte there is
    }
    // The lane's scale in step s of those 8, 2^(b - 127): its byte b is fp32's
    // exponent field; b = 0 is a subnormal, 255 is NaN.
    static __device__ __forceinline__ float scale(const Scales& f, int s) {
        const uint32_t lane = threadIdx.x % kWave;
        const uint32_t from = lane % 16 / 4 * 4 + lane / 32 + (uint32_t)(s / 2 * 16 + s % 2 * 2);
        const uint32_t four = (uint32_t)__builtin_amdgcn_ds_bpermute((int)(from * 4), (int)f.now);
        const uint32_t b = four >> (lane / 16 % 2 * 16 + lane % 4 / 2 * 8) & 0xFFu;
        return __builtin_bit_cast(float, b << 23);
    }
    template <int M>
    static __device__ __forceinline__ bf16x8 values(const Frag& f, float s) {
        const uint32_t v = f[M];
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

// The rows of RT tiles: tile r's rows 0 to last[r] <= 3 follow each other from
// byte at[r] of w0 (even r) or w1 (odd r) on, their scales from scales[r] on; all
// uniform.  Lanes of rows past the last take it again.
template <int RT>
struct RowTiles {
    uint32_t at[RT];
    const uint8_t* scales[RT];
    uint32_t last[RT];
};

// acc[r][c] += row tile r times column tile c over the steps [s0, s1) of K, both
// uniform.  col[c]: the byte offset of the lane's column in x, or kNowhere.
// The loads of U steps are in flight: a step's registers are loaded again, for
// the step U later, as soon as it is multiplied.  In a step that K ends inside,
// lanes past K hold zeros.  CACHE: the weight loads' cache bits, kCacheNt where
// no other wave will read them.  CT = 2: odd row tiles have columns of their own,
// col[1] (two products side by side, for the loads in flight); CT = 1: all share
// col[0].
template <class W, int RT, int NT, int U, int CACHE, int CT>
__device__ __forceinline__ void multiply_rows(__amdgpu_buffer_rsrc_t w0, __amdgpu_buffer_rsrc_t w1,
                                              const RowTiles<RT>& rows, __amdgpu_buffer_rsrc_t x,
                                              const uint32_t (&col)[CT][NT], int K, int s0, int s1,
                                              f32x4 (&acc)[RT][NT]) {
    constexpr int PIECE = W::STEP / 16;
    static_assert(PIECE == 8 * W::SUB, "a lane's piece is its MFMAs' k");
    const uint32_t lane = threadIdx.x % kWave;
    const uint32_t piece = (lane / 16 * 4 + lane % 4) * PIECE;
    const uint32_t row = lane % 16 / 4;
    uint32_t a_at[RT], sc_row[RT], b_at[CT][NT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        a_at[r] = min(row, rows.last[r]) * W::bytes_of((uint32_t)K) + W::bytes_of(piece);
        sc_row[r] = min(row, rows.last[r]) * W::row_scales(K);
    }
#pragma unroll
    for (int g = 0; g < CT; ++g)
#pragma unroll
        for (int c = 0; c < NT; ++c) b_at[g][c] = col[g][c] < kNowhere ? col[g][c] + piece * 2 : kNowhere;
    typename W::Frag a[U][RT];
    typename W::Scales sc[RT];
    u32x4 b[U][CT][NT][W::SUB];
    const int partial = K / W::STEP;  // the step that K ends inside, if it does
    const auto load = [&](auto index, int s, bool whole) {
        constexpr int u = decltype(index)::value;
        const uint32_t k = (uint32_t)s * W::STEP;
        const bool past = !whole && s == partial && k + piece >= (uint32_t)K;
#pragma unroll
        for (int r = 0; r < RT; ++r)
            a[u][r] = W::template load<CACHE>(r % 2 == 0 ? w0 : w1, past ? kNowhere : a_at[r],
                                              rows.at[r] + W::bytes_of(k));
#pragma unroll
        for (int g = 0; g < CT; ++g)
#pragma unroll
            for (int c = 0; c < NT; ++c)
#pragma unroll
                for (int m = 0; m < W::SUB; ++m)
                    b[u][g][c][m] = __builtin_bit_cast(
                        u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                   x, (int)((past ? kNowhere : b_at[g][c]) + m * 16), (int)(k * 2), 0));
    };
    const auto scales_at = [&](int s) {  // at a group's first step
        if constexpr (W::SCALE_STEPS > 0)
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                sc[r].now = W::shifted(sc[r].next, K, s);
                if (s + W::SCALE_STEPS < s1)
                    sc[r].next = W::load_scales(rows.scales[r], sc_row[r], K, s + W::SCALE_STEPS);
            }
    };
    const auto multiply = [&](auto index, int in_group) {
        constexpr int u = decltype(index)::value;
        float scale[RT] = {};
        if constexpr (W::SCALE_STEPS > 0)
#pragma unroll
            for (int r = 0; r < RT; ++r) scale[r] = W::scale(sc[r], in_group);
        unrolled<W::SUB>([&](auto sub) {
            constexpr int m = decltype(sub)::value;
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const bf16x8 av = W::template values<m>(a[u][r], scale[r]);
#pragma unroll
                for (int c = 0; c < NT; ++c)
                    acc[r][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        av, __builtin_bit_cast(bf16x8, b[u][r % CT][c][m]), acc[r][c], 0, 0, 0);
            }
        });
    };
    static_assert(W::SCALE_STEPS % U == 0, "a group of scales is whole rounds");
    constexpr int GROUP = W::SCALE_STEPS > 0 ? W::SCALE_STEPS : U;
    if (s0 >= s1) return;
    if constexpr (W::SCALE_STEPS > 0)
#pragma unroll
        for (int r = 0; r < RT; ++r) sc[r].next = W::first_scales(rows.scales[r], sc_row[r], K, s0);
    scales_at(s0);
    // Rounds of U steps.  The loads of a whole round are not under a condition:
    // behind one, the wait for a step's registers would have to assume that the
    // later loads were not issued, and drain the ones that were.
    if (s1 - s0 < U) {
        unrolled<U>([&](auto index) {
            if (s0 + index < s1) load(index, s0 + index, false);
        });
        unrolled<U>([&](auto index) {
            if (s0 + index < s1) multiply(index, index);
        });
        return;
    }
    unrolled<U>([&](auto index) { load(index, s0 + index, false); });
    const int whole = min(s1, partial);
    int s = s0;
    for (; s + 2 * U <= whole; s += U) {
        const int in_group = (s - s0) % GROUP;
        if (in_group == 0 && s > s0) scales_at(s);
        unrolled<U>([&](auto index) {
            multiply(index, in_group + index);
            load(index, s + U + index, true);
        });
    }
    const int in_group = (s - s0) % GROUP;
    if (in_group == 0 && s > s0) scales_at(s);
    unrolled<U>([&](auto index) {
        multiply(index, in_group + index);
        if (s + U + index < s1) load(index, s + U + index, false);
    });
    s += U;
    if (s >= s1) return;
    const int rest = (s - s0) % GROUP;
    if (rest == 0) scales_at(s);
    unrolled<U>([&](auto index) {
        if (s + index < s1) multiply(index, rest + index);
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
