// gdn_e4m3.h -- 8-bit floats (OCP e4m3) and the fp32 scales that stand beside them, as the RMS norm, the quantiser
// and the feed-forward block write them: scale = max|x| / 448 over the values that share it (at least 2^-126; 1 where
// all are zero), q = e4m3(x / scale) to nearest even.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn_common.h"

namespace gdn {

constexpr float kE4m3Max = 448.f;

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

template <int kCtrl>
__device__ __forceinline__ uint32_t dpp_u(uint32_t x) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, kCtrl, 0xF, 0xF, true);
}
// Largest over the 16 lanes of a row, to each of them (bit patterns of absolute values: NaN above
// infinity above the rest).
__device__ __forceinline__ uint32_t umax_ln(uint32_t x) {
    x = max(x, dpp_u<0xB1>(x));
    x = max(x, dpp_u<0x4E>(x));
    x = max(x, dpp_u<0x141>(x));
    return max(x, dpp_u<0x140>(x));
}

// Two values in e4m3 (OCP), to nearest even, clamped to +-448; NaN stays NaN.
__device__ __forceinline__ float clamp_e4m3(float v) {
    return v > kE4m3Max ? kE4m3Max : (v < -kE4m3Max ? -kE4m3Max : v);
}
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(clamp_e4m3(a), clamp_e4m3(b), 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(clamp_e4m3(c), clamp_e4m3(d), w, true);
}
// The same for quotients by a scale of theirs, none of which lies above 448 by more than its rounding: half a step, 16, more
// would be the next value.
__device__ __forceinline__ uint32_t pack_e4m3_within(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}
__device__ __forceinline__ float scale_of(uint32_t amax_bits) {
    if (amax_bits == 0) return 1.f;
    const float s = __uint_as_float(amax_bits) / kE4m3Max;
    return s < 0x1p-126f ? 0x1p-126f : s;  // its reciprocal stays finite (NaN stays NaN)
}
// y / scale to nearest, from the scale's reciprocal: y inv is off by up to 1.5 fp32 steps, which put values that lie on
// an 8-bit tie to either side (0.2% of the values of rows of small whole numbers); what it leaves of y, times inv
// again, makes it the nearest in three operations (32,768 x 2,048 80.8 us, one product alone 80.1). What it leaves has to
// be an fp32 value itself: by scales near fp32's smallest normal one (below 2^-120 or so) it fell under 2^-149 and was lost, ties
// with it; scales below 2^-100 and their values are taken 2^64 times as large. An infinite scale
// has inv = 0, and its finite values are 0 / inf = 0: with 0 in place of the scale nothing is added to them.
struct Divisor {
    float scale, inv;
    bool tiny;
    __device__ __forceinline__ explicit Divisor(float s) : tiny(s < 0x1p-100f) {
        if (tiny) s *= 0x1p64f;
        inv = 1.f / s;
        scale = inv == 0.f ? 0.f : s;
    }
    template <int N>
    __device__ __forceinline__ void quotients(float (&y)[N]) const {
        if (__builtin_expect(tiny, 0))
#pragma unroll
            for (int i = 0; i < N; ++i) y[i] *= 0x1p64f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float q = y[i] * inv;
            y[i] = fmaf(fmaf(-q, scale, y[i]), inv, q);
        }
    }
};

// 8 bytes of 8-bit values, of which the lane owns those from `skip` on.
template <bool kOdd>
__device__ __forceinline__ void store_e4m3(uint8_t* p, uint32_t lo, uint32_t hi, int skip) {
    if (!kOdd || skip == 0) {
        typedef uint32_t words __attribute__((ext_vector_type(2), aligned(1)));
        __builtin_nontemporal_store(words{lo, hi}, reinterpret_cast<words*>(p));
        return;
    }
#pragma unroll
    for (int i = 1; i < 8; ++i)
        if (i >= skip) p[i] = (uint8_t)((i < 4 ? lo : hi) >> (8 * (i & 3)));
}

}  // namespace gdn
