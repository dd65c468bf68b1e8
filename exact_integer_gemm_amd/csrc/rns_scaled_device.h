// Device helpers of the block-scaled 8-bit operators: vector types, scale
// access, conversions and lane reductions.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/rns_scaled.h"

namespace rns {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef unsigned v2u __attribute__((ext_vector_type(2)));
typedef unsigned v4u __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

__host__ __device__ constexpr int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The factor an 8-bit exponent stands for: 2^(e - 127), NaN for 255.
__device__ __forceinline__ float e8m0_factor(uint32_t e) {
    const uint32_t bits = e == 0 ? 0x00400000u : (e == 255 ? 0x7fc00000u : e << 23);
    return __uint_as_float(bits);
}

// A scale as it is stored, and the factor it stands for.  Kernels that fetch
// ahead keep the first: working on a value is waiting for it, and for every
// load before it.
template <int ST>
__device__ __forceinline__ uint32_t load_scale(const void *s, int64_t i) {
    if constexpr (ST == RNS_T_F32) return ((const uint32_t *)s)[i];
    else return ((const uint8_t *)s)[i];
}
template <int ST>
__device__ __forceinline__ float scale_factor(uint32_t w) {
    if constexpr (ST == RNS_T_F32) return __uint_as_float(w);
    else return e8m0_factor(w);
}

// A block's product p (0 or 2^-25 .. 2^32 in magnitude) times both scales.
// By two multiplications p sa or sa sb can overflow, or fall below the smallest
// normal number, where p sa sb does neither; so the significands are
// multiplied, and the exponents added.
__device__ __forceinline__ float scaled(float p, float sa, float sb) {
    const float x = p * __builtin_amdgcn_frexp_mantf(sa) * __builtin_amdgcn_frexp_mantf(sb);
    return __builtin_amdgcn_ldexpf(x, __builtin_amdgcn_frexp_expf(sa) + __builtin_amdgcn_frexp_expf(sb));
}
// A scale as a power of two 2^(e - 127) that an instruction can apply to its
// operand, times the rest, which is below 2 and at least 1 where the scale's
// own exponent is one of LO .. HI (1 .. 253, so that the inverse is normal too).
struct Split {
    uint32_t e;
    float r;
    __device__ __forceinline__ float power() const { return __uint_as_float(e << 23); }
};
template <int LO, int HI>
__device__ __forceinline__ Split split_scale(float s) {
    const uint32_t e = min(max((__float_as_uint(s) >> 23) & 0xff, (uint32_t)LO), (uint32_t)HI);
    return Split{e, s * __uint_as_float((254 - e) << 23)};
}
// Where multiplications have to be few, scales are looked at first: with both
// within 2^-46 .. 2^46, or their product normal, two multiplications (or the
// one by the product) stay in range.
constexpr float kScaleLow = 1.42108547e-14f, kScaleHigh = 7.03687442e13f;         // 2^-46, 2^46
constexpr float kSmallestNormal = 1.17549435e-38f, kLargestFinite = 3.4028235e38f;
struct Extent {
    float low = kScaleHigh, high = kScaleLow;
    __device__ __forceinline__ void add(float s) {           // a NaN changes nothing, and needs no care
        low = fminf(low, fabsf(s));
        high = fmaxf(high, fabsf(s));
    }
    __device__ __forceinline__ bool beyond(float l, float h) const { return low < l || high > h; }
};

__device__ __forceinline__ uint32_t bf16_bits(float f) {
    const __bf16 h = (__bf16)f;                    // nearest, ties to even
    return __builtin_bit_cast(uint16_t, h);
}
__device__ __forceinline__ uint32_t f16_bits(float f) {
    const _Float16 h = (_Float16)f;
    return __builtin_bit_cast(uint16_t, h);
}
__device__ __forceinline__ float bf16_float(uint32_t b) { return __uint_as_float(b << 16); }
__device__ __forceinline__ float f16_float(uint32_t b) {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)b);
}

// Eight 8-bit values (two words), times a power of two of 2^-100 .. 2^100, as bfloat16, which holds every one of them.
template <int TYPE>
__device__ __forceinline__ v8bf widen8(uint32_t w0, uint32_t w1, float scale = 1.0f) {
    v2bf a, b, c, d;
    if constexpr (TYPE == RNS_T_E4M3) {
        a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, scale, false);
        b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, scale, true);
        c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, scale, false);
        d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, scale, true);
    } else {
        a = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w0, scale, false);
        b = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w0, scale, true);
        c = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w1, scale, false);
        d = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w1, scale, true);
    }
    return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// x from the lane that the DPP control names (every lane has a source here)
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}
constexpr int kRowRor = 0x120;                     // + n: rotate right by n in a row of 16 lanes

// The largest of a row of 16 lanes, in all of them.
__device__ __forceinline__ float row_max(float x) {
    x = fmaxf(x, dpp<kRowRor + 8>(x));
    x = fmaxf(x, dpp<kRowRor + 4>(x));
    x = fmaxf(x, dpp<kRowRor + 2>(x));
    return fmaxf(x, dpp<kRowRor + 1>(x));
}

}  // namespace rns
