// Device helpers of the microscaled 4-bit matrices: conversion of one block
// of 32 elements, and the matrix instruction on blocks.
#pragma once
#include <type_traits>
#include <utility>

#include "common.hpp"
#include "iqlher.h"
#include "launch.hpp"

namespace iqlh {

typedef int mx_i8 __attribute__((ext_vector_type(8)));
typedef float mx_f4 __attribute__((ext_vector_type(4)));

template <int DT> struct MxFloat;
template <> struct MxFloat<IQLH_F32> {
    typedef float type;
    static IQLH_DEV float get(float x) { return x; }
    static IQLH_DEV float put(float x) { return x; }
};
template <> struct MxFloat<IQLH_BF16> {
    typedef uint16_t type;
    static IQLH_DEV float get(uint16_t x) { return bf2f(x); }
    static IQLH_DEV uint16_t put(float x) { return f2bf(x); }
};
template <> struct MxFloat<IQLH_F16> {
    typedef _Float16 type;
    static IQLH_DEV float get(_Float16 x) { return (float)x; }
    static IQLH_DEV _Float16 put(float x) { return (_Float16)x; }
};

// |x| as its bits: ordered as the values are, infinities and NaN on top
IQLH_DEV uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
IQLH_DEV uint32_t umax2(uint32_t a, uint32_t b) { return a > b ? a : b; }

// The scale byte of a block whose largest |x| has these bits, and the factor
// 1 / scale (a power of two, exact; 0 for a block that is not finite, whose
// codes are then forced to 0).  e - 2 = the byte of 2^(floor(log2 a) - 2) for
// a normal a of biased exponent e; subnormal a have e = 0 and take the
// smallest scale.
IQLH_DEV uint32_t mx4_scale(uint32_t amax) {
    const int e = (int)(amax >> 23) - 2;
    return amax >= 0x7F800000u ? 255u : (uint32_t)(e < 0 ? 0 : e);
}
IQLH_DEV float mx4_inverse(uint32_t scale) { return __uint_as_float((254u - scale) << 23); }  // scale <= 252
IQLH_DEV float mx4_scale_value(uint32_t scale) {
    return scale == 0u ? __uint_as_float(0x00400000u) : scale == 255u ? __uint_as_float(0x7FC00000u)
                                                                     : __uint_as_float(scale << 23);
}

// Eight values of a block times `inv` as eight codes, the first in the lowest
// bits.  The conversion instruction rounds to nearest, ties to even, and
// saturates at 6 (its scale operand is 1: the product with the power of two is
// exact, subnormals included).
IQLH_DEV uint32_t mx4_codes8(const float* x, float inv) {
    uint32_t w = 0u;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0] * inv, x[1] * inv, 1.f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2] * inv, x[3] * inv, 1.f, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4] * inv, x[5] * inv, 1.f, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6] * inv, x[7] * inv, 1.f, 3);
    return w;
}

// Eight neighbouring elements at p, which is aligned to its element only (the
// hardware takes 16-byte loads at any address), as they lie in memory.
// count < 8: the rest are 0, and all eight are read where that does not pass
// `end`.
template <int DT>
struct Eight {
    typedef typename MxFloat<DT>::type T;
    typedef T vec __attribute__((ext_vector_type(DT == IQLH_F32 ? 4 : 8), aligned(sizeof(T))));
    static constexpr int kVecs = DT == IQLH_F32 ? 2 : 1, kPer = 8 / kVecs;
    vec v[kVecs];
    IQLH_DEV void load(const T* p, int count, const T* end = nullptr) {
        if (count >= 8 || (count > 0 && end && p + 8 <= end)) {
#pragma unroll
            for (int i = 0; i < kVecs; ++i) v[i] = *(const vec*)(p + i * kPer);
            if (count < 8) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j / kPer][j % kPer] = j < count ? v[j / kPer][j % kPer] : T(0);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j / kPer][j % kPer] = j < count ? p[j] : T(0);
        }
    }
    IQLH_DEV void get(float* x) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = MxFloat<DT>::get(v[j / kPer][j % kPer]);
    }
};
template <int DT>
IQLH_DEV void load8(const typename MxFloat<DT>::type* p, int count, float* v) {
    Eight<DT> e;
    e.load(p, count);
    e.get(v);
}

// 16 rows from row0 on, blocks 4 step .. 4 step + 3, of a matrix in memory:
// this lane's 16 bytes and scale.  Rows past the end read the last one (their
// outputs are never stored), blocks past the end are zeros of scale 1.
struct RowFrag {
    const uint4* codes;
    const uint8_t* scales;
    int64_t kb;
    IQLH_DEV RowFrag(const Mx4Mat& q, int64_t row) : kb(q.kb()) {
        const int64_t r = row < q.rows ? row : q.rows - 1;
        codes = (const uint4*)q.codes + r * kb;
        scales = q.scales + r * kb;
    }
    IQLH_DEV void load(int64_t block, uint4& v, uint32_t& s) const {
        const bool in = block < kb;
        v = codes[in ? block : 0];
        s = scales[in ? block : 0];
        const uint32_t keep = in ? 0xFFFFFFFFu : 0u;
        v = uint4{v.x & keep, v.y & keep, v.z & keep, v.w & keep};
        s = in ? s : 127u;
    }
};

// largest of the four lanes 4j .. 4j + 3, in all of them
IQLH_DEV uint32_t quad_umax(uint32_t v) {
    v = umax2(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));  // quad_perm 1,0,3,2
    v = umax2(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));  // quad_perm 2,3,0,1
    return v;
}

// D[i][j] += sum over 128 k of A[i][k] B[j][k], both 16 x 128 in 4 bits with
// scales: lane l holds row l & 15, block l >> 4 (32 elements, 16 bytes) of
// each, the scale in byte 0; of D it holds column (l & 15) and rows
// 4 (l >> 4) + 0..3.  Checked against binary64 sums lane by lane, NaN scales
// included.
IQLH_DEV mx_f4 mx4_mma(uint4 a, uint4 b, mx_f4 c, uint32_t sa, uint32_t sb) {
    const mx_i8 a8 = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
    const mx_i8 b8 = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b8, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

// D[i][j] += sum over 64 k of A[i][k] B[j][k], both 32 x 64: lane l holds row
// l & 31, block l >> 5 of each, the scales in bytes OA, OB; of D column l & 31 and
// the rows 8 (e >> 2) + 4 (l >> 5) + (e & 3).
typedef float mx_f16 __attribute__((ext_vector_type(16)));
template <int OA, int OB>
IQLH_DEV mx_f16 mx4_mma32(uint4 a, uint4 b, mx_f16 c, uint32_t sa, uint32_t sb) {
    const mx_i8 a8 = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
    const mx_i8 b8 = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a8, b8, c, 4, 4, OA, (int)sa, OB, (int)sb);
}

// f(std::integral_constant<int, 0>) .. f(<N - 1>)
template <class F, int... I>
IQLH_DEV void static_for_impl(F&& f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>()), ...);
}
template <int N, class F>
IQLH_DEV void static_for(F&& f) {
    static_for_impl(f, std::make_integer_sequence<int, N>());
}

// bias[n .. n + 3], 0 without a bias and behind the last of N
IQLH_DEV void mx4_bias4(const Mx4Out& o, int64_t n, int64_t N, float* bias) {
    if (!o.bias) {
#pragma unroll
        for (int e = 0; e < 4; ++e) bias[e] = 0.f;
    } else if (n + 4 <= N) {
        typedef float f4u __attribute__((ext_vector_type(4), aligned(4)));
        const f4u w = *(const f4u*)(o.bias + n);
#pragma unroll
        for (int e = 0; e < 4; ++e) bias[e] = w[e];
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) bias[e] = n + e < N ? o.bias[n + e] : 0.f;
    }
}

// Four values rounded and stored at once, at any address of an element
template <int DT>
IQLH_DEV void mx4_put4(typename MxFloat<DT>::type* p, const float* y) {
    const mx_f4 v = {y[0], y[1], y[2], y[3]};
    if constexpr (DT == IQLH_F32) {
        typedef float f4u __attribute__((ext_vector_type(4), aligned(4)));
        *(f4u*)p = v;
    } else if constexpr (DT == IQLH_BF16) {
        typedef __bf16 b4 __attribute__((ext_vector_type(4)));
        typedef uint16_t u4 __attribute__((ext_vector_type(4), aligned(2)));
        *(u4*)p = __builtin_bit_cast(u4, __builtin_convertvector(v, b4));  // nearest even; a NaN stays one
    } else {
        typedef _Float16 h4 __attribute__((ext_vector_type(4), aligned(2)));
        *(h4*)p = h4{(_Float16)y[0], (_Float16)y[1], (_Float16)y[2], (_Float16)y[3]};
    }
}

// Four neighbouring outputs of a row, n .. n + 3 of N: bias, activation, one
// rounding, one store where all four are inside.
template <int DT>
IQLH_DEV void mx4_store4(const Mx4Out& o, int64_t m, int64_t n, int64_t N, mx_f4 acc) {
    typedef typename MxFloat<DT>::type T;
    if (n >= N) return;
    const float lowest = o.relu ? 0.f : -__builtin_huge_valf();
    float y[4];
    mx4_bias4(o, n, N, y);
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = __builtin_elementwise_maximum(acc[e] + y[e], lowest);  // a NaN stays
    T* p = (T*)o.p + m * o.ld + n;
    if (n + 4 <= N) {
        mx4_put4<DT>(p, y);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (n + e < N) p[e] = MxFloat<DT>::put(y[e]);
    }
}

}  // namespace iqlh
