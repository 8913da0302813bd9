// Device code shared by the Newton-Schulz kernels: the planes' scales, loading of G and small helpers.
#pragma once

#include <type_traits>
#include <utility>

#include "kgw_device.h"
#include "kgw_layer.h"

namespace kgw {

constexpr float kXScale = 8192.0f, kAScale = 1024.0f, kBScale = 128.0f;

typedef __attribute__((__vector_size__(8 * sizeof(_Float16)))) _Float16 f16x8;
__device__ __forceinline__ f32x16 mfma_f16_32x32x16(i32x4 a, i32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Two floats as two halves, rounded to nearest even by one instruction (v_cvt_pk_f16_f32).
__device__ __forceinline__ uint32_t to_halves(float lo, float hi) {
    typedef __attribute__((ext_vector_type(2))) float f2;
    typedef __attribute__((ext_vector_type(2))) _Float16 h2;
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{lo, hi}), h2));
}

// x as it is in fp32: the compiler does not take its last operation together with what follows (a product and its
// conversion to half as one rounding), so that a value does not depend on the code around it.
__device__ __forceinline__ float as_fp32(float x) {
    asm("" : "+v"(x));
    return x;
}

// Two values as their halves and the halves of what is left of them.
struct HalfPair {
    uint32_t hi, lo;
};
__device__ __forceinline__ HalfPair split_pair(float a, float b) {
    HalfPair p;
    p.hi = to_halves(a, b);
    p.lo = to_halves(a - f16_lo(p.hi), b - f16_hi(p.hi));
    return p;
}

__device__ __forceinline__ float half_bits(uint16_t h) { return (float)__builtin_bit_cast(_Float16, h); }

// f(0), f(1), .. f(N - 1) with compile-time arguments: register arrays indexed by them stay in registers.
template <class F, int... I>
__device__ __forceinline__ void each_of(std::integer_sequence<int, I...>, F f) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void each(F f) {
    each_of(std::make_integer_sequence<int, N>{}, f);
}

// Eight consecutive elements of row `row` of matrix b, zeros past the matrix; rows may start at any element.
struct __attribute__((packed, aligned(2))) Halves8 { i32x4 v; };
struct __attribute__((packed, aligned(4))) Floats4 { f32x4 v; };
template <int DT>
__device__ __forceinline__ void load_eight(const NewtonParams& p, int b, int64_t row, int64_t col, float (&v)[8]) {
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = 0.0f;
    if (row >= p.m || col >= p.n) return;
    const int64_t at = (int64_t)b * p.stride + row * p.ld + col;
    if constexpr (DT == kOutF32) {
        const float* const from = (const float*)p.G + at;
        if (col + 8 <= p.n) {
            const f32x4 x = ((const __attribute__((address_space(1))) Floats4*)from)[0].v;
            const f32x4 y = ((const __attribute__((address_space(1))) Floats4*)from)[1].v;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                v[u] = x[u];
                v[4 + u] = y[u];
            }
        } else {
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (col + u < p.n) v[u] = from[u];
        }
    } else {
        const uint16_t* const from = (const uint16_t*)p.G + at;
        if (col + 8 <= p.n) {
            const i32x4 x = ((const __attribute__((address_space(1))) Halves8*)from)->v;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                v[2 * u] = half_lo<DT>((uint32_t)x[u]);
                v[2 * u + 1] = half_hi<DT>((uint32_t)x[u]);
            }
        } else {
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (col + u < p.n) v[u] = half_lo<DT>((uint32_t)from[u]);
        }
    }
}

// What the first iterate multiplies G by, 2^13 / (|G|_F + eps), in two factors: where the norm is so small that
// the quotient leaves fp32's range, G is first brought up by 2^100.
struct FirstScale {
    float before, scale;
    __device__ __forceinline__ float of(float g) const { return as_fp32(g * before * scale); }
};
__device__ __forceinline__ FirstScale scale_of_norm(double norm, float eps) {
    const double d = norm + (double)eps;
    FirstScale f;
    f.before = d < 0x1p-100 ? 0x1p100f : 1.0f;
    f.scale = (float)((double)kXScale / (d * (double)f.before));
    return f;
}
// The same in every wave of matrix b, from the parts of its norm.
__device__ __forceinline__ FirstScale first_scale(const NewtonParams& p, int b) {
    double s = 0.0;
    for (int i = threadIdx.x & 63; i < p.num_parts; i += 64) s += p.parts[(int64_t)b * kNewtonParts + i];
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d);
    return scale_of_norm(__builtin_sqrt(s), p.eps);
}

}  // namespace kgw
