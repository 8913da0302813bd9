// Device code shared by the Newton-Schulz kernels: the planes' scales, loading of G and small helpers.
#pragma once

#include <type_traits>
#include <utility>

#include "kgw_device.h"
#include "kgw_layer.h"

namespace kgw {

// The planes of X, A = X X^T and B = b A + c A A hold them times powers of two, chosen per matrix and step so that
// a matrix as large as its bound allows comes to 2^13 .. 2^14, 2^10 .. 2^12 and 2^8 .. 2^9: well inside fp16's range
// above, and with as much room as there is below, where planes lose bits from 2^-3 on.  The power of A is that of X
// squared times this.
constexpr float kGramScale = 0x1p-16f;

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

// What the first iterate multiplies G by, 2^(13 - e) / (|G|_F + eps), in two factors: where the norm is near either end
// of fp32's range the quotient may leave it, and G is first brought nearer by a power of two.
struct FirstScale {
    float before, scale;
    bool unit;              // |X_0| is 1 but for rounding: the scales that the host made hold
    SingularBound bound;
    __device__ __forceinline__ float of(float g) const { return as_fp32(g * before * scale); }
};
__device__ __forceinline__ FirstScale scale_of_norm(double norm, float eps) {
    const double d = norm + (double)eps, inverse = 1.0 / d;
    FirstScale f;
    // |X_0| = norm / d, far below 1 where eps is what counts; a zero matrix, infinities and NaN go with the usual ones
    const double first = norm * inverse;
    f.unit = __builtin_amdgcn_readfirstlane(!(first > 0.0 && first < 1.0 - 0x1p-20));       // the same in all lanes
    f.bound = unit_bound(1.0f);
    if (!f.unit) {
        f.bound.m = 2.0f * (float)__builtin_frexp(first, &f.bound.e);
        f.bound.plane = --f.bound.e;
    }
    const int nearer = norm < 0x1p-100 ? 100 : norm > 0x1p100 ? -60 : 0;
    f.before = __builtin_ldexpf(1.0f, nearer);
    f.scale = (float)__builtin_ldexp(inverse, 13 - f.bound.e - nearer);
    if (norm == 0.0 && d > 0.0) f.scale = 1.0f;             // zeros stay zeros, however small eps is
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

// The usual scales of all steps of matrix b, by one wave, as early as it can: loading kernel arguments lane by lane takes long.
__device__ __forceinline__ void write_unit_scales(const NewtonParams& p, const NewtonCoefficients& co, int b) {
    const int lane = threadIdx.x & 63;
    if (lane < p.steps) p.scales[(int64_t)b * kNewtonMaxSteps + lane] = co.unit[lane];
}
// The others, by the same wave afterwards.
__device__ __forceinline__ void write_scales(const NewtonParams& p, const NewtonCoefficients& co, int b, const FirstScale& scale) {
    const int lane = threadIdx.x & 63;
    if (co.measured) {
        if (lane == 0) p.planes[b] = scale.bound.plane;
        return;
    }
    if (scale.unit) return;
    SingularBound s = scale.bound;
    for (int step = 0; step < p.steps; ++step) {
        const StepScales r = step_scales(s, co.v + 3 * step, step + 1 == p.steps);
        if (lane == step) p.scales[(int64_t)b * kNewtonMaxSteps + step] = r;     // the lane that wrote the usual ones
    }
}

// The bound that the plane of A gives, from the sum of its squares: the largest singular value is at most the square
// root of |A|_F, and at least r^(-1/4) of that.
__device__ __forceinline__ SingularBound measured_bound(double squares, int plane) {
    // the plane holds A times 2^(10 - 2 plane)
    const double s = __builtin_sqrt(__builtin_sqrt(squares));
    SingularBound f = unit_bound(1.0f);
    f.e = f.plane = plane;                                  // of zeros, infinities and NaN
    if (s > 0.0 && s < 0x1p100) {
        f.m = 2.0f * (float)__builtin_frexp(s, &f.e);
        f.e += plane - 6;
    }
    return f;
}

}  // namespace kgw
