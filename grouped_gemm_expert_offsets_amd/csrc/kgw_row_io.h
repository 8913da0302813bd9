// Elements of a row of fp32, bf16 or fp16, four or eight at a time, at element alignment (gfx950 takes wide global
// accesses at any element-aligned address), and sums and maxima over the lanes that share a row.
#pragma once

#include "kgw_device.h"
#include "kgw_quant_device.h"

namespace kgw {

template <int DT>
struct RowElem {
    static constexpr int size = DT == kOutF32 ? 4 : 2;
};

typedef i32x4 Words4At2 __attribute__((aligned(2)));
typedef i32x4 Words4At4 __attribute__((aligned(4)));
typedef i32x2 Words2At2 __attribute__((aligned(2)));
#define KGW_GLOBAL __attribute__((address_space(1)))

template <int DT>
__device__ __forceinline__ float load_elem(const char* p) {
    if constexpr (DT == kOutF32) return *(const KGW_GLOBAL float*)p;
    else return half_lo<DT>((uint32_t) * (const KGW_GLOBAL uint16_t*)p);
}
template <int DT>
__device__ __forceinline__ void store_elem(char* p, float f) {
    if constexpr (DT == kOutF32) *(KGW_GLOBAL float*)p = f;
    else *(KGW_GLOBAL uint16_t*)p = (uint16_t)pack_half2<DT>(f, 0.0f);
}

template <int DT>
__device__ __forceinline__ void load4(const char* p, float (&f)[4]) {
    if constexpr (DT == kOutF32) {
        const f32x4 v = __builtin_bit_cast(f32x4, *(const KGW_GLOBAL Words4At4*)p);
#pragma unroll
        for (int c = 0; c < 4; ++c) f[c] = v[c];
    } else {
        const i32x2 v = *(const KGW_GLOBAL Words2At2*)p;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            f[2 * c] = half_lo<DT>((uint32_t)v[c]);
            f[2 * c + 1] = half_hi<DT>((uint32_t)v[c]);
        }
    }
}
template <int DT>
__device__ __forceinline__ void store4(char* p, const float (&f)[4]) {
    if constexpr (DT == kOutF32) {
        const f32x4 v = {f[0], f[1], f[2], f[3]};
        *(KGW_GLOBAL Words4At4*)p = __builtin_bit_cast(i32x4, v);
    } else {
        const i32x2 v = {(int)pack_half2<DT>(f[0], f[1]), (int)pack_half2<DT>(f[2], f[3])};
        *(KGW_GLOBAL Words2At2*)p = v;
    }
}

// Combines a value over the L lanes that share a row: swaps within quads, then the half-row mirror and the row mirror (as in
// kgw_quant_device.h).  After each step every lane holds the combination over its group so far, in an order that is the
// same for all of its lanes up to commuting, so every lane ends with the same bits.  Groups of 64 go on through the
// LDS crossbar.
// (bound_ctrl lets the compiler make the move part of the instruction that takes its result; no lane is out of bounds)
template <int CTRL>
__device__ __forceinline__ int lane_dpp(int v) { return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, true); }
template <int CTRL>
__device__ __forceinline__ float lane_dpp(float v) {
    return __builtin_bit_cast(float, lane_dpp<CTRL>(__builtin_bit_cast(int, v)));
}
template <int L, class T, class F>
__device__ __forceinline__ T over_lanes(T v, F f) {
    static_assert(L == 4 || L == 8 || L == 16 || L == 64, "lanes of a row");
    v = f(v, lane_dpp<kDppXor1>(v));
    v = f(v, lane_dpp<kDppXor2>(v));
    if constexpr (L >= 8) v = f(v, lane_dpp<kDppHalfMirror>(v));
    if constexpr (L >= 16) v = f(v, lane_dpp<kDppMirror>(v));
    if constexpr (L == 64) {
        v = f(v, __shfl_xor(v, 16));
        v = f(v, __shfl_xor(v, 32));
    }
    return v;
}
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
    return over_lanes<L>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
    return over_lanes<L>(v, [](float a, float b) { return a + b; });
}
template <int L>
__device__ __forceinline__ int lanes_sum(int v) {
    return over_lanes<L>(v, [](int a, int b) { return a + b; });
}
template <int L>
__device__ __forceinline__ int lanes_max(int v) {
    return over_lanes<L>(v, [](int a, int b) { return max(a, b); });
}
template <int L>
__device__ __forceinline__ int lanes_min(int v) {
    return over_lanes<L>(v, [](int a, int b) { return min(a, b); });
}

// 2^x and 1 / x to about one step of fp32.
__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float reciprocal(float x) { return __builtin_amdgcn_rcpf(x); }
constexpr float kLog2e = 1.44269504088896340736f;
// 1 / (1 + e^-x): 0 and 1 at the infinities
__device__ __forceinline__ float sigmoid_of(float x) { return reciprocal(1.0f + exp2_of(-kLog2e * x)); }

}  // namespace kgw
