// What the kernels share that write e4m3 values with a power of two (UE8M0) for every block.
#pragma once

#include "kgw_device.h"

namespace kgw {

// Biased UE8M0 exponent of the smallest 2^k with amax <= 448 * 2^k, from the
// fp32 bits of amax (amax = 1.f * 2^E; 448 = 1.75 * 2^8: k = E - 8 when
// 1.f <= 1.75, else E - 7), clamped to [1, 254]; 127 for zero.
__device__ __forceinline__ uint32_t e8m0_for_amax(float amax) {
    const uint32_t bits = __builtin_bit_cast(uint32_t, amax);
    if (bits == 0u) return 127u;
    const int E = (int)(bits >> 23) - 127;               // subnormal amax gives -127: clamps to 1
    const int k = E - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    const int e = k + 127;
    return (uint32_t)(e < 1 ? 1 : (e > 254 ? 254 : e));
}

// 2^(127 - e) as an fp32, for e in [1, 254] (normal for every e a finite bf16
// block can produce; e = 254 would need amax above the bf16 range).
__device__ __forceinline__ float inv_scale(uint32_t e) {
    const uint32_t field = 254u - e;
    return __builtin_bit_cast(float, field == 0u ? 0x00400000u : (field << 23));
}

// Reductions over an aligned group of G lanes (4, 8 or 16) inside one 16-lane
// row, on the DPP data paths (no LDS round trip): swaps within quads (lanes
// xor 1, xor 2), then the half-row mirror (lane i <-> 7 - i of each 8) and the
// row mirror (i <-> 15 - i); after each step every lane holds the combination
// over its group so far, so the mirrors join whole sub-groups.
template <int CTRL>
__device__ __forceinline__ int dpp_mov(int v) {
    return __builtin_amdgcn_mov_dpp(v, CTRL, 0xF, 0xF, false);
}
constexpr int kDppXor1 = 0xB1;        // quad_perm [1, 0, 3, 2]
constexpr int kDppXor2 = 0x4E;        // quad_perm [2, 3, 0, 1]
constexpr int kDppHalfMirror = 0x141;
constexpr int kDppMirror = 0x140;

template <int G>
__device__ __forceinline__ int group_or(int v) {
    static_assert(G == 4 || G == 8 || G == 16, "group of 4, 8 or 16 lanes");
    v |= dpp_mov<kDppXor1>(v);
    v |= dpp_mov<kDppXor2>(v);
    if constexpr (G >= 8) v |= dpp_mov<kDppHalfMirror>(v);
    if constexpr (G >= 16) v |= dpp_mov<kDppMirror>(v);
    return v;
}

// 2^(e - 127) as an fp32, for e in [1, 254] (always normal).
__device__ __forceinline__ float e8m0_scale(uint32_t e) { return __builtin_bit_cast(float, e << 23); }

// Unsigned maximum over an aligned group of G lanes (as group_or).
template <int G>
__device__ __forceinline__ uint32_t group_umax(uint32_t v) {
    static_assert(G == 4 || G == 8 || G == 16, "group of 4, 8 or 16 lanes");
    v = max(v, (uint32_t)dpp_mov<kDppXor1>((int)v));
    v = max(v, (uint32_t)dpp_mov<kDppXor2>((int)v));
    if constexpr (G >= 8) v = max(v, (uint32_t)dpp_mov<kDppHalfMirror>((int)v));
    if constexpr (G >= 16) v = max(v, (uint32_t)dpp_mov<kDppMirror>((int)v));
    return v;
}

// Four fp32 -> four e4m3fn bytes (little-endian order).
__device__ __forceinline__ int cvt4(float a, float b, float c, float d) {
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return __builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
}

}  // namespace kgw
