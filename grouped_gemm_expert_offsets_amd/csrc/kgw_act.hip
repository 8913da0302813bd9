// The activation between the two expert products (gfx950), with its input kept for the backward pass in 8 bits:
//
//   swiglu  h (R, 2I) = [g | u]    y = g s u,  s = 1 / (1 + e^-g)     dg = dy u s (1 + g (1 - s)),  du = dy g s
//   relu2   h (R, I)               y = max(h, 0)^2                    dh = 2 max(h, 0) dy
//
// h is kept as e4m3 with one power of two for every 128 values of a row (the two halves of a gated row have blocks of their
// own): half of bf16's memory between the passes, and the operand format of the grouped fp8 products.  The backward pass
// reads it instead of h, and gives y again from it where that was not kept.  y and dh leave as rows of h's type or in
// 8 bits, as operands of the products that follow.
//
// 16 lanes hold a block, 8 values each; its largest magnitude goes round them on the DPP paths and every value is computed
// in fp32 and rounded once.  A workgroup takes 512, 256 or 128 columns, as they fit the row's length (blocks_of), of a run
// of rows; the scales, one byte for a block, collect in LDS and leave as runs of bytes along the rows, as their layout
// (blocks, R) has them.  Rows past the last offset belong to no expert: they are neither read nor written.
//
// HBM bounds both directions from some megabytes on, a launch (4 us) and its issue below.  Measured, bf16 swiglu, MI355X:
// 65536 x 2048 forward 166 us with a 16-bit result (6.5 TB/s), gradient 210 us, with the activation again 231 us (5.8);
// 8192 x 4096 forward 44 us (6.1 TB/s), gradient 45 us; 33024 x 768 forward 38.6 us, gradient 37.1 us.  A copy
// of such sizes moves 4.9 TB/s: reads outnumber writes here, which the memory takes faster.
#include <type_traits>

#include "kgw_layer.h"
#include "kgw_quant_device.h"
#include "kgw_row_io.h"

namespace kgw {
namespace {

constexpr int NT = 256, WAVES = NT / 64;
constexpr int MOST_ROWS = 64;                   // of a workgroup

// Eight values of a row as they are in memory.
template <int DT>
struct Raw8 {
    i32x4 v[DT == kOutF32 ? 2 : 1];
};
template <int DT>
__device__ __forceinline__ Raw8<DT> load8_once(const char* p) {
    Raw8<DT> r;
    using Words = std::conditional_t<DT == kOutF32, Words4At4, Words4At2>;
#pragma unroll
    for (int i = 0; i < (DT == kOutF32 ? 2 : 1); ++i)
        r.v[i] = __builtin_nontemporal_load((const KGW_GLOBAL Words*)(p + 16 * i));
    return r;
}
template <int DT>
__device__ __forceinline__ void values8(const Raw8<DT>& r, float (&f)[8]) {
    if constexpr (DT == kOutF32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __builtin_bit_cast(f32x4, r.v[i >> 2])[i & 3];
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = half_lo<DT>((uint32_t)r.v[0][i]);
            f[2 * i + 1] = half_hi<DT>((uint32_t)r.v[0][i]);
        }
    }
}
// Results, past the caches' retention or not (see kStreamBytes).
template <bool STREAM, class T>
__device__ __forceinline__ void store_result(T v, KGW_GLOBAL T* p) {
    if constexpr (STREAM) __builtin_nontemporal_store(v, p);
    else *p = v;
}
template <int DT, bool STREAM>
__device__ __forceinline__ void store8(char* p, const float (&f)[8]) {
    using Words = std::conditional_t<DT == kOutF32, Words4At4, Words4At2>;
    if constexpr (DT == kOutF32) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const f32x4 v = {f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]};
            store_result<STREAM, Words>(__builtin_bit_cast(i32x4, v), (KGW_GLOBAL Words*)(p + 16 * i));
        }
    } else {
        const i32x4 v = {(int)pack_half2<DT>(f[0], f[1]), (int)pack_half2<DT>(f[2], f[3]),
                         (int)pack_half2<DT>(f[4], f[5]), (int)pack_half2<DT>(f[6], f[7])};
        store_result<STREAM, Words>(v, (KGW_GLOBAL Words*)p);
    }
}

// Eight values of a block of 16 lanes to e4m3 bytes; the block's scale byte comes back.  Every lane of the
// block calls it (lanes past the row's end with zeros).
__device__ __forceinline__ uint32_t quantise8(const float (&f)[8], i32x2& codes) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __builtin_bit_cast(uint32_t, f[i]) & 0x7FFFFFFFu);
    top = group_umax<16>(top);
    if (top >= 0x7F800000u) {
        codes = i32x2{0x7F7F7F7F, 0x7F7F7F7F};
        return 255u;
    }
    const uint32_t e = e8m0_for_amax(__builtin_bit_cast(float, top));
    const float s = inv_scale(e);
    codes[0] = cvt4(f[0] * s, f[1] * s, f[2] * s, f[3] * s);
    codes[1] = cvt4(f[4] * s, f[5] * s, f[6] * s, f[7] * s);
    return e;
}
__device__ __forceinline__ void store_codes(uint8_t* p, i32x2 codes) {
    __builtin_nontemporal_store(codes, (KGW_GLOBAL i32x2*)p);
}
__device__ __forceinline__ void decode8(i32x2 codes, uint32_t scale, float (&f)[8]) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const float s = e8m0_to_f32(scale);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(codes[i], false), b = __builtin_amdgcn_cvt_pk_f32_fp8(codes[i], true);
        f[4 * i] = a[0] * s;
        f[4 * i + 1] = a[1] * s;
        f[4 * i + 2] = b[0] * s;
        f[4 * i + 3] = b[1] * s;
    }
}

__device__ __forceinline__ float relu_of(float x) { return x < 0.0f ? 0.0f : x; }     // NaN stays

// Rows that belong to an expert.
__device__ __forceinline__ int64_t live_rows(const ActParams& p) {
    if (!p.offsets) return p.rows;
    const int64_t last = p.offsets[p.num_experts - 1];
    return last < 0 ? 0 : min(last, p.rows);
}

// The workgroup's scale bytes of one tensor: (blocks, rows) in LDS to (blocks, p.rows), whole runs along the rows.
__device__ __forceinline__ void store_scales(const uint8_t (*sc)[MOST_ROWS], uint8_t* out, int64_t rows, int64_t b0,
                                             int blocks, int64_t r0, int count, int tid) {
    const int quads = (count + 3) / 4;
    for (int i = tid; i < blocks * quads; i += NT) {
        const int b = i / quads, r = 4 * (i - b * quads);
        uint8_t* dst = out + (b0 + b) * rows + r0 + r;
        if (r + 4 <= count) {
            typedef int Word __attribute__((aligned(1)));
            *(KGW_GLOBAL Word*)dst = *(const int*)&sc[b][r];
        } else {
            for (int k = r; k < count; ++k) dst[k - r] = sc[b][k];
        }
    }
}

// Where this lane works: the workgroup's rows and blocks, and its 8 columns of some rows.  A wave takes PASS rows at a
// time, 16 BLOCKS lanes each.
template <int BLOCKS>
struct Place {
    static constexpr int COLS = 128 * BLOCKS, PASS = 4 / BLOCKS;
    int64_t r0;             // first row of the workgroup
    int count;              // its rows
    int64_t b0;             // its first block of a half
    int blocks;             // its blocks
    int64_t nb;             // blocks of a half
    int64_t col;            // the lane's first column
    bool in;                // it has columns
    int first, passes;      // the lane's first row, and how often the wave goes on by PASS rows

    __device__ __forceinline__ bool init(const ActParams& p, int tid) {
        const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int64_t chunks = (p.inner + COLS - 1) / COLS;
        const int64_t run = blockIdx.x / chunks, chunk = blockIdx.x - run * chunks;
        r0 = run * p.group_rows;
        const int64_t left = live_rows(p) - r0;
        if (left <= 0) return false;
        count = (int)min<int64_t>(left, p.group_rows);
        nb = (p.inner + 127) / 128;
        b0 = chunk * BLOCKS;
        blocks = (int)min<int64_t>(BLOCKS, nb - b0);
        col = chunk * COLS + 8 * (lane & (16 * BLOCKS - 1));
        in = col < p.inner;                     // inner is a multiple of 8
        const int each = p.group_rows / WAVES;
        first = wave * each + lane / (16 * BLOCKS);
        passes = (max(0, min(each, count - wave * each)) + PASS - 1) / PASS;
        return true;
    }
    __device__ __forceinline__ bool has(int r) const { return in && r < count; }
};

template <int DT, bool GATED, int BLOCKS>
__global__ __launch_bounds__(NT) void act_kernel(ActParams p) {
    constexpr int S = RowElem<DT>::size, HALVES = GATED ? 2 : 1;
    __shared__ __attribute__((aligned(4))) uint8_t sc[HALVES + 1][BLOCKS][MOST_ROWS];
    const int tid = threadIdx.x, lane = tid & 63, block = (lane >> 4) & (BLOCKS - 1);
    constexpr int PASS = Place<BLOCKS>::PASS;
    Place<BLOCKS> at;
    if (!at.init(p, tid)) return;
    const int64_t wide = HALVES * p.inner;
    auto load = [&](int r, Raw8<DT> (&raw)[HALVES]) __attribute__((always_inline)) {
        const char* row = (const char*)p.h + ((at.r0 + r) * p.ld_h + at.col) * S;
#pragma unroll
        for (int k = 0; k < HALVES; ++k) {
            if (at.has(r)) raw[k] = load8_once<DT>(row + k * p.inner * S);
            else raw[k] = Raw8<DT>{};
        }
    };
    Raw8<DT> now[HALVES], next[HALVES];
    if (at.passes > 0) load(at.first, now);
    for (int i = 0; i < at.passes; ++i) {
        const int r = at.first + i * PASS;
        const bool in = at.has(r);
        if (i + 1 < at.passes) load(r + PASS, next);
        float f[HALVES][8], y[8];
#pragma unroll
        for (int k = 0; k < HALVES; ++k) values8<DT>(now[k], f[k]);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            if constexpr (GATED) {
                y[c] = f[0][c] * sigmoid_of(f[0][c]) * f[1][c];
            } else {
                const float v = relu_of(f[0][c]);
                y[c] = v * v;
            }
        }
        const int64_t row = at.r0 + r;
        if (p.saved) {
#pragma unroll
            for (int k = 0; k < HALVES; ++k) {
                i32x2 codes;
                const uint32_t e = quantise8(f[k], codes);
                if (in) store_codes(p.saved + row * wide + k * p.inner + at.col, codes);
                if ((lane & 15) == 0) sc[k][block][r] = (uint8_t)e;
            }
        }
        if (p.y_scales) {
            i32x2 codes;
            const uint32_t e = quantise8(y, codes);
            if (in) store_result<false>(codes, (KGW_GLOBAL i32x2*)((uint8_t*)p.y + row * p.inner + at.col));
            if ((lane & 15) == 0) sc[HALVES][block][r] = (uint8_t)e;
        } else if (in) {
            store8<DT, false>((char*)p.y + (row * p.inner + at.col) * S, y);
        }
#pragma unroll
        for (int k = 0; k < HALVES; ++k) now[k] = next[k];
    }
    if (!p.saved && !p.y_scales) return;
    __syncthreads();
    if (p.saved) {
#pragma unroll
        for (int k = 0; k < HALVES; ++k)
            store_scales(sc[k], p.saved_scales, p.rows, k * at.nb + at.b0, at.blocks, at.r0, at.count, tid);
    }
    if (p.y_scales) store_scales(sc[HALVES], p.y_scales, p.rows, at.b0, at.blocks, at.r0, at.count, tid);
}

template <int DT, bool GATED, int BLOCKS, bool STREAM, bool STREAM_Y>
__global__ __launch_bounds__(NT) void act_grad_kernel(ActParams p) {
    constexpr int S = RowElem<DT>::size, HALVES = GATED ? 2 : 1;
    __shared__ __attribute__((aligned(4))) uint8_t sc[HALVES + 1][BLOCKS][MOST_ROWS];
    const int tid = threadIdx.x, lane = tid & 63, block = (lane >> 4) & (BLOCKS - 1);
    constexpr int PASS = Place<BLOCKS>::PASS;
    Place<BLOCKS> at;
    if (!at.init(p, tid)) return;
    const int64_t wide = HALVES * p.inner;
    struct Row {
        i32x2 codes[HALVES];
        uint32_t scale[HALVES];
        Raw8<DT> dy;
    };
    auto load = [&](int r, Row& raw) __attribute__((always_inline)) {
        const int64_t row = at.r0 + r;
        if (at.has(r)) {
            raw.dy = load8_once<DT>((const char*)p.dy + (row * p.ld_dy + at.col) * S);
#pragma unroll
            for (int k = 0; k < HALVES; ++k) {
                raw.codes[k] = __builtin_nontemporal_load((const KGW_GLOBAL i32x2*)(p.saved + row * wide + k * p.inner + at.col));
                raw.scale[k] = *(const KGW_GLOBAL uint8_t*)(p.saved_scales + (k * at.nb + at.b0 + block) * p.rows + row);
            }
        } else {
            raw = Row{};
        }
    };
    Row now, next;
    if (at.passes > 0) load(at.first, now);
    for (int i = 0; i < at.passes; ++i) {
        const int r = at.first + i * PASS;
        const bool in = at.has(r);
        if (i + 1 < at.passes) load(r + PASS, next);
        float f[HALVES][8], dy[8], y[8], d[HALVES][8];
#pragma unroll
        for (int k = 0; k < HALVES; ++k) decode8(now.codes[k], now.scale[k], f[k]);
        values8<DT>(now.dy, dy);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            if constexpr (GATED) {
                const float g = f[0][c], u = f[1][c], s = sigmoid_of(g), silu = g * s;
                d[0][c] = dy[c] * u * (s + silu * (1.0f - s));
                d[1][c] = dy[c] * silu;
                y[c] = silu * u;
            } else {
                const float v = relu_of(f[0][c]);
                d[0][c] = 2.0f * v * dy[c];
                y[c] = v * v;
            }
        }
        const int64_t row = at.r0 + r;
#pragma unroll
        for (int k = 0; k < HALVES; ++k) {
            const int64_t to = row * wide + k * p.inner + at.col;
            if (p.dh_scales) {
                i32x2 codes;
                const uint32_t e = quantise8(d[k], codes);
                if (in) store_result<STREAM>(codes, (KGW_GLOBAL i32x2*)((uint8_t*)p.dh + to));
                if ((lane & 15) == 0) sc[k][block][r] = (uint8_t)e;
            } else if (in) {
                store8<DT, STREAM>((char*)p.dh + to * S, d[k]);
            }
        }
        if (p.y_scales) {
            i32x2 codes;
            const uint32_t e = quantise8(y, codes);
            if (in) store_result<STREAM_Y>(codes, (KGW_GLOBAL i32x2*)((uint8_t*)p.y + row * p.inner + at.col));
            if ((lane & 15) == 0) sc[HALVES][block][r] = (uint8_t)e;
        } else if (p.y && in) {
            store8<DT, STREAM_Y>((char*)p.y + (row * p.inner + at.col) * S, y);
        }
        now = next;
    }
    if (!p.dh_scales && !p.y_scales) return;
    __syncthreads();
    if (p.dh_scales) {
#pragma unroll
        for (int k = 0; k < HALVES; ++k)
            store_scales(sc[k], p.dh_scales, p.rows, k * at.nb + at.b0, at.blocks, at.r0, at.count, tid);
    }
    if (p.y_scales) store_scales(sc[HALVES], p.y_scales, p.rows, at.b0, at.blocks, at.r0, at.count, tid);
}

// A workgroup's blocks: as many as leave at most an eighth of the lanes idle (768 columns, six blocks: three workgroups
// of two; with four a half-empty one a row cost a quarter of the bandwidth).
int blocks_of(int64_t inner) {
    const int64_t nb = (inner + 127) / 128;
    for (int blocks = 4; blocks > 1; blocks /= 2)
        if (8 * nb >= 7 * ((nb + blocks - 1) / blocks * blocks)) return blocks;
    return 1;
}

// Gradients of this and more go past the caches' retention: half as much again as the Infinity Cache's 256 MB, so that the
// product that reads them does not find them there anyway.  dh goes where it and y together reach this, y where it
// does by itself: y then keeps the caches, and its product is the next to run.  bf16 swiglu, the gradient with the
// activation again: 65536 x 2048 (dh 0.54 GB, y 0.27) 274 us with neither, 264 with both, 231 with dh alone;
// 131072 x 2048 541 with neither, 524 with both.  Below it: 65536 x 2048 relu2 (0.27 GB) 110 -> 121 us.  fp32 rows are
// written every other 16 bytes a store and lose (204 -> 213 us), and so does the forward pass (y 0.54 GB: 367 -> 407 us).
constexpr int64_t kStreamBytes = (int64_t)384 << 20;
int64_t bytes_of_y(const ActParams& p) { return !p.y ? 0 : p.rows * p.inner * (p.y_scales ? 1 : 2); }
int64_t bytes_of_dh(const ActParams& p, int halves) { return p.rows * p.inner * halves * (p.dh_scales ? 1 : 2); }

template <int DT, bool GATED, int BLOCKS>
void launch_blocks(const ActParams& p, bool grad, unsigned grid, hipStream_t stream) {
    const auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(grid), dim3(NT), 0, stream, p); };
    const int64_t y = bytes_of_y(p), all = bytes_of_dh(p, GATED ? 2 : 1) + y;
    if (!grad) go(act_kernel<DT, GATED, BLOCKS>);
    else if (DT == kOutF32 || all < kStreamBytes) go(act_grad_kernel<DT, GATED, BLOCKS, false, false>);
    else if (y < kStreamBytes) go(act_grad_kernel<DT, GATED, BLOCKS, true, false>);
    else go(act_grad_kernel<DT, GATED, BLOCKS, true, true>);
}
template <int DT, bool GATED>
void launch_gated(const ActParams& p, bool grad, unsigned grid, hipStream_t stream) {
    const int blocks = blocks_of(p.inner);
    if (blocks == 4) launch_blocks<DT, GATED, 4>(p, grad, grid, stream);
    else if (blocks == 2) launch_blocks<DT, GATED, 2>(p, grad, grid, stream);
    else launch_blocks<DT, GATED, 1>(p, grad, grid, stream);
}
template <int DT>
void launch_dtype(const ActParams& p, bool gated, bool grad, unsigned grid, hipStream_t stream) {
    if (gated) launch_gated<DT, true>(p, grad, grid, stream);
    else launch_gated<DT, false>(p, grad, grid, stream);
}

}  // namespace

// Rows of a workgroup: 64 where that makes enough of them (runs of 64 scale bytes), fewer down to a pass of its waves.
int act_group_rows(int64_t rows, int64_t inner) {
    const int blocks = blocks_of(inner), least = WAVES * (4 / blocks);
    const int64_t chunks = (inner + 128 * blocks - 1) / (128 * blocks);
    for (int each = MOST_ROWS; each > least; each /= 2)
        if ((rows + each - 1) / each * chunks >= 1024) return each;
    return least;
}

int64_t act_grid(int64_t rows, int64_t inner) {
    const int64_t each = act_group_rows(rows, inner), cols = 128 * blocks_of(inner);
    return (rows + each - 1) / each * ((inner + cols - 1) / cols);
}

hipError_t launch_act(const ActParams& p, int dtype, bool gated, bool grad, hipStream_t stream) {
    const unsigned grid = (unsigned)act_grid(p.rows, p.inner);
    if (dtype == kOutF32) launch_dtype<kOutF32>(p, gated, grad, grid, stream);
    else if (dtype == kOutBf16) launch_dtype<kOutBf16>(p, gated, grad, grid, stream);
    else launch_dtype<kOutF16>(p, gated, grad, grid, stream);
    return hipGetLastError();
}

}  // namespace kgw
