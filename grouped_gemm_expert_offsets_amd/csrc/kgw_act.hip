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
// HBM bounds both directions from some megabytes on, a launch (4 us) and its issue below.  Measured, MI355X, every call with
// results of its own: bf16 swiglu of 65536 x 2048 forward 204 us (5.3 TB/s), gradient 211 us (5.1), with the activation again
// 265 us (5.1); 8192 x 4096 53, 57 and 71 us; 33024 x 768 43, 45 and 56 us; fp32, 16384 x 4096 181, 192 and 247 us.  A copy of such
// sizes moves 4.7 to 5.4 TB/s; the counters show that no byte moves twice.  Results that the last call left in the caches
// are quicker (8192 x 4096 44, 45 and 54 us).
#include <type_traits>

#include "kgw_layer.h"
#include "kgw_quant_device.h"
#include "kgw_row_io.h"

namespace kgw {
namespace {

constexpr int NT = 256, WAVES = NT / 64;
constexpr int MOST_ROWS = 64;                   // of a workgroup

// A lane's eight values of a block: eight in a row of 16-bit types, so that a load or store of 16 bytes a lane takes whole
// lines; for fp32 four of the block's first half and four of its second, for the same reason (with eight in a row, 16
// bytes in every 32 a load, the gradient of 33024 x 768 with the activation again took 99 us, with fours 80; the codes go by
// fours then too, which costs 8-bit results 2 to 6%).
template <int DT>
constexpr int kSecond = DT == kOutF32 ? 64 : 4;        // column of the second four, from the first's
template <int DT>
constexpr int kFours = DT == kOutF32 ? 2 : 1;          // runs of a lane

// As they are in memory; `in` tells which of the lane's runs the row has.
template <int DT>
struct Raw8 {
    i32x4 v[kFours<DT>];
};
template <int DT>
__device__ __forceinline__ Raw8<DT> load8_once(const char* p, const bool (&in)[2]) {
    Raw8<DT> r{};
    using Words = std::conditional_t<DT == kOutF32, Words4At4, Words4At2>;
#pragma unroll
    for (int i = 0; i < kFours<DT>; ++i)
        if (in[i]) r.v[i] = __builtin_nontemporal_load((const KGW_GLOBAL Words*)(p + 4 * kSecond<DT> * i));
    return r;
}
template <int DT>
__device__ __forceinline__ i32x2 load_codes(const uint8_t* p, const bool (&in)[2]) {
    i32x2 c = {0, 0};
    if constexpr (kFours<DT> == 2) {
        if (in[0]) c[0] = __builtin_nontemporal_load((const KGW_GLOBAL int*)p);
        if (in[1]) c[1] = __builtin_nontemporal_load((const KGW_GLOBAL int*)(p + kSecond<DT>));
    } else {
        if (in[0]) c = __builtin_nontemporal_load((const KGW_GLOBAL i32x2*)p);
    }
    return c;
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
__device__ __forceinline__ void store8(char* p, const float (&f)[8], const bool (&in)[2]) {
    using Words = std::conditional_t<DT == kOutF32, Words4At4, Words4At2>;
    if constexpr (DT == kOutF32) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const f32x4 v = {f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]};
            if (in[i]) store_result<STREAM, Words>(__builtin_bit_cast(i32x4, v), (KGW_GLOBAL Words*)(p + 4 * kSecond<DT> * i));
        }
    } else {
        const i32x4 v = {(int)pack_half2<DT>(f[0], f[1]), (int)pack_half2<DT>(f[2], f[3]),
                         (int)pack_half2<DT>(f[4], f[5]), (int)pack_half2<DT>(f[6], f[7])};
        if (in[0]) store_result<STREAM, Words>(v, (KGW_GLOBAL Words*)p);
    }
}
template <int DT, bool STREAM>
__device__ __forceinline__ void store_codes(uint8_t* p, i32x2 codes, const bool (&in)[2]) {
    if constexpr (kFours<DT> == 2) {
        if (in[0]) store_result<STREAM>((int)codes[0], (KGW_GLOBAL int*)p);
        if (in[1]) store_result<STREAM>((int)codes[1], (KGW_GLOBAL int*)(p + kSecond<DT>));
    } else {
        if (in[0]) store_result<STREAM>(codes, (KGW_GLOBAL i32x2*)p);
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

// Where this lane works: the workgroup's rows and blocks, and its 8 columns of some rows, `SECOND` between the fours.  A
// wave takes PASS rows at a time, 16 BLOCKS lanes each.
template <int BLOCKS, int SECOND>
struct Place {
    static constexpr int COLS = 128 * BLOCKS, PASS = 4 / BLOCKS;
    int64_t r0;             // first row of the workgroup
    int count;              // its rows
    int64_t b0;             // its first block of a half
    int blocks;             // its blocks
    int64_t nb;             // blocks of a half
    int64_t col;            // the lane's first column
    bool in[2];             // whether the row has its fours
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
        const int at = lane & (16 * BLOCKS - 1);
        col = chunk * COLS + (SECOND == 4 ? 8 * at : 128 * (at >> 4) + 4 * (at & 15));
        in[0] = col < p.inner;                  // inner is a multiple of 8
        in[1] = col + SECOND < p.inner;
        const int each = p.group_rows / WAVES;
        first = wave * each + lane / (16 * BLOCKS);
        passes = (max(0, min(each, count - wave * each)) + PASS - 1) / PASS;
        return true;
    }
    __device__ __forceinline__ void has(int r, bool (&here)[2]) const {
        here[0] = in[0] && r < count;
        here[1] = in[1] && r < count;
    }
};

template <int DT, bool GATED, int BLOCKS, bool STREAM_Y>
__global__ __launch_bounds__(NT) void act_kernel(ActParams p) {
    constexpr int S = RowElem<DT>::size, HALVES = GATED ? 2 : 1;
    __shared__ __attribute__((aligned(4))) uint8_t sc[HALVES + 1][BLOCKS][MOST_ROWS];
    const int tid = threadIdx.x, lane = tid & 63, block = (lane >> 4) & (BLOCKS - 1);
    using At = Place<BLOCKS, kSecond<DT>>;
    constexpr int PASS = At::PASS;
    At at;
    if (!at.init(p, tid)) return;
    const int64_t wide = HALVES * p.inner;
    auto load = [&](int r, Raw8<DT> (&raw)[HALVES]) __attribute__((always_inline)) {
        const char* row = (const char*)p.h + ((at.r0 + r) * p.ld_h + at.col) * S;
        bool in[2];
        at.has(r, in);
        if (in[0]) {
#pragma unroll
            for (int k = 0; k < HALVES; ++k) raw[k] = load8_once<DT>(row + k * p.inner * S, in);
        } else {
#pragma unroll
            for (int k = 0; k < HALVES; ++k) raw[k] = Raw8<DT>{};
        }
    };
    Raw8<DT> now[HALVES], next[HALVES];
    if (at.passes > 0) load(at.first, now);
    for (int i = 0; i < at.passes; ++i) {
        const int r = at.first + i * PASS;
        bool in[2];
        at.has(r, in);
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
                store_codes<DT, true>(p.saved + row * wide + k * p.inner + at.col, codes, in);
                if ((lane & 15) == 0) sc[k][block][r] = (uint8_t)e;
            }
        }
        if (p.y_scales) {
            i32x2 codes;
            const uint32_t e = quantise8(y, codes);
            store_codes<DT, STREAM_Y>((uint8_t*)p.y + row * p.inner + at.col, codes, in);
            if ((lane & 15) == 0) sc[HALVES][block][r] = (uint8_t)e;
        } else {
            store8<DT, STREAM_Y>((char*)p.y + (row * p.inner + at.col) * S, y, in);
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
    using At = Place<BLOCKS, kSecond<DT>>;
    constexpr int PASS = At::PASS;
    At at;
    if (!at.init(p, tid)) return;
    const int64_t wide = HALVES * p.inner;
    struct Row {
        i32x2 codes[HALVES];
        uint32_t scale[HALVES];
        Raw8<DT> dy;
    };
    auto load = [&](int r, Row& raw) __attribute__((always_inline)) {
        const int64_t row = at.r0 + r;
        bool in[2];
        at.has(r, in);
        if (!in[0]) {
            raw = Row{};
            return;
        }
        raw.dy = load8_once<DT>((const char*)p.dy + (row * p.ld_dy + at.col) * S, in);
#pragma unroll
        for (int k = 0; k < HALVES; ++k) {
            raw.codes[k] = load_codes<DT>(p.saved + row * wide + k * p.inner + at.col, in);
            raw.scale[k] = *(const KGW_GLOBAL uint8_t*)(p.saved_scales + (k * at.nb + at.b0 + block) * p.rows + row);
        }
    };
    Row now, next;
    if (at.passes > 0) load(at.first, now);
    for (int i = 0; i < at.passes; ++i) {
        const int r = at.first + i * PASS;
        bool in[2];
        at.has(r, in);
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
                store_codes<DT, STREAM>((uint8_t*)p.dh + to, codes, in);
                if ((lane & 15) == 0) sc[k][block][r] = (uint8_t)e;
            } else {
                store8<DT, STREAM>((char*)p.dh + to * S, d[k], in);
            }
        }
        if (p.y_scales) {
            i32x2 codes;
            const uint32_t e = quantise8(y, codes);
            store_codes<DT, STREAM_Y>((uint8_t*)p.y + row * p.inner + at.col, codes, in);
            if ((lane & 15) == 0) sc[HALVES][block][r] = (uint8_t)e;
        } else if (p.y) {
            store8<DT, STREAM_Y>((char*)p.y + (row * p.inner + at.col) * S, y, in);
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

// Results of this and more go past the caches' retention: the Infinity Cache's 256 MB could not hold them for the product
// that reads them next.  bf16 swiglu, every call with results of its own (65536 x 2048, y 0.27 GB, dh 0.54): forward 215 us, past the
// caches 204; gradient 219 and 211, with the activation again 274 and 265; fp32 16384 x 4096 190 and 182, 201 and 192, 259 and
// 248.  Smaller ones may still be there when they are read, or written anew (32768 x 2048, y of 0.13 GB written every
// second time: 87 us, past the caches 104).
constexpr int64_t kStreamBytes = (int64_t)256 << 20;

template <int DT, bool GATED, int BLOCKS>
void launch_blocks(const ActParams& p, bool grad, unsigned grid, hipStream_t stream) {
    const auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(grid), dim3(NT), 0, stream, p); };
    const int64_t values = p.rows * p.inner, S = RowElem<DT>::size;
    const bool y = p.y && values * (p.y_scales ? 1 : S) >= kStreamBytes;
    if (!grad) {
        if (y) go(act_kernel<DT, GATED, BLOCKS, true>);
        else go(act_kernel<DT, GATED, BLOCKS, false>);
    } else {
        if (y) go(act_grad_kernel<DT, GATED, BLOCKS, true, true>);
        else if (values * (GATED ? 2 : 1) * (p.dh_scales ? 1 : S) >= kStreamBytes) go(act_grad_kernel<DT, GATED, BLOCKS, true, false>);
        else go(act_grad_kernel<DT, GATED, BLOCKS, false, false>);
    }
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
