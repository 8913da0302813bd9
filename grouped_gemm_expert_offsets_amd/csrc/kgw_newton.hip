// Newton-Schulz orthogonalisation of a batch of matrices (gfx950), the update of a
// weight gradient:
//
//     X_0 = G / (|G|_F + eps)                     (transposed when m > n, so r <= c)
//     A = X X^T,   B = b A + c A A,   X <- a X + B X,   `steps` times
//
// The iterate is held as two fp16 planes, X = (hi + lo) / 2^13: hi is X rounded to 11 bits, lo
// the remainder rounded again, 22 bits and more together, so the linear term a X, which multiplies
// small singular values by a at every step, loses nothing.  The products run on the matrix cores in fp16
// with fp32 sums:
//   one product each (results rounded to bf16): A = hi hi^T, B from fp16 A, B hi.  The
//     operands' rounding (2^-12) enters only through B X, which is small where the singular values are, and
//     leaves 0.5e-3 .. 1.7e-3 of the result's norm, at most bf16's own rounding (1.7e-3 rms);
//     bf16 operands would leave 4e-3 .. 2e-2.
//   three products each (fp32 and fp16 results): every matrix as hi + lo, hi hi + hi lo + lo hi;
//     the dropped lo lo is 2^-24 of the product.  1e-6 .. 1e-5, what fp32 arithmetic leaves.
// Powers of two keep the planes inside fp16's range: X * 2^13 (|X| <= 1.2 with the usual
// coefficients, below 8 allowed), A * 2^10 (below 64) and B * 2^7 (below 512).
//
// A and A A are symmetric: only tiles on and below the diagonal are computed and their mirror
// images written along.
#include <type_traits>

#include "kgw_device.h"
#include "kgw_internal.h"

namespace kgw {
namespace {

constexpr float kXScale = 8192.0f, kAScale = 1024.0f, kBScale = 128.0f;
constexpr int NT = 256;

// ----------------------------------------------------------------------------
// storage
// ----------------------------------------------------------------------------
// One product: a matrix of `cols` columns is a plane of halves, and the iterate's lo plane lies
// behind the whole batch of hi planes.  Three products: rows interleave 32 hi and 32 lo halves, so
// one 128-byte line holds both planes of 32 columns.
template <bool SPLIT>
__device__ __forceinline__ int64_t element(int64_t row, int64_t col, int64_t cols) {
    if constexpr (SPLIT) return row * 2 * cols + (col >> 5) * 64 + (col & 31);
    else return row * cols + col;
}

__device__ __forceinline__ float half_bits(uint16_t h) { return (float)__builtin_bit_cast(_Float16, h); }
__device__ __forceinline__ uint16_t to_half(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }

// ----------------------------------------------------------------------------
// |G|_F and the first iterate
// ----------------------------------------------------------------------------
template <int DT>
__device__ __forceinline__ float load_value(const void* p, int64_t i) {
    if constexpr (DT == kOutF32) return ((const float*)p)[i];
    else return half_lo<DT>((uint32_t)((const uint16_t*)p)[i]);
}

// Sum of squares of rows part, part + parts, ... of one matrix, in 64 bits: gradients may be so
// large or small that their squares leave fp32's range.
template <int DT>
__global__ __launch_bounds__(NT) void newton_norm_kernel(NewtonParams p) {
    __shared__ double sums[NT / 64];
    const int tid = threadIdx.x;
    const int64_t base = (int64_t)blockIdx.y * p.stride;
    double s = 0.0;
    for (int64_t row = blockIdx.x; row < p.m; row += kNewtonParts)
        for (int64_t col = tid; col < p.n; col += NT) {
            const double v = (double)load_value<DT>(p.G, base + row * p.ld + col);
            s += v * v;
        }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d);
    if ((tid & 63) == 0) sums[tid >> 6] = s;
    __syncthreads();
    if (tid == 0) p.parts[(int64_t)blockIdx.y * kNewtonParts + blockIdx.x] = (sums[0] + sums[1]) + (sums[2] + sums[3]);
}

// 2^13 / (|G|_F + eps) of matrix b, the same in every workgroup.
__device__ __forceinline__ float first_scale(const NewtonParams& p, int b) {
    double s = p.parts[(int64_t)b * kNewtonParts + (threadIdx.x & 63)];
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d);
    return (float)((double)kXScale / (__builtin_sqrt(s) + (double)p.eps));
}

// One 64 x 64 tile of the padded first iterate.
template <int DT, bool SPLIT, bool TALL>
__global__ __launch_bounds__(NT) void newton_first_kernel(NewtonParams p, int64_t R, int64_t C) {
    __shared__ float tile[64][65];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, b = blockIdx.z;
    const int64_t r0 = (int64_t)blockIdx.y * 64, c0 = (int64_t)blockIdx.x * 64;
    const float scale = first_scale(p, b);
    const int64_t base = (int64_t)b * p.stride;
    for (int i = wave; i < 64; i += NT / 64) {
        // TALL: row i of the tile read is row c0 + i of G
        const int64_t gr = (TALL ? c0 : r0) + i, gc = (TALL ? r0 : c0) + lane;
        const float v = gr < p.m && gc < p.n ? load_value<DT>(p.G, base + gr * p.ld + gc) * scale : 0.0f;
        if constexpr (TALL) tile[lane][i] = v;
        else tile[i][lane] = v;
    }
    __syncthreads();
    uint16_t* const hi = (uint16_t*)p.x[0] + (int64_t)b * R * C * (SPLIT ? 2 : 1);
    uint16_t* const lo = SPLIT ? hi + 32 : (uint16_t*)p.x[0] + ((int64_t)p.batch + b) * R * C;
    for (int i = wave; i < 64; i += NT / 64) {
        const float v = tile[i][lane];
        const uint16_t h = to_half(v);
        const int64_t at = element<SPLIT>(r0 + i, c0 + lane, C);
        hi[at] = h;
        lo[at] = to_half(v - half_bits(h));
    }
}

// One 64 x 64 tile of the result from the last iterate.
template <int DT, bool SPLIT, bool TALL>
__global__ __launch_bounds__(NT) void newton_last_kernel(NewtonParams p, const char* x, int64_t R, int64_t C) {
    __shared__ float tile[64][65];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, b = blockIdx.z;
    const int64_t r0 = (int64_t)blockIdx.y * 64, c0 = (int64_t)blockIdx.x * 64;
    const uint16_t* const hi = (const uint16_t*)x + (int64_t)b * R * C * (SPLIT ? 2 : 1);
    const uint16_t* const lo = SPLIT ? hi + 32 : (const uint16_t*)x + ((int64_t)p.batch + b) * R * C;
    for (int i = wave; i < 64; i += NT / 64) {
        const int64_t at = element<SPLIT>(r0 + i, c0 + lane, C);
        const float v = (half_bits(hi[at]) + half_bits(lo[at])) * (1.0f / kXScale);
        if constexpr (TALL) tile[lane][i] = v;
        else tile[i][lane] = v;
    }
    __syncthreads();
    for (int i = wave; i < 64; i += NT / 64) {
        const int64_t gr = (TALL ? c0 : r0) + i, gc = (TALL ? r0 : c0) + lane;
        if (gr >= p.m || gc >= p.n) continue;
        const int64_t at = ((int64_t)b * p.m + gr) * p.n + gc;
        if constexpr (DT == kOutF32) ((float*)p.out)[at] = tile[i][lane];
        else ((uint16_t*)p.out)[at] = (uint16_t)pack_half2<DT>(tile[i][lane], 0.0f);
    }
}

// ----------------------------------------------------------------------------
// the products
// ----------------------------------------------------------------------------
enum NewtonProduct { kGram, kSquare, kUpdate };

struct NewtonGemm {
    const char* left;       // (batch, R, K) rows of the product
    const char* right;      // gram, square: left again; update: the iterate (batch, K, C)
    char* out;              // gram: A; square: B; update: the next iterate
    const char* add;        // square: A; update: the iterate
    float scale, add_scale; // out = scale * product + add_scale * add
    int64_t rows, cols, k;  // padded sizes of the product
    int32_t batch, tiles_m, tiles_n, items;
    int32_t num_xcds;
};

// One TILE x TILE tile, 4 waves of a quarter each.  A stage of the K loop is a 128-byte line of
// every row of the left tile (64 halves of K, or 32 of both planes) and as many bytes of the right one,
// in two slots: while one is multiplied the next one lands.  Left tiles, and the right ones of the symmetric
// products, are read as K-contiguous rows with 16-byte chunk q of row i in slot q ^ ((i >> 1) & 7); the
// iterate's rows (K across them) through the transposing reads, chunk q of row k in slot
// q ^ 4 (k & 3).  Both keep every read free of bank conflicts.
template <int TILE, bool SPLIT, NewtonProduct KIND>
__global__ __launch_bounds__(NT, TILE == 256 ? 1 : 2) void newton_gemm_kernel(NewtonGemm p) {
    constexpr int WT = TILE / 2;                        // a wave's quarter
    constexpr int NB = WT / 32;                         // 32 x 32 blocks along it
    constexpr int STAGE = TILE * 128;                   // bytes of one operand's stage
    constexpr int LOADS = STAGE / 1024 / 4;             // direct loads a wave and operand
    constexpr int KSTAGE = SPLIT ? 32 : 64;
    constexpr int ROWB = TILE * (SPLIT ? 4 : 2);        // update: bytes of one k-row of the right tile
    constexpr int CPR = ROWB / 16;
    __shared__ __attribute__((aligned(1024))) char smem[4 * STAGE];
    lds_char* const lds = (lds_char*)smem;
    const uint32_t lds0 = lds_addr(smem);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave & 1, wn = wave >> 1;
    const int l32 = lane & 31, lhi = lane >> 5, g16 = lane >> 4, i16 = lane & 15;

    const int item = xcd_slot(blockIdx.x, gridDim.x, p.num_xcds);
    if (item >= p.items) return;
    const int per = p.items / p.batch;
    const int b = item / per;
    const int local = item - b * per;
    int tm, tn;
    if constexpr (KIND == kUpdate) {
        tile_coords(local, p.tiles_m, p.tiles_n, 4, tm, tn);
    } else {
        tm = (int)((__builtin_sqrtf(8.0f * (float)local + 1.0f) - 1.0f) * 0.5f);
        while ((tm + 1) * (tm + 2) / 2 <= local) ++tm;
        while (tm * (tm + 1) / 2 > local) --tm;
        tn = local - tm * (tm + 1) / 2;
    }
    const int64_t m0 = (int64_t)tm * TILE, n0 = (int64_t)tn * TILE;
    const int64_t ldl = p.k * (SPLIT ? 4 : 2);                                    // bytes of a left row
    const int64_t ldr = (KIND == kUpdate ? p.cols : p.k) * (SPLIT ? 4 : 2);       // of a right row
    const char* const left = p.left + ((int64_t)b * p.rows + m0) * ldl;
    const char* const right = KIND == kUpdate ? p.right + (int64_t)b * p.k * ldr + n0 * (SPLIT ? 4 : 2)
                                              : p.right + ((int64_t)b * p.rows + n0) * ldr;

    uint32_t l_off[LOADS], r_off[LOADS];
#pragma unroll
    for (int t = 0; t < LOADS; ++t) {
        const int row = (wave * LOADS + t) * 8 + (lane >> 3);
        const uint32_t chunk = (uint32_t)((lane & 7) ^ ((row >> 1) & 7));
        l_off[t] = (uint32_t)row * (uint32_t)ldl + chunk * 16u;
        if constexpr (KIND == kUpdate) {
            const int at = (wave * LOADS + t) * 64 + lane;
            const int krow = at / CPR;
            r_off[t] = (uint32_t)krow * (uint32_t)ldr + (uint32_t)((at % CPR) ^ ((krow & 3) << 2)) * 16u;
        } else {
            r_off[t] = (uint32_t)row * (uint32_t)ldr + chunk * 16u;
        }
    }
    const int stages = (int)(p.k / KSTAGE);
    const int64_t r_step = KIND == kUpdate ? KSTAGE * ldr : 128;
    auto load_stage = [&](int s) __attribute__((always_inline)) {
        const uint32_t dst = lds0 + (uint32_t)((s & 1) * 2 * STAGE) + (uint32_t)(wave * LOADS) * 1024u;
        const i32x4 rl = rsrc_words(left + (int64_t)s * 128);
        const i32x4 rr = rsrc_words(right + s * r_step);
#pragma unroll
        for (int t = 0; t < LOADS; ++t) {
            dma_16B(rl, l_off[t], dst + (uint32_t)t * 1024u);
            dma_16B(rr, r_off[t], dst + (uint32_t)(STAGE + t * 1024));
        }
    };

    // fragment q (0..3) of a stage: one product: K = 16 q ..; three: plane q >> 1, K = 16 (q & 1) ..
    const uint32_t l_row = (uint32_t)(wm * WT + l32) * 128u, r_row = (uint32_t)(wn * WT + l32) * 128u;
    const int sw = (l32 >> 1) & 7;
    const int kr = 8 * (g16 >> 1) + (i16 >> 2);
    const int cq = 2 * (g16 & 1) + ((i16 & 3) >> 1);
    auto read_left = [&](const lds_char* base, int q, int i) __attribute__((always_inline)) {
        return lds_load_16B(base, l_row + (uint32_t)i * 4096u + (uint32_t)(((2 * q + lhi) ^ sw) << 4));
    };
    auto read_right = [&](const lds_char* base, int q, int j) __attribute__((always_inline)) {
        if constexpr (KIND == kUpdate) {
            const int chunk = SPLIT ? (wn * (WT / 32) + j) * 8 + (q >> 1) * 4 + cq : wn * (WT / 8) + 4 * j + cq;
            const uint32_t at = (uint32_t)((SPLIT ? 16 * (q & 1) : 16 * q) + kr) * (uint32_t)ROWB +
                                (uint32_t)((chunk ^ ((i16 >> 2) << 2)) << 4) + (uint32_t)(i16 & 1) * 8u;
            const i16x4 lo = lds_read_tr16(base + STAGE, at);
            const i16x4 hi = lds_read_tr16(base + STAGE, at + 4 * ROWB);
            const i16x8 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            return __builtin_bit_cast(i32x4, v);
        } else {
            return lds_load_16B(base + STAGE, r_row + (uint32_t)j * 4096u + (uint32_t)(((2 * q + lhi) ^ sw) << 4));
        }
    };

    f32x16 acc[NB][NB];
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[j][i][r] = 0.0f;

    load_stage(0);
    for (int s = 0; s < stages; ++s) {
        wait_lgkmcnt0();
        wait_vmcnt<0>();                 // stage s has landed, for this wave's loads ...
        barrier_no_fence();              // ... and for all; all have read stage s - 1
        if (s + 1 < stages) load_stage(s + 1);
        const lds_char* const base = lds + (s & 1) * 2 * STAGE;
        if constexpr (!SPLIT) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                i32x4 l[NB], r[NB];
#pragma unroll
                for (int i = 0; i < NB; ++i) l[i] = read_left(base, q, i);
#pragma unroll
                for (int j = 0; j < NB; ++j) r[j] = read_right(base, q, j);
#pragma unroll
                for (int j = 0; j < NB; ++j)
#pragma unroll
                    for (int i = 0; i < NB; ++i) acc[j][i] = mfma_f16_32x32x16(r[j], l[i], acc[j][i]);
            }
        } else {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                i32x4 lh[NB], rh[NB], ll[NB], rl[NB];
#pragma unroll
                for (int i = 0; i < NB; ++i) lh[i] = read_left(base, q, i);
#pragma unroll
                for (int j = 0; j < NB; ++j) rh[j] = read_right(base, q, j);
#pragma unroll
                for (int j = 0; j < NB; ++j)
#pragma unroll
                    for (int i = 0; i < NB; ++i) acc[j][i] = mfma_f16_32x32x16(rh[j], lh[i], acc[j][i]);
#pragma unroll
                for (int j = 0; j < NB; ++j) rl[j] = read_right(base, q + 2, j);
#pragma unroll
                for (int j = 0; j < NB; ++j)
#pragma unroll
                    for (int i = 0; i < NB; ++i) acc[j][i] = mfma_f16_32x32x16(rl[j], lh[i], acc[j][i]);
#pragma unroll
                for (int i = 0; i < NB; ++i) ll[i] = read_left(base, q + 2, i);
#pragma unroll
                for (int j = 0; j < NB; ++j)
#pragma unroll
                    for (int i = 0; i < NB; ++i) acc[j][i] = mfma_f16_32x32x16(rh[j], ll[i], acc[j][i]);
            }
        }
    }

    // acc[j][i][4g + t] is the product at row m0 + wm WT + 32 i + l32 and column
    // n0 + wn WT + 32 j + 8 g + 4 lhi + t
    const int64_t matrix = p.rows * p.cols * (SPLIT ? 2 : 1);
    const int64_t lo_off = SPLIT ? 32 : (int64_t)p.batch * p.rows * p.cols;
    uint16_t* const out = (uint16_t*)p.out + (int64_t)b * matrix;
    const uint16_t* const add = (const uint16_t*)p.add + (int64_t)b * matrix;
    constexpr bool TWO = SPLIT || KIND == kUpdate;      // both planes are kept
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        const int64_t row = m0 + wm * WT + 32 * i + l32;
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int64_t col = n0 + wn * WT + 32 * j + 8 * g + 4 * lhi;
                const int64_t at = element<SPLIT>(row, col, p.cols);
                float v[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) v[t] = acc[j][i][4 * g + t] * p.scale;
                if constexpr (KIND != kGram) {
                    const i16x4 h = *(const i16x4*)(add + at);
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        float old = half_bits((uint16_t)h[t]);
                        if constexpr (TWO) old += half_bits(add[at + lo_off + t]);
                        v[t] += p.add_scale * old;
                    }
                }
                i16x4 h, l;
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const uint16_t hb = to_half(v[t]);
                    h[t] = (short)hb;
                    l[t] = (short)to_half(v[t] - half_bits(hb));
                }
                *(i16x4*)(out + at) = h;
                if constexpr (TWO) *(i16x4*)(out + at + lo_off) = l;
                if constexpr (KIND != kUpdate) {
                    if (tm != tn) {
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            const int64_t mirror = element<SPLIT>(col + t, row, p.cols);
                            out[mirror] = (uint16_t)h[t];
                            if constexpr (TWO) out[mirror + lo_off] = (uint16_t)l[t];
                        }
                    }
                }
            }
    }
}

template <int TILE, bool SPLIT>
void launch_steps(const NewtonParams& p, const NewtonPlan& plan, const float* co, int num_xcds, hipStream_t stream) {
    const int64_t R = plan.r, C = plan.c;
    NewtonGemm g;
    g.batch = p.batch;
    g.num_xcds = num_xcds;
    const int32_t tr = (int32_t)(R / TILE), tc = (int32_t)(C / TILE);
    auto run = [&](auto kernel) {
        const int grid = (g.items + 7) / 8 * 8;
        hipLaunchKernelGGL(kernel, dim3((uint32_t)grid), dim3(NT), 0, stream, g);
    };
    for (int s = 0; s < p.steps; ++s) {
        const char* const x = p.x[s & 1];
        g.rows = R;
        g.cols = R;
        g.tiles_m = g.tiles_n = tr;
        g.items = p.batch * (tr * (tr + 1) / 2);
        g.left = g.right = x;
        g.out = p.a;
        g.add = nullptr;
        g.k = C;
        g.scale = kAScale / (kXScale * kXScale);
        g.add_scale = 0.0f;
        run(newton_gemm_kernel<TILE, SPLIT, kGram>);
        g.left = g.right = p.a;
        g.out = p.b;
        g.add = p.a;
        g.k = R;
        g.scale = co[3 * s + 2] * (kBScale / (kAScale * kAScale));
        g.add_scale = co[3 * s + 1] * (kBScale / kAScale);
        run(newton_gemm_kernel<TILE, SPLIT, kSquare>);
        g.cols = C;
        g.tiles_n = tc;
        g.items = p.batch * tr * tc;
        g.left = p.b;
        g.right = x;
        g.add = x;
        g.out = p.x[(s + 1) & 1];
        g.scale = 1.0f / kBScale;
        g.add_scale = co[3 * s];
        run(newton_gemm_kernel<TILE, SPLIT, kUpdate>);
    }
}

template <bool SPLIT, bool TALL>
void launch_all(const NewtonParams& p, const NewtonPlan& plan, const float* co, int num_xcds, hipStream_t stream) {
    const dim3 norm_grid(kNewtonParts, (uint32_t)p.batch);
    const dim3 tiles((uint32_t)(plan.c / 64), (uint32_t)(plan.r / 64), (uint32_t)p.batch);
    auto first = [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        hipLaunchKernelGGL((newton_norm_kernel<DT>), norm_grid, dim3(NT), 0, stream, p);
        hipLaunchKernelGGL((newton_first_kernel<DT, SPLIT, TALL>), tiles, dim3(NT), 0, stream, p, plan.r, plan.c);
    };
    if (p.dtype == kOutBf16) first(std::integral_constant<int, kOutBf16>{});
    else if (p.dtype == kOutF16) first(std::integral_constant<int, kOutF16>{});
    else first(std::integral_constant<int, kOutF32>{});
    if (plan.tile == 256) launch_steps<256, SPLIT>(p, plan, co, num_xcds, stream);
    else launch_steps<128, SPLIT>(p, plan, co, num_xcds, stream);
    const char* const x = p.x[p.steps & 1];
    auto last = [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        hipLaunchKernelGGL((newton_last_kernel<DT, SPLIT, TALL>), tiles, dim3(NT), 0, stream, p, x, plan.r, plan.c);
    };
    if constexpr (!SPLIT) {
        last(std::integral_constant<int, kOutBf16>{});
    } else {
        if (p.out_dtype == kOutF16) last(std::integral_constant<int, kOutF16>{});
        else last(std::integral_constant<int, kOutF32>{});
    }
}

}  // namespace

NewtonPlan newton_plan(int32_t batch, int64_t m, int64_t n, int32_t out_dtype) {
    NewtonPlan plan;
    const int64_t r = m < n ? m : n, c = m < n ? n : m;
    plan.split = out_dtype != kOutBf16;
    plan.tall = m > n;
    // 256 x 256 tiles where the update alone has one for every CU, else four times as many of 128 x 128
    plan.tile = ((r + 255) / 256) * ((c + 255) / 256) * batch >= 256 ? 256 : 128;
    plan.r = (r + plan.tile - 1) / plan.tile * plan.tile;
    plan.c = (c + plan.tile - 1) / plan.tile * plan.tile;
    plan.x_bytes = (size_t)batch * plan.r * plan.c * 4;
    plan.a_bytes = (size_t)batch * plan.r * plan.r * (plan.split ? 4 : 2);
    plan.parts_bytes = ((size_t)batch * kNewtonParts * sizeof(double) + 1023) / 1024 * 1024;
    plan.total = plan.parts_bytes + 2 * plan.x_bytes + 2 * plan.a_bytes;
    return plan;
}

hipError_t launch_newton(const NewtonParams& p, const NewtonPlan& plan, const float* coefficients, int num_cus,
                         int num_xcds, hipStream_t stream) {
    if (plan.split) {
        if (plan.tall) launch_all<true, true>(p, plan, coefficients, num_xcds, stream);
        else launch_all<true, false>(p, plan, coefficients, num_xcds, stream);
    } else {
        if (plan.tall) launch_all<false, true>(p, plan, coefficients, num_xcds, stream);
        else launch_all<false, false>(p, plan, coefficients, num_xcds, stream);
    }
    return hipGetLastError();
}

}  // namespace kgw
