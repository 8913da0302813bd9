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
    int32_t batch, tiles_m, tiles_n;
    int32_t items;          // workgroups with work
    int32_t whole;          // the first of them: one tile each; the others a quarter of one
    int32_t num_xcds;
};

// Item of workgroup bid of `items`: workgroups are dealt to the XCDs in turn, and one XCD's get a
// contiguous run of items, so that the tiles it works on at a time share panels in its L2.
__device__ __forceinline__ int item_of(int bid, int items, int num_xcds) {
    const int each = items / num_xcds, more = items - each * num_xcds, x = bid % num_xcds;
    return x * each + min(x, more) + bid / num_xcds;
}

// Tile `index` of a product with tiles_m x tiles_n tiles a matrix: all of them (update), or those on
// and below the diagonal.
template <NewtonProduct KIND>
__device__ __forceinline__ void tile_of(const NewtonGemm& p, int index, int& b, int& tm, int& tn) {
    const int per = KIND == kUpdate ? p.tiles_m * p.tiles_n : p.tiles_m * (p.tiles_m + 1) / 2;
    b = index / per;
    const int local = index - b * per;
    if constexpr (KIND == kUpdate) {
        tile_coords(local, p.tiles_m, p.tiles_n, 4, tm, tn);
    } else {
        tm = (int)((__builtin_sqrtf(8.0f * (float)local + 1.0f) - 1.0f) * 0.5f);
        while ((tm + 1) * (tm + 2) / 2 <= local) ++tm;
        while (tm * (tm + 1) / 2 > local) --tm;
        tn = local - tm * (tm + 1) / 2;
    }
}

// Rows x 32-column-group image of a wave's accumulators in LDS: 32 rows of W fp32, 16-byte chunk q
// of row r in slot q ^ (r & mask), so that rows of registers written and rows read back both spread over all banks.
template <int W>
__device__ __forceinline__ uint32_t image_at(int row, int chunk) {
    return (uint32_t)(row * W * 4 + ((chunk ^ (row & (W / 4 - 1))) << 4));
}

// Eight consecutive elements of one row of the result: v = product, then scaled, added to and stored
// as one or two planes of halves.
template <NewtonProduct KIND, bool TWO>
struct Addend {
    i32x4 hi, lo;
    __device__ __forceinline__ void load(const uint16_t* add, int64_t at, int64_t lo_off) {
        if constexpr (KIND != kGram) {
            hi = *(const gbl_i32x4*)(add + at);
            if constexpr (TWO) lo = *(const gbl_i32x4*)(add + at + lo_off);
        }
    }
};
template <NewtonProduct KIND, bool TWO>
__device__ __forceinline__ void store_eight(const NewtonGemm& p, const float (&v)[8], const Addend<KIND, TWO>& old,
                                            uint16_t* out, int64_t at, int64_t lo_off) {
    i32x4 h, l;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        float x[2] = {v[2 * u] * p.scale, v[2 * u + 1] * p.scale};
        if constexpr (KIND != kGram) {
            float y[2] = {f16_lo((uint32_t)old.hi[u]), f16_hi((uint32_t)old.hi[u])};
            if constexpr (TWO) {
                y[0] += f16_lo((uint32_t)old.lo[u]);
                y[1] += f16_hi((uint32_t)old.lo[u]);
            }
            x[0] += p.add_scale * y[0];
            x[1] += p.add_scale * y[1];
        }
        h[u] = (int)pack_f16x2(x[0], x[1]);
        if constexpr (TWO) l[u] = (int)pack_f16x2(x[0] - f16_lo((uint32_t)h[u]), x[1] - f16_hi((uint32_t)h[u]));
    }
    *(gbl_i32x4*)(out + at) = h;
    if constexpr (TWO) *(gbl_i32x4*)(out + at + lo_off) = l;
}

// One TILE x TILE tile at rows m0 and columns n0 of matrix b.  A stage of the K loop is a 128-byte line
// of every row of the left tile (64 halves of K, or 32 of both planes) and as many bytes of the right
// one, in two slots.  Left tiles, and the right ones of the symmetric products, are read as
// K-contiguous rows with 16-byte chunk q of row i in slot q ^ ((i >> 1) & 7); the iterate's rows (K
// across them) through the transposing reads, chunk q of row k in slot q ^ 4 (k & 3).  Both keep every
// read free of bank conflicts.
//
// A stage is four (six) groups of matrix products; each group's fragments are read while the group before
// multiplies.  Before the last group every read of the stage is done, so the barrier that hands the
// slot over stands there, and the next stage's first fragments and the loads of the one after
// next go out under the last group's products.
template <int TILE, int WAVES, bool SPLIT, NewtonProduct KIND>
__device__ __forceinline__ void newton_tile(const NewtonGemm& p, char* smem, int b, int64_t m0, int64_t n0) {
    constexpr int WM = 2, WN = WAVES / 2;               // waves along rows and columns
    constexpr int WTM = TILE / WM, WTN = TILE / WN;     // a wave's part
    constexpr int NBM = WTM / 32, NBN = WTN / 32;       // 32 x 32 blocks of it
    constexpr int STAGE = TILE * 128;                   // bytes of one operand's stage
    constexpr int LOADS = STAGE / 1024 / WAVES;         // direct loads a wave and operand
    constexpr int KSTAGE = SPLIT ? 32 : 64;
    constexpr int ROWB = TILE * (SPLIT ? 4 : 2);        // update: bytes of one k-row of the right tile
    constexpr int CPR = ROWB / 16;
    constexpr int PRODUCTS = NBM * NBN;                 // of one group
    lds_char* const lds = (lds_char*)smem;
    const uint32_t lds0 = lds_addr(smem);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % WM, wn = wave / WM;
    const int l32 = lane & 31, lhi = lane >> 5, g16 = lane >> 4, i16 = lane & 15;

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
    // load t of stage s; past the last stage an empty range (no memory is read)
    auto load_one = [&](int s, int t) __attribute__((always_inline)) {
        const uint32_t dst = lds0 + (uint32_t)((s & 1) * 2 * STAGE) + (uint32_t)(wave * LOADS) * 1024u;
        const uint32_t range = s < stages ? 0xFFFFFFFFu : 0u;
        const int u = t >> 1;
        if (t & 1) dma_16B(rsrc_words(right + s * r_step, range), r_off[u], dst + (uint32_t)(STAGE + u * 1024));
        else dma_16B(rsrc_words(left + (int64_t)s * 128, range), l_off[u], dst + (uint32_t)u * 1024u);
    };

    // fragment q (0..3) of a stage: one product: K = 16 q ..; three: plane q >> 1, K = 16 (q & 1) ..
    const uint32_t l_row = (uint32_t)(wm * WTM + l32) * 128u, r_row = (uint32_t)(wn * WTN + l32) * 128u;
    const int sw = (l32 >> 1) & 7;
    const int kr = 8 * (g16 >> 1) + (i16 >> 2);
    const int cq = 2 * (g16 & 1) + ((i16 & 3) >> 1);
    auto read_left = [&](int s, int q, int i) __attribute__((always_inline)) {
        const lds_char* const base = lds + (s & 1) * 2 * STAGE;
        return lds_load_16B(base, l_row + (uint32_t)i * 4096u + (uint32_t)(((2 * q + lhi) ^ sw) << 4));
    };
    auto read_right = [&](int s, int q, int j) __attribute__((always_inline)) {
        const lds_char* const base = lds + (s & 1) * 2 * STAGE + STAGE;
        if constexpr (KIND == kUpdate) {
            const int chunk = SPLIT ? (wn * NBN + j) * 8 + (q >> 1) * 4 + cq : wn * (WTN / 8) + 4 * j + cq;
            const uint32_t at = (uint32_t)((SPLIT ? 16 * (q & 1) : 16 * q) + kr) * (uint32_t)ROWB +
                                (uint32_t)((chunk ^ ((i16 >> 2) << 2)) << 4) + (uint32_t)(i16 & 1) * 8u;
            const i16x4 lo = lds_read_tr16(base, at);
            const i16x4 hi = lds_read_tr16(base, at + 4 * ROWB);
            const i16x8 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            return __builtin_bit_cast(i32x4, v);
        } else {
            return lds_load_16B(base, r_row + (uint32_t)j * 4096u + (uint32_t)(((2 * q + lhi) ^ sw) << 4));
        }
    };

    f32x16 acc[NBN][NBM];
#pragma unroll
    for (int j = 0; j < NBN; ++j)
#pragma unroll
        for (int i = 0; i < NBM; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[j][i][r] = 0.0f;

    struct Left { i32x4 v[NBM]; };
    struct Right { i32x4 v[NBN]; };
    // All products of one group; `other(k)` goes out after product k.
    auto group = [&](const Left& l, const Right& r, auto other) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < PRODUCTS; ++k) {
            const int j = k / NBM, i = k % NBM;
            acc[j][i] = mfma_f16_32x32x16(r.v[j], l.v[i], acc[j][i]);
            __builtin_amdgcn_sched_barrier(0);
            other(k);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // Share of `n` things that go out after product k, as evenly as they come.
    auto share = [](int k, int n, auto one) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < n; ++t)
            if (t * PRODUCTS / n == k) one(t);
    };
    auto read_both = [&](int s, int q, Left& l, Right& r, int t) __attribute__((always_inline)) {
        if (t < NBM) l.v[t] = read_left(s, q, t);
        else r.v[t - NBM] = read_right(s, q, t - NBM);
    };
    // The stage's reads are done: wait for the next one's loads and hand the slots over.
    auto hand_over = [&]() __attribute__((always_inline)) {
        wait_lgkmcnt0();
        wait_vmcnt<0>();
        barrier_no_fence();
        __builtin_amdgcn_sched_barrier(0);
    };

#pragma unroll
    for (int t = 0; t < 2 * LOADS; ++t) load_one(0, t);
#pragma unroll
    for (int t = 0; t < 2 * LOADS; ++t) load_one(1, t);
    wait_vmcnt<2 * LOADS>();
    barrier_no_fence();
    Left l0, l1;
    Right r0, r1;
#pragma unroll
    for (int t = 0; t < NBM + NBN; ++t) read_both(0, 0, l0, r0, t);
    for (int s = 0; s < stages; ++s) {
        // under the last group: the next stage's first fragments, then the loads of the stage after it
        auto next_stage = [&](Left& l, Right& r) {
            return [&, s](int k) __attribute__((always_inline)) {
                share(k, NBM + NBN, [&](int t) { read_both(s + 1, 0, l, r, t); });
                share(k, 2 * LOADS, [&](int t) { load_one(s + 2, t); });
            };
        };
        if constexpr (!SPLIT) {
            group(l0, r0, [&](int k) { share(k, NBM + NBN, [&](int t) { read_both(s, 1, l1, r1, t); }); });
            group(l1, r1, [&](int k) { share(k, NBM + NBN, [&](int t) { read_both(s, 2, l0, r0, t); }); });
            group(l0, r0, [&](int k) { share(k, NBM + NBN, [&](int t) { read_both(s, 3, l1, r1, t); }); });
            hand_over();
            group(l1, r1, next_stage(l0, r0));
        } else {
            Left low_l;
            Right low_r;
            group(l0, r0, [&](int k) { share(k, NBN, [&](int t) { low_r.v[t] = read_right(s, 2, t); }); });
            group(l0, low_r, [&](int k) { share(k, NBM, [&](int t) { low_l.v[t] = read_left(s, 2, t); }); });
            group(low_l, r0, [&](int k) { share(k, NBM + NBN, [&](int t) { read_both(s, 1, l1, r1, t); }); });
            group(l1, r1, [&](int k) { share(k, NBN, [&](int t) { low_r.v[t] = read_right(s, 3, t); }); });
            group(l1, low_r, [&](int k) { share(k, NBM, [&](int t) { low_l.v[t] = read_left(s, 3, t); }); });
            hand_over();
            group(low_l, r1, next_stage(l0, r0));
        }
    }
    wait_lgkmcnt0();
    wait_vmcnt<0>();
    barrier_no_fence();

    // acc[j][i][4g + t] is the product at row 32 i + l32 and column 32 j + 8 g + 4 lhi + t of the
    // wave's part.  It goes out through LDS, 32 rows at a time, so that every store writes whole runs of a row: once as
    // it is and, for a tile below the diagonal, once transposed.
    constexpr bool TWO = SPLIT || KIND == kUpdate;      // both planes are kept
    const int64_t lo_off = SPLIT ? 32 : (int64_t)p.batch * p.rows * p.cols;
    const int64_t matrix = (int64_t)b * p.rows * p.cols * (SPLIT ? 2 : 1);
    uint16_t* const out = (uint16_t*)p.out + matrix;
    const uint16_t* const add = (const uint16_t*)p.add + matrix;
    lds_char* const mine = lds + wave * (4 * STAGE / WAVES);
    static_assert(32 * (WTM > WTN ? WTM : WTN) * 4 <= 4 * STAGE / WAVES, "the image fits the wave's share of LDS");
    // the wave's own LDS accesses keep their order; this keeps the compiler from changing it
    auto image_written = [] { asm volatile("" ::: "memory"); };
    auto drain = [&](auto width, int64_t row0, int64_t col0) __attribute__((always_inline)) {
        constexpr int W = decltype(width)::value, LPR = W / 8, RPI = 64 / LPR, N = 32 / RPI;
        int64_t at[N];
        Addend<KIND, TWO> old[N];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            at[n] = element<SPLIT>(row0 + n * RPI + lane / LPR, col0 + 8 * (lane % LPR), p.cols);
            old[n].load(add, at[n], lo_off);
        }
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int r = n * RPI + lane / LPR, c = 2 * (lane % LPR);
            const f32x4 u = __builtin_bit_cast(f32x4, lds_load_16B(mine, image_at<W>(r, c)));
            const f32x4 w = __builtin_bit_cast(f32x4, lds_load_16B(mine, image_at<W>(r, c + 1)));
            const float v[8] = {u[0], u[1], u[2], u[3], w[0], w[1], w[2], w[3]};
            store_eight<KIND, TWO>(p, v, old[n], out, at[n], lo_off);
        }
        asm volatile("" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < NBM; ++i) {
#pragma unroll
        for (int j = 0; j < NBN; ++j)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const f32x4 v = {acc[j][i][4 * g], acc[j][i][4 * g + 1], acc[j][i][4 * g + 2], acc[j][i][4 * g + 3]};
                lds_store_16B(mine, image_at<WTN>(l32, 8 * j + 2 * g + lhi), __builtin_bit_cast(i32x4, v));
            }
        image_written();
        drain(std::integral_constant<int, WTN>{}, m0 + wm * WTM + 32 * i, n0 + wn * WTN);
    }
    if (KIND != kUpdate && m0 != n0) {
#pragma unroll
        for (int j = 0; j < NBN; ++j) {
#pragma unroll
            for (int i = 0; i < NBM; ++i)
#pragma unroll
                for (int g = 0; g < 4; ++g)
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const uint32_t at = image_at<WTM>(8 * g + 4 * lhi + t, 8 * i + (l32 >> 2)) + (l32 & 3) * 4u;
                        *reinterpret_cast<__attribute__((address_space(3))) float*>(mine + at) = acc[j][i][4 * g + t];
                    }
            image_written();
            drain(std::integral_constant<int, WTM>{}, n0 + wn * WTN + 32 * j, m0 + wm * WTM);
        }
    }
}

template <bool SPLIT>
constexpr int kBigWaves = 8;

// 256 x 256 tiles; the items past p.whole are quarters of one.
template <bool SPLIT, NewtonProduct KIND>
__global__ __launch_bounds__(64 * kBigWaves<SPLIT>, kBigWaves<SPLIT> / 4) void newton_big_kernel(NewtonGemm p) {
    __shared__ __attribute__((aligned(1024))) char smem[4 * 256 * 128];
    const int bid = blockIdx.x;
    int b, tm, tn;
    if (bid < p.whole) {
        tile_of<KIND>(p, item_of(bid, p.whole, p.num_xcds), b, tm, tn);
        newton_tile<256, kBigWaves<SPLIT>, SPLIT, KIND>(p, smem, b, (int64_t)tm * 256, (int64_t)tn * 256);
    } else {
        const int part = bid - p.whole;
        tile_of<KIND>(p, p.whole + (part >> 2), b, tm, tn);
        const int64_t m0 = (int64_t)tm * 256 + (part & 1) * 128, n0 = (int64_t)tn * 256 + ((part >> 1) & 1) * 128;
        if (KIND != kUpdate && n0 > m0) return;         // the mirror image of another quarter
        newton_tile<128, kBigWaves<SPLIT>, SPLIT, KIND>(p, smem, b, m0, n0);
    }
}

template <bool SPLIT, NewtonProduct KIND>
__global__ __launch_bounds__(256, 2) void newton_small_kernel(NewtonGemm p) {
    __shared__ __attribute__((aligned(1024))) char smem[4 * 128 * 128];
    int b, tm, tn;
    tile_of<KIND>(p, item_of(blockIdx.x, p.items, p.num_xcds), b, tm, tn);
    newton_tile<128, 4, SPLIT, KIND>(p, smem, b, (int64_t)tm * 128, (int64_t)tn * 128);
}

template <bool SPLIT, NewtonProduct KIND>
void launch_product(NewtonGemm g, int tile, int num_cus, hipStream_t stream) {
    g.tiles_m = (int32_t)(g.rows / tile);
    g.tiles_n = (int32_t)(g.cols / tile);
    const int tiles = g.batch * (KIND == kUpdate ? g.tiles_m * g.tiles_n : g.tiles_m * (g.tiles_m + 1) / 2);
    if (tile == 256) {
        // whole rounds of tiles on all CUs, then the rest as quarters when they fill two rounds at most
        const int rest = tiles % num_cus;
        g.whole = 2 * rest <= num_cus ? tiles - rest : tiles;
        g.items = g.whole + 4 * (tiles - g.whole);
        hipLaunchKernelGGL((newton_big_kernel<SPLIT, KIND>), dim3((uint32_t)g.items), dim3(64 * kBigWaves<SPLIT>), 0,
                           stream, g);
    } else {
        g.items = g.whole = tiles;
        hipLaunchKernelGGL((newton_small_kernel<SPLIT, KIND>), dim3((uint32_t)g.items), dim3(256), 0, stream, g);
    }
}

template <bool SPLIT>
void launch_steps(const NewtonParams& p, const NewtonPlan& plan, const float* co, int num_cus, int num_xcds,
                  hipStream_t stream) {
    NewtonGemm g = {};
    g.batch = p.batch;
    g.num_xcds = num_xcds;
    g.rows = plan.r;
    for (int s = 0; s < p.steps; ++s) {
        const char* const x = p.x[s & 1];
        g.cols = plan.r;
        g.k = plan.c;
        g.left = g.right = x;
        g.out = p.a;
        g.scale = kAScale / (kXScale * kXScale);
        launch_product<SPLIT, kGram>(g, plan.tile, num_cus, stream);
        g.k = plan.r;
        g.left = g.right = g.add = p.a;
        g.out = p.b;
        g.scale = co[3 * s + 2] * (kBScale / (kAScale * kAScale));
        g.add_scale = co[3 * s + 1] * (kBScale / kAScale);
        launch_product<SPLIT, kSquare>(g, plan.tile, num_cus, stream);
        g.cols = plan.c;
        g.left = p.b;
        g.right = g.add = x;
        g.out = p.x[(s + 1) & 1];
        g.scale = 1.0f / kBScale;
        g.add_scale = co[3 * s];
        launch_product<SPLIT, kUpdate>(g, plan.tile, num_cus, stream);
    }
}

template <bool SPLIT, bool TALL>
void launch_all(const NewtonParams& p, const NewtonPlan& plan, const float* co, int num_cus, int num_xcds,
                hipStream_t stream) {
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
    launch_steps<SPLIT>(p, plan, co, num_cus, num_xcds, stream);
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
        if (plan.tall) launch_all<true, true>(p, plan, coefficients, num_cus, num_xcds, stream);
        else launch_all<true, false>(p, plan, coefficients, num_cus, num_xcds, stream);
    } else {
        if (plan.tall) launch_all<false, true>(p, plan, coefficients, num_cus, num_xcds, stream);
        else launch_all<false, false>(p, plan, coefficients, num_cus, num_xcds, stream);
    }
    return hipGetLastError();
}

}  // namespace kgw
