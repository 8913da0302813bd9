// Newton-Schulz orthogonalisation of matrices whose short side is at most 128 (gfx950).
//
// Such a matrix has so little work that launches and the way through memory decide its time.  Where the
// iterate fits into one workgroup's LDS (64 x 512 or 128 x 128), one launch runs everything, the norm
// included (narrow_whole_kernel).  Longer ones take a launch a step: every workgroup holds all r rows of
// its columns, squares the r x r matrix A = X X^T for itself
// (128^3 products, 1.3 us), updates its columns and adds up their part of the next A:
//
//     A = sum of the parts;  B = b A + c A A;  X <- a X + B X;  part = X X^T over the own columns
//
// Every operand is kept as two fp16 planes and multiplied by three products (hi hi, hi lo,
// lo hi), also for bf16 results: short sides average rounding errors less (r = 24: 2.0e-3 with one
// product, more than bf16's own 1.7e-3), and here they cost next to nothing.
//
// Everything moves in one unit, a "fragment": 64 lanes x 16 bytes, an operand of the matrix core
// for 32 rows and 16 values of K.  Lane l holds row l & 31 and, with h = l >> 5, the K values 4 h .. 4 h + 3
// and 8 + 4 h .. 8 + 4 h + 3.  A product's sums lie in the registers in that same order (its
// columns over the lanes, its rows in runs of four), so converting 8 sums of a lane to halves makes a
// fragment of the transposed matrix without moving anything between lanes: the sums of an update are the next
// product X X^T's fragments.  Where X is needed the other way round (K along its rows), the transposing LDS
// reads turn the same image.  The order of K inside a fragment does not matter, as long as both operands have it.
//
// Iterates are stored as fragments, chunk by chunk of 128 columns: [chunk][16 columns][32 rows][plane],
// so loads and stores are whole kilobytes.
#include "kgw_newton_device.h"

namespace kgw {
namespace {

constexpr int NT = 256;
constexpr int CHUNK = 128;                       // columns
constexpr int SLICES = CHUNK / 16;

struct NarrowParams {
    NewtonParams p;
    const char* x_in;       // iterates (NULL: made from G)
    char* x_out;            // (NULL: the result is written)
    const float* parts_in;  // (batch, groups_in, RB * RB, 64 lanes, 16) sums of X X^T
    float* parts_out;
    int32_t groups_in;      // parts of A to be added up
    int32_t groups, chunks, per_group;
    int32_t tall;
    int32_t step;
    float co[3];            // a, b, c of the step
};

// 8 sums of one lane -> its 16 bytes of a fragment, high and low plane.
__device__ __forceinline__ void split_eight(const float (&v)[8], i32x4& hi, i32x4& lo) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const HalfPair p = split_pair(v[2 * u], v[2 * u + 1]);
        hi[u] = (int)p.hi;
        lo[u] = (int)p.lo;
    }
}

// RB: blocks of 32 rows of the short side (2 or 4).
template <int RB>
struct Narrow {
    // Eight waves for r = 128, so that one wave's conversions go under another one's products; four for 64.
    static constexpr int WAVES = RB == 4 ? 8 : 4;
    static constexpr int THREADS = 64 * WAVES;
    static constexpr int MINE = RB * RB / WAVES;                // blocks of an r x r matrix a wave has
    static constexpr int ROWS = 4 * RB / WAVES;                 // rows blocks a wave updates, in 32 columns
    static constexpr uint32_t X_BYTES = SLICES * RB * 2048u;    // one chunk of the iterate
    static constexpr uint32_t A_BYTES = RB * 2 * RB * 2048u;    // an r x r matrix
    // A wave's blocks: rows block (of fragments), columns block j.
    static __device__ __forceinline__ int row_of(int wave, int) { return wave >> 1; }
    static __device__ __forceinline__ int col_of(int wave, int j) { return MINE * (wave & 1) + j; }
    // A wave's columns of a chunk and first rows block in the update.
    static __device__ __forceinline__ int columns(int wave) { return wave & 3; }
    static __device__ __forceinline__ int rows(int wave) { return (wave >> 2) * ROWS; }
    // Fragment of rows block `rows`, slice `k` of 16 K values, in a chunk of X or in A.
    static __device__ __forceinline__ uint32_t x_at(int k, int rows, int plane) { return (uint32_t)((k * RB + rows) * 2 + plane) * 1024u; }
    static __device__ __forceinline__ uint32_t a_at(int k, int rows, int plane) { return x_at(k, rows, plane); }
};

// acc[j] += col[j] x row over K slices of 16, each operand as three products of its planes, col (ROW_FIRST: row) down
// the registers and the other one over the lanes; read(k, f) reads the fragments of slice k.  The next slice is
// read under the products of this one, and the products go over
// all of acc in turn, so that no product waits for a read or for the one just before it.
template <int COLS>
struct Slice {
    i32x4 row[2], col[COLS][2];                         // high and low plane
};
template <int SLICES_OF_K, bool ROW_FIRST, int COLS, class Read>
__device__ __forceinline__ void multiply(f32x16 (&acc)[COLS], Read read) {
    Slice<COLS> f[2];
    auto product = [&](const Slice<COLS>& g, int j, int col_plane, int row_plane) __attribute__((always_inline)) {
        const i32x4 c = g.col[j][col_plane], r = g.row[row_plane];
        acc[j] = ROW_FIRST ? mfma_f16_32x32x16(r, c, acc[j]) : mfma_f16_32x32x16(c, r, acc[j]);
    };
    read(std::integral_constant<int, 0>{}, f[0]);
    each<SLICES_OF_K>([&](auto k) __attribute__((always_inline)) {
        if constexpr (k + 1 < SLICES_OF_K) read(std::integral_constant<int, k + 1>{}, f[(k + 1) & 1]);
        __builtin_amdgcn_sched_barrier(0);
        const Slice<COLS>& g = f[k & 1];
#pragma unroll
        for (int j = 0; j < COLS; ++j) product(g, j, 0, 1);
#pragma unroll
        for (int j = 0; j < COLS; ++j) product(g, j, 1, 0);
#pragma unroll
        for (int j = 0; j < COLS; ++j) product(g, j, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
    });
}

// Adds this wave's blocks of M M^T to acc: the rows block over the lanes, columns blocks down the registers.
template <int RB, int SLICES_OF_K>
__device__ __forceinline__ void add_gram(const lds_char* m, int wave, int lane, f32x16 (&acc)[Narrow<RB>::MINE]) {
    using N = Narrow<RB>;
    multiply<SLICES_OF_K, false>(acc, [&](auto k, Slice<N::MINE>& f) __attribute__((always_inline)) {
#pragma unroll
        for (int plane = 0; plane < 2; ++plane) {
            f.row[plane] = lds_load_16B(m, N::x_at(k, N::row_of(wave, 0), plane) + lane * 16u);
#pragma unroll
            for (int j = 0; j < N::MINE; ++j)
                f.col[j][plane] = lds_load_16B(m, N::x_at(k, N::col_of(wave, j), plane) + lane * 16u);
        }
    });
}

template <int RB>
__device__ __forceinline__ void store_part(const NarrowParams& q, int b, int group, int wave, int lane,
                                           const f32x16 (&acc)[Narrow<RB>::MINE]) {
    using N = Narrow<RB>;
    float* const to = q.parts_out + ((int64_t)b * q.groups + group) * (RB * RB * 1024);
#pragma unroll
    for (int j = 0; j < N::MINE; ++j) {
        const int block = N::row_of(wave, j) * RB + N::col_of(wave, j);
#pragma unroll
        for (int g = 0; g < 4; ++g)
            *(gbl_f32x4*)(to + block * 1024 + g * 256 + lane * 4) =
                f32x4{acc[j][4 * g], acc[j][4 * g + 1], acc[j][4 * g + 2], acc[j][4 * g + 3]};
    }
}

template <int N>
__device__ __forceinline__ void clear(f32x16 (&m)[N]) {
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) m[j][e] = 0.0f;
}

// One chunk of the first iterate into LDS.
template <int RB, int DT>
__device__ __forceinline__ void first_chunk(const NarrowParams& q, int b, int chunk, FirstScale scale, lds_char* x, int tid) {
    using N = Narrow<RB>;
    const int64_t n0 = (int64_t)chunk * CHUNK;
    if (!q.tall) {
        // eight consecutive columns of one row: two runs of four, for the two lane halves
        for (int i = tid; i < 32 * RB * (CHUNK / 8); i += N::THREADS) {
            const int row = i / (CHUNK / 8), c8 = i % (CHUNK / 8);
            float v[8];
            load_eight<DT>(q.p, b, row, n0 + 8 * c8, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = scale.of(v[e]);
            i32x4 hi, lo;
            split_eight(v, hi, lo);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int plane = 0; plane < 2; ++plane) {
                    const i32x4 w = plane ? lo : hi;
                    const i32x2 half = {w[2 * h], w[2 * h + 1]};
                    const uint32_t at = N::x_at(c8 >> 1, row >> 5, plane) + (uint32_t)(32 * h + (row & 31)) * 16u +
                                        (uint32_t)(c8 & 1) * 8u;
                    *reinterpret_cast<__attribute__((address_space(3))) i32x2*>(x + at) = half;
                }
        }
    } else {
        // G is (c, r): eight consecutive rows of the iterate in one of its columns
        for (int i = tid; i < CHUNK * 4 * RB; i += N::THREADS) {
            const int col = i / (4 * RB), r8 = i % (4 * RB);
            float v[8];
            load_eight<DT>(q.p, b, n0 + col, 8 * r8, v);
            const int in = col & 15;                         // column 4 h + 8 s + t: half h, run s, place t
            const uint32_t place = (uint32_t)((in >> 2) & 1) * 512u + (uint32_t)(in >> 3) * 8u + (uint32_t)(in & 3) * 2u;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int row = 8 * r8 + e;
                const HalfPair u = split_pair(scale.of(v[e]), 0.0f);
                const uint32_t at = place + (uint32_t)(row & 31) * 16u;
                *reinterpret_cast<__attribute__((address_space(3))) uint16_t*>(x + N::x_at(col >> 4, row >> 5, 0) + at) = (uint16_t)u.hi;
                *reinterpret_cast<__attribute__((address_space(3))) uint16_t*>(x + N::x_at(col >> 4, row >> 5, 1) + at) = (uint16_t)u.lo;
            }
        }
    }
}

// This wave's blocks of an r x r matrix as fragments into LDS: rows over the lanes, K = columns.
template <int RB>
__device__ __forceinline__ void write_blocks(lds_char* a, int wave, int lane, const f32x16 (&m)[Narrow<RB>::MINE]) {
    using N = Narrow<RB>;
#pragma unroll
    for (int j = 0; j < N::MINE; ++j)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = m[j][8 * s + e];
            i32x4 hi, lo;
            split_eight(v, hi, lo);
            const int k = 2 * N::col_of(wave, j) + s, rows = N::row_of(wave, j);
            lds_store_16B(a, N::a_at(k, rows, 0) + lane * 16u, hi);
            lds_store_16B(a, N::a_at(k, rows, 1) + lane * 16u, lo);
        }
}

// Scales measured on A (kBoundLoss): from the sum of its squares, the same in every workgroup of the matrix.
template <int RB>
__device__ __forceinline__ StepScales measured_scales(const f32x16 (&mine)[Narrow<RB>::MINE], double* sums, SingularBound& bound,
                                                      const float* co, bool last, int wave, int lane) {
    double s = 0.0;
#pragma unroll
    for (int j = 0; j < Narrow<RB>::MINE; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const double x = (double)(mine[j][e] * kGramScale);
            s += x * x;
        }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d);
    if (lane == 0) sums[wave] = s;
    __syncthreads();
    double squares = 0.0;
#pragma unroll
    for (int w = 0; w < Narrow<RB>::WAVES; ++w) squares += sums[w];
    __syncthreads();
    bound = measured_bound(squares, bound.plane);
    return step_scales(bound, co, last);
}

// B = square (A A + square_linear A) as fragments in LDS, from the blocks of X X^T that each wave has.
// The caller's barriers: no one reads `a` any more before, all have written it after.
template <int RB>
__device__ __forceinline__ void make_b(const StepScales& scales, lds_char* a, int wave, int lane,
                                       f32x16 (&mine)[Narrow<RB>::MINE]) {
    using N = Narrow<RB>;
#pragma unroll
    for (int j = 0; j < N::MINE; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) mine[j][e] *= kGramScale;
    write_blocks<RB>(a, wave, lane, mine);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < N::MINE; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) mine[j][e] *= scales.square_linear;
    add_gram<RB, 2 * RB>(a, wave, lane, mine);
#pragma unroll
    for (int j = 0; j < N::MINE; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) mine[j][e] *= scales.square;
    __syncthreads();
    write_blocks<RB>(a, wave, lane, mine);
}

// acc = update (B X + update_linear X) in this wave's 32 columns of a chunk: columns down the registers, rows
// over the lanes.
template <int RB>
__device__ __forceinline__ void update_chunk(const StepScales& scales, const lds_char* x, const lds_char* a, int wave, int lane,
                                             f32x16 (&acc)[Narrow<RB>::ROWS]) {
    using N = Narrow<RB>;
    const int g16 = lane >> 4, i16 = lane & 15;
    clear(acc);
    // row: 32 columns of X; col: the rows blocks of B
    multiply<2 * RB, true>(acc, [&](auto k, Slice<N::ROWS>& f) __attribute__((always_inline)) {
        // Transposed fragment of rows 16 k .. of X: 16 lanes read 4 rows x 16 columns, of which
        // piece c (4 columns) of a row is half c & 1, run c >> 1 of its place in the image.
#pragma unroll
        for (int plane = 0; plane < 2; ++plane) {
            const int slice = 2 * N::columns(wave) + (g16 & 1), c = i16 & 3;
            const int row = 16 * k + 4 * (g16 >> 1) + (i16 >> 2);
            const uint32_t at = N::x_at(slice, 0, plane) + (uint32_t)(k >> 1) * 2048u + (uint32_t)(c & 1) * 512u +
                                (uint32_t)(row & 31) * 16u + (uint32_t)(c >> 1) * 8u;
            const i16x4 v0 = lds_read_tr16(x, at);
            const i16x4 v1 = lds_read_tr16(x, at + 8 * 16);
            const i16x8 v = {v0[0], v0[1], v0[2], v0[3], v1[0], v1[1], v1[2], v1[3]};
            f.row[plane] = __builtin_bit_cast(i32x4, v);
#pragma unroll
            for (int i = 0; i < N::ROWS; ++i)
                f.col[i][plane] = lds_load_16B(a, N::a_at(k, N::rows(wave) + i, plane) + lane * 16u);
        }
    });
    // a X from the same image, added last: it decides the small singular values
#pragma unroll
    for (int i = 0; i < N::ROWS; ++i)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const i32x4 hi = lds_load_16B(x, N::x_at(2 * N::columns(wave) + s, N::rows(wave) + i, 0) + lane * 16u);
            const i32x4 lo = lds_load_16B(x, N::x_at(2 * N::columns(wave) + s, N::rows(wave) + i, 1) + lane * 16u);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float x0 = acc[i][8 * s + 2 * u] + scales.update_linear * f16_lo((uint32_t)lo[u]);
                const float x1 = acc[i][8 * s + 2 * u + 1] + scales.update_linear * f16_hi((uint32_t)lo[u]);
                acc[i][8 * s + 2 * u] = scales.update * (x0 + scales.update_linear * f16_lo((uint32_t)hi[u]));
                acc[i][8 * s + 2 * u + 1] = scales.update * (x1 + scales.update_linear * f16_hi((uint32_t)hi[u]));
            }
        }
}

// This wave's part of the next iterate into the image, and to `to` where that is not NULL.
template <int RB>
__device__ __forceinline__ void store_chunk(lds_char* x, char* to, int wave, int lane, const f32x16 (&acc)[Narrow<RB>::ROWS]) {
    using N = Narrow<RB>;
#pragma unroll
    for (int i = 0; i < N::ROWS; ++i)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = acc[i][8 * s + e];
            i32x4 hi, lo;
            split_eight(v, hi, lo);
            const uint32_t at = N::x_at(2 * N::columns(wave) + s, N::rows(wave) + i, 0) + lane * 16u;
            lds_store_16B(x, at, hi);
            lds_store_16B(x, at + 1024u, lo);
            if (to) {
                *(gbl_i32x4*)(to + at) = hi;
                *(gbl_i32x4*)(to + at + 1024u) = lo;
            }
        }
}

template <int RB>
__device__ __forceinline__ void store_result(const NarrowParams& q, int b, int chunk, int wave, int lane,
                                             const f32x16 (&acc)[Narrow<RB>::ROWS]) {
    using N = Narrow<RB>;
    // at most 128 x 2^20 elements a matrix: 32-bit offsets
    const int r = (int)(q.tall ? q.p.n : q.p.m), c = (int)(q.tall ? q.p.m : q.p.n), ld = (int)q.p.n;
    const int row_step = q.tall ? 1 : ld, col_step = q.tall ? ld : 1;
    const int c0 = chunk * CHUNK + 32 * N::columns(wave) + 4 * (lane >> 5);
    const int r0 = 32 * N::rows(wave) + (lane & 31);
    const int at0 = r0 * row_step + c0 * col_step;
    char* const out = (char*)q.p.out + (int64_t)b * q.p.m * q.p.n * (q.p.out_dtype == kOutF32 ? 4 : 2);
#pragma unroll
    for (int i = 0; i < N::ROWS; ++i) {
        if (32 * i + r0 >= r) continue;
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                if (c0 + 8 * g + t >= c) continue;
                const int at = at0 + 32 * i * row_step + (8 * g + t) * col_step;
                const float v = acc[i][4 * g + t];
                if (q.p.out_dtype == kOutF32) ((float*)out)[at] = v;
                else ((uint16_t*)out)[at] = (uint16_t)(q.p.out_dtype == kOutBf16 ? pack_bf16x2(v, 0.0f) : to_halves(v, 0.0f));
            }
    }
}

// The first iterate's chunks and their parts of A: 12.4 us for 8 x 128 x 4096 bf16 (8 MB in, 17 MB out), 5.3 us for 24 x 5000.
template <int RB, int DT>
__global__ __launch_bounds__(Narrow<RB>::THREADS, 1) void narrow_first_kernel(NarrowParams q, NewtonCoefficients co) {
    using N = Narrow<RB>;
    __shared__ __attribute__((aligned(1024))) char smem[N::X_BYTES];
    lds_char* const x = (lds_char*)smem;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int b = blockIdx.y, group = blockIdx.x;
    if (group == 0 && wave == 0) write_unit_scales(q.p, co, b);
    const FirstScale scale = first_scale(q.p, b);
    if (group == 0 && wave == 0) write_scales(q.p, co, b, scale);
    f32x16 part[N::MINE];
    clear(part);
    const int first = group * q.per_group, last = min(q.chunks, first + q.per_group);
    for (int chunk = first; chunk < last; ++chunk) {
        __syncthreads();
        first_chunk<RB, DT>(q, b, chunk, scale, x, tid);
        __syncthreads();
        char* const to = q.x_out + ((int64_t)b * q.chunks + chunk) * N::X_BYTES;
        for (uint32_t i = tid * 16u; i < N::X_BYTES; i += N::THREADS * 16u) *(gbl_i32x4*)(to + i) = lds_load_16B(x, i);
        add_gram<RB, SLICES>(x, wave, lane, part);
    }
    store_part<RB>(q, b, group, wave, lane, part);
}

// One step.  LAST: the result instead of the next iterate and its part of A.
// 8 x 128 x 4096: 18 us for 17 MB read and 17 written (L2 and Infinity Cache) and 9.7 GFLOP of fp16 products, all
// of them one after the other in a workgroup of its own chunk: latencies bound it, as they do the
// 5.6 us of a step of 24 x 5000 or 6.5 us of 8 x 64 x 512.
template <int RB, bool LAST, bool MEASURED>
__global__ __launch_bounds__(Narrow<RB>::THREADS, 1) void narrow_step_kernel(NarrowParams q) {
    using N = Narrow<RB>;
    __shared__ __attribute__((aligned(1024))) char smem[N::X_BYTES + N::A_BYTES];
    __shared__ double sums[N::WAVES];
    lds_char* const x = (lds_char*)smem;
    lds_char* const a = x + N::X_BYTES;
    const uint32_t x_addr = lds_addr(smem);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int b = blockIdx.y, group = blockIdx.x;
    const int first = group * q.per_group, last = min(q.chunks, first + q.per_group);

    auto load_chunk = [&](int chunk) __attribute__((always_inline)) {
        const i32x4 r = rsrc_words(q.x_in + ((int64_t)b * q.chunks + chunk) * N::X_BYTES);
#pragma unroll
        for (uint32_t t = 0; t < N::X_BYTES / 1024 / N::WAVES; ++t) {
            const uint32_t at = (wave * (N::X_BYTES / 1024 / N::WAVES) + t) * 1024u;
            dma_16B(r, at + lane * 16u, x_addr + at);
        }
    };
    load_chunk(first);
    StepScales scales;
    if constexpr (!MEASURED) scales = q.p.scales[(int64_t)b * kNewtonMaxSteps + q.step];

    // A: this wave's blocks, added up in the order of the parts
    f32x16 mine[N::MINE];
    clear(mine);
    const float* from = q.parts_in + (int64_t)b * q.groups_in * (RB * RB * 1024);
    for (int w = 0; w < q.groups_in; ++w, from += RB * RB * 1024) {
#pragma unroll
        for (int j = 0; j < N::MINE; ++j) {
            const int block = N::row_of(wave, j) * RB + N::col_of(wave, j);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const f32x4 v = *(const gbl_f32x4*)(from + block * 1024 + g * 256 + lane * 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) mine[j][4 * g + e] += v[e];
            }
        }
    }
    if constexpr (MEASURED) {
        SingularBound bound = unit_bound(1.0f);
        bound.plane = q.p.planes[(int64_t)(q.step & 1) * q.p.batch + b];
        scales = measured_scales<RB>(mine, sums, bound, q.co, LAST, wave, lane);
        if (group == 0 && tid == 0) q.p.planes[(int64_t)(~q.step & 1) * q.p.batch + b] = bound.plane;
    }
    make_b<RB>(scales, a, wave, lane, mine);

    f32x16 part[N::MINE];
    clear(part);
    for (int chunk = first; chunk < last; ++chunk) {
        wait_vmcnt<0>();
        __syncthreads();                                // the chunk and B are in LDS
        f32x16 acc[N::ROWS];
        update_chunk<RB>(scales, x, a, wave, lane, acc);
        __syncthreads();                                // all have read the chunk
        if constexpr (LAST) {
            if (chunk + 1 < last) load_chunk(chunk + 1);
            store_result<RB>(q, b, chunk, wave, lane, acc);
        } else {
            store_chunk<RB>(x, q.x_out + ((int64_t)b * q.chunks + chunk) * N::X_BYTES, wave, lane, acc);
            __syncthreads();
            add_gram<RB, SLICES>(x, wave, lane, part);
            if (chunk + 1 < last) {
                __syncthreads();                        // all have read the image
                load_chunk(chunk + 1);
            }
        }
    }
    if constexpr (!LAST) store_part<RB>(q, b, group, wave, lane, part);
}

// Short matrices, all steps of one in one workgroup: its iterate stays in LDS.  64 x 64 x 64 fp32: 22.5 us, 4.5 a
// step, its chain of three products with a barrier after each; the launches of separate steps would take as long.
template <int RB>
constexpr int kWholeChunks = RB == 2 ? 4 : 1;

template <int RB, int DT, bool MEASURED>
__global__ __launch_bounds__(Narrow<RB>::THREADS, 1) void narrow_whole_kernel(NarrowParams q, NewtonCoefficients co) {
    using N = Narrow<RB>;
    __shared__ __attribute__((aligned(1024))) char smem[kWholeChunks<RB> * N::X_BYTES + N::A_BYTES];
    __shared__ double sums[N::WAVES];
    lds_char* const x = (lds_char*)smem;
    lds_char* const a = x + kWholeChunks<RB> * N::X_BYTES;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int b = blockIdx.x;
    // |G|_F, in 64 bits as in newton_norm_kernel
    const int per_row = (int)((q.p.n + 7) / 8);
    double s = 0.0;
    for (int i = tid; i < (int)q.p.m * per_row; i += N::THREADS) {
        const int row = i / per_row;
        float v[8];
        load_eight<DT>(q.p, b, row, 8 * (i - row * per_row), v);
#pragma unroll
        for (int u = 0; u < 8; ++u) s += (double)v[u] * (double)v[u];
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d);
    if (lane == 0) sums[wave] = s;
    __syncthreads();
    double squares = 0.0;
#pragma unroll
    for (int w = 0; w < N::WAVES; ++w) squares += sums[w];
    const FirstScale scale = scale_of_norm(__builtin_sqrt(squares), q.p.eps);

    SingularBound bound = scale.bound;
    __shared__ StepScales table[MEASURED ? 1 : kNewtonMaxSteps];
    if (!MEASURED && wave == 0) {
        if (scale.unit) {
            if (lane < q.p.steps) table[lane] = co.unit[lane];
        } else {
            for (int step = 0; step < q.p.steps; ++step) table[step] = step_scales(bound, co.v + 3 * step, step + 1 == q.p.steps);
        }
    }

    f32x16 mine[N::MINE];
    for (int chunk = 0; chunk < q.chunks; ++chunk) first_chunk<RB, DT>(q, b, chunk, scale, x + chunk * N::X_BYTES, tid);
    __syncthreads();
    clear(mine);
    for (int chunk = 0; chunk < q.chunks; ++chunk) add_gram<RB, SLICES>(x + chunk * N::X_BYTES, wave, lane, mine);
    for (int step = 0; step < q.p.steps; ++step) {
        const bool last = step + 1 == q.p.steps;
        StepScales scales;
        if constexpr (MEASURED) scales = measured_scales<RB>(mine, sums, bound, co.v + 3 * step, last, wave, lane);
        else scales = table[step];
        make_b<RB>(scales, a, wave, lane, mine);
        __syncthreads();
        clear(mine);
        for (int chunk = 0; chunk < q.chunks; ++chunk) {
            lds_char* const at = x + chunk * N::X_BYTES;
            f32x16 acc[N::ROWS];
            update_chunk<RB>(scales, at, a, wave, lane, acc);
            if (last) {
                store_result<RB>(q, b, chunk, wave, lane, acc);
                continue;
            }
            __syncthreads();                            // all have read the chunk
            store_chunk<RB>(at, nullptr, wave, lane, acc);
            __syncthreads();
            add_gram<RB, SLICES>(at, wave, lane, mine);
        }
        __syncthreads();                                // all have read B
    }
}

// Adds up many parts of A, in their order: 16 bytes a thread.  4.9 us for 8 x 32 parts of 128 x 128; left to
// the steps, every workgroup would read all parts.
__global__ __launch_bounds__(NT) void narrow_sum_kernel(const float* in, float* out, int32_t groups, int32_t floats) {
    const int i = ((int)blockIdx.x * NT + (int)threadIdx.x) * 4;
    if (i >= floats) return;
    const float* from = in + (int64_t)blockIdx.y * groups * floats + i;
    f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
    for (int w = 0; w < groups; ++w) s += *(const gbl_f32x4*)(from + (int64_t)w * floats);
    *(gbl_f32x4*)(out + (int64_t)blockIdx.y * floats + i) = s;
}

// Up to this many parts every workgroup adds up for itself; more go through narrow_sum_kernel.
constexpr int kOwnSums = 4;

template <int RB>
void launch(const NewtonParams& p, const NewtonPlan& plan, const NewtonCoefficients& co, hipStream_t stream) {
    const dim3 grid((uint32_t)plan.groups, (uint32_t)p.batch);
    const dim3 threads(Narrow<RB>::THREADS);
    const int floats = RB * RB * 1024;
    NarrowParams q = {};
    q.p = p;
    q.groups = plan.groups;
    q.chunks = plan.chunks;
    q.per_group = plan.per_group;
    q.tall = plan.tall ? 1 : 0;
    if (plan.groups == 0) {
        const dim3 all((uint32_t)p.batch);
        auto run = [&](auto kernel) { hipLaunchKernelGGL(kernel, all, threads, 0, stream, q, co); };
        auto whole = [&](auto dt) {
            constexpr int DT = decltype(dt)::value;
            co.measured ? run(narrow_whole_kernel<RB, DT, true>) : run(narrow_whole_kernel<RB, DT, false>);
        };
        if (p.dtype == kOutBf16) whole(std::integral_constant<int, kOutBf16>{});
        else if (p.dtype == kOutF16) whole(std::integral_constant<int, kOutF16>{});
        else whole(std::integral_constant<int, kOutF32>{});
        return;
    }
    launch_newton_norm(p, stream);
    q.x_out = p.x[0];
    q.parts_out = (float*)p.a;
    if (p.dtype == kOutBf16) hipLaunchKernelGGL((narrow_first_kernel<RB, kOutBf16>), grid, threads, 0, stream, q, co);
    else if (p.dtype == kOutF16) hipLaunchKernelGGL((narrow_first_kernel<RB, kOutF16>), grid, threads, 0, stream, q, co);
    else hipLaunchKernelGGL((narrow_first_kernel<RB, kOutF32>), grid, threads, 0, stream, q, co);
    // the parts of one step are read while the next ones are written: two sets in turn
    const size_t half = plan.a_bytes / 2;
    for (int s = 0; s < p.steps; ++s) {
        const bool last = s + 1 == p.steps;
        q.parts_in = (const float*)(p.a + (s & 1 ? half : 0));
        q.parts_out = (float*)(p.a + (s & 1 ? 0 : half));
        q.groups_in = plan.groups;
        if (plan.groups > kOwnSums) {
            hipLaunchKernelGGL(narrow_sum_kernel, dim3((uint32_t)(floats / 4 / NT), (uint32_t)p.batch), dim3(NT), 0, stream,
                               q.parts_in, (float*)p.b, plan.groups, floats);
            q.parts_in = (const float*)p.b;
            q.groups_in = 1;
        }
        q.x_in = p.x[s & 1];
        q.x_out = p.x[(s + 1) & 1];
        q.step = s;
        for (int u = 0; u < 3; ++u) q.co[u] = co.v[3 * s + u];
        auto run = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, threads, 0, stream, q); };
        if (co.measured) last ? run(narrow_step_kernel<RB, true, true>) : run(narrow_step_kernel<RB, false, true>);
        else last ? run(narrow_step_kernel<RB, true, false>) : run(narrow_step_kernel<RB, false, false>);
    }
}

}  // namespace

void newton_narrow_plan(int32_t batch, int64_t r, int64_t c, NewtonPlan* plan) {
    const int64_t rb = r <= 64 ? 2 : 4;
    plan->split = true;
    plan->tile = 0;
    plan->r = 32 * rb;
    plan->chunks = (int32_t)((c + CHUNK - 1) / CHUNK);
    plan->c = (int64_t)plan->chunks * CHUNK;
    // One workgroup a matrix while that is quicker than a workgroup a chunk: 16 x 48 x 384, three chunks, takes 51 us
    // against 44, but 200 x 60 x 500, four, 76 against 110.
    if (plan->chunks <= (rb == 2 ? (batch >= 64 ? kWholeChunks<2> : 2) : kWholeChunks<4>)) {
        plan->total = 256;                               // everything in LDS; a workspace is asked for all the same
        return;
    }
    // a workgroup of one chunk each until they are two rounds of the chip's 256 compute units
    const int64_t total = (int64_t)plan->chunks * batch;
    plan->per_group = (int32_t)(total <= 512 ? 1 : (total + 511) / 512);
    plan->groups = (plan->chunks + plan->per_group - 1) / plan->per_group;
    plan->x_bytes = (size_t)batch * plan->chunks * SLICES * rb * 2048;
    plan->a_bytes = (size_t)2 * batch * plan->groups * rb * rb * 4096;
    plan->b_bytes = (size_t)batch * rb * rb * 4096;
    plan->total = plan->parts_bytes + 2 * plan->x_bytes + plan->a_bytes + plan->b_bytes + plan->scales_bytes;
}

void launch_newton_narrow(const NewtonParams& p, const NewtonPlan& plan, const NewtonCoefficients& co, hipStream_t stream) {
    if (plan.r == 64) launch<2>(p, plan, co, stream);
    else launch<4>(p, plan, co, stream);
}

}  // namespace kgw
