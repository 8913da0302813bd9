// Newton-Schulz orthogonalisation of matrices whose short side is at most 128 (gfx950).
//
// Such a matrix has so little work that launches and the way through memory decide its time, so a
// step is one launch: every workgroup holds all r rows of its columns, squares the r x r matrix A = X X^T for itself
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
    float a_scale;          // 2^10 A = a_scale * sum of the parts
    float b_scale, b_linear;// 2^7 B = b_scale * (A A + b_linear * A), in the planes' scales
    float x_scale, linear;  // X = x_scale * (B X + linear * X)
};

// 8 sums of one lane -> its 16 bytes of a fragment, high and low plane.
__device__ __forceinline__ void split_eight(const float (&v)[8], i32x4& hi, i32x4& lo) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        hi[u] = (int)pack_f16x2(v[2 * u], v[2 * u + 1]);
        lo[u] = (int)pack_f16x2(v[2 * u] - f16_lo((uint32_t)hi[u]), v[2 * u + 1] - f16_hi((uint32_t)hi[u]));
    }
}

// RB: blocks of 32 rows of the short side (2 or 4).
template <int RB>
struct Narrow {
    static constexpr int MINE = RB * RB / 4;                    // blocks of an r x r matrix a wave has
    static constexpr uint32_t X_BYTES = SLICES * RB * 2048u;    // one chunk of the iterate
    static constexpr uint32_t A_BYTES = RB * 2 * RB * 2048u;    // an r x r matrix
    // A wave's blocks: rows block (of fragments), columns block j.
    static __device__ __forceinline__ int row_of(int wave, int) { return RB == 4 ? wave : wave >> 1; }
    static __device__ __forceinline__ int col_of(int wave, int j) { return RB == 4 ? j : wave & 1; }
    // Fragment of rows block `rows`, slice `k` of 16 K values, in a chunk of X or in A.
    static __device__ __forceinline__ uint32_t x_at(int k, int rows, int plane) { return (uint32_t)((k * RB + rows) * 2 + plane) * 1024u; }
    static __device__ __forceinline__ uint32_t a_at(int k, int rows, int plane) { return x_at(k, rows, plane); }
};

// sums += three products of the fragments (hi, lo) x (hi, lo).
__device__ __forceinline__ f32x16 mfma3(i32x4 ah, i32x4 al, i32x4 bh, i32x4 bl, f32x16 c) {
    c = mfma_f16_32x32x16(ah, bl, c);
    c = mfma_f16_32x32x16(al, bh, c);
    return mfma_f16_32x32x16(ah, bh, c);
}

// Adds this wave's blocks of X X^T over a chunk in LDS to acc.
template <int RB>
__device__ __forceinline__ void add_gram(const lds_char* x, int wave, int lane, f32x16 (&acc)[Narrow<RB>::MINE]) {
    using N = Narrow<RB>;
#pragma unroll
    for (int k = 0; k < SLICES; ++k) {
        const i32x4 rh = lds_load_16B(x, N::x_at(k, N::row_of(wave, 0), 0) + lane * 16u);
        const i32x4 rl = lds_load_16B(x, N::x_at(k, N::row_of(wave, 0), 1) + lane * 16u);
#pragma unroll
        for (int j = 0; j < N::MINE; ++j) {
            const i32x4 ch = lds_load_16B(x, N::x_at(k, N::col_of(wave, j), 0) + lane * 16u);
            const i32x4 cl = lds_load_16B(x, N::x_at(k, N::col_of(wave, j), 1) + lane * 16u);
            acc[j] = mfma3(ch, cl, rh, rl, acc[j]);     // columns block down the registers, rows over the lanes
        }
    }
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

// The first iterate's chunks and their parts of A.
template <int RB, int DT>
__global__ __launch_bounds__(NT, 1) void narrow_first_kernel(NarrowParams q) {
    using N = Narrow<RB>;
    __shared__ __attribute__((aligned(1024))) char smem[N::X_BYTES];
    lds_char* const x = (lds_char*)smem;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int b = blockIdx.y, group = blockIdx.x;
    const float scale = first_scale(q.p, b);
    f32x16 acc[N::MINE];
#pragma unroll
    for (int j = 0; j < N::MINE; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[j][e] = 0.0f;
    const int first = group * q.per_group, last = min(q.chunks, first + q.per_group);
    for (int chunk = first; chunk < last; ++chunk) {
        const int64_t n0 = (int64_t)chunk * CHUNK;
        __syncthreads();
        if (!q.tall) {
            // eight consecutive columns of one row: two runs of four, for the two lane halves
            for (int i = tid; i < 32 * RB * (CHUNK / 8); i += NT) {
                const int row = i / (CHUNK / 8), c8 = i % (CHUNK / 8);
                float v[8];
                load_eight<DT>(q.p, b, row, n0 + 8 * c8, v);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= scale;
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
            for (int i = tid; i < CHUNK * 4 * RB; i += NT) {
                const int col = i / (4 * RB), r8 = i % (4 * RB);
                float v[8];
                load_eight<DT>(q.p, b, n0 + col, 8 * r8, v);
                const int in = col & 15;                         // column 4 h + 8 s + t: half h, run s, place t
                const uint32_t place = (uint32_t)((in >> 2) & 1) * 512u + (uint32_t)(in >> 3) * 8u + (uint32_t)(in & 3) * 2u;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int row = 8 * r8 + e;
                    const float u = v[e] * scale;
                    const uint32_t hi = pack_f16x2(u, 0.0f);
                    const uint32_t lo = pack_f16x2(u - f16_lo(hi), 0.0f);
                    const uint32_t at = place + (uint32_t)(row & 31) * 16u;
                    *reinterpret_cast<__attribute__((address_space(3))) uint16_t*>(x + N::x_at(col >> 4, row >> 5, 0) + at) = (uint16_t)hi;
                    *reinterpret_cast<__attribute__((address_space(3))) uint16_t*>(x + N::x_at(col >> 4, row >> 5, 1) + at) = (uint16_t)lo;
                }
            }
        }
        __syncthreads();
        char* const to = q.x_out + ((int64_t)b * q.chunks + chunk) * N::X_BYTES;
        for (uint32_t i = tid * 16u; i < N::X_BYTES; i += NT * 16u) *(gbl_i32x4*)(to + i) = lds_load_16B(x, i);
        add_gram<RB>(x, wave, lane, acc);
    }
    store_part<RB>(q, b, group, wave, lane, acc);
}

// One step.  LAST: the result instead of the next iterate and its part of A.
template <int RB, bool LAST>
__global__ __launch_bounds__(NT, 1) void narrow_step_kernel(NarrowParams q) {
    using N = Narrow<RB>;
    __shared__ __attribute__((aligned(1024))) char smem[N::X_BYTES + N::A_BYTES];
    lds_char* const x = (lds_char*)smem;
    lds_char* const a = x + N::X_BYTES;
    const uint32_t x_addr = lds_addr(smem);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l32 = lane & 31, lhi = lane >> 5, g16 = lane >> 4, i16 = lane & 15;
    const int b = blockIdx.y, group = blockIdx.x;
    const int first = group * q.per_group, last = min(q.chunks, first + q.per_group);

    auto load_chunk = [&](int chunk) __attribute__((always_inline)) {
        const i32x4 r = rsrc_words(q.x_in + ((int64_t)b * q.chunks + chunk) * N::X_BYTES);
#pragma unroll
        for (uint32_t t = 0; t < N::X_BYTES / 4096; ++t) {
            const uint32_t at = (wave * (N::X_BYTES / 4096) + t) * 1024u;
            dma_16B(r, at + lane * 16u, x_addr + at);
        }
    };
    load_chunk(first);

    // A: this wave's blocks, added up in the order of the parts
    f32x16 mine[N::MINE];
    {
        const float* from = q.parts_in + (int64_t)b * q.groups_in * (RB * RB * 1024);
#pragma unroll
        for (int j = 0; j < N::MINE; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) mine[j][e] = 0.0f;
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
    }
    // Blocks of an r x r matrix as fragments into LDS: rows over the lanes, K = columns.
    auto write_blocks = [&](const f32x16 (&m)[N::MINE]) __attribute__((always_inline)) {
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
    };
#pragma unroll
    for (int j = 0; j < N::MINE; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) mine[j][e] *= q.a_scale;
    write_blocks(mine);
    __syncthreads();
    // B = b_scale (A A + b_linear A)
    f32x16 square[N::MINE];
#pragma unroll
    for (int j = 0; j < N::MINE; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) square[j][e] = q.b_linear * mine[j][e];
#pragma unroll
    for (int k = 0; k < 2 * RB; ++k) {
        const i32x4 rh = lds_load_16B(a, N::a_at(k, N::row_of(wave, 0), 0) + lane * 16u);
        const i32x4 rl = lds_load_16B(a, N::a_at(k, N::row_of(wave, 0), 1) + lane * 16u);
#pragma unroll
        for (int j = 0; j < N::MINE; ++j) {
            const i32x4 ch = lds_load_16B(a, N::a_at(k, N::col_of(wave, j), 0) + lane * 16u);
            const i32x4 cl = lds_load_16B(a, N::a_at(k, N::col_of(wave, j), 1) + lane * 16u);
            square[j] = mfma3(ch, cl, rh, rl, square[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < N::MINE; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) square[j][e] *= q.b_scale;
    __syncthreads();
    write_blocks(square);

    f32x16 part[N::MINE];
#pragma unroll
    for (int j = 0; j < N::MINE; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) part[j][e] = 0.0f;
    for (int chunk = first; chunk < last; ++chunk) {
        wait_vmcnt<0>();
        __syncthreads();                                // the chunk and B are in LDS
        // this wave's 32 columns: rows of X over K, columns down the registers, rows of the result over the lanes
        f32x16 acc[RB];
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][e] = 0.0f;
#pragma unroll
        for (int k = 0; k < 2 * RB; ++k) {
            // Transposed fragment of rows 16 k .. of X: 16 lanes read 4 rows x 16 columns, of which
            // piece c (4 columns) of a row is half c & 1, run c >> 1 of its place in the image.
            i32x4 xt[2];
#pragma unroll
            for (int plane = 0; plane < 2; ++plane) {
                const int slice = 2 * wave + (g16 & 1), c = i16 & 3;
                const int row = 16 * k + 4 * (g16 >> 1) + (i16 >> 2);
                const uint32_t at = N::x_at(slice, 0, plane) + (uint32_t)(k >> 1) * 2048u + (uint32_t)(c & 1) * 512u +
                                    (uint32_t)(row & 31) * 16u + (uint32_t)(c >> 1) * 8u;
                const i16x4 v0 = lds_read_tr16(x, at);
                const i16x4 v1 = lds_read_tr16(x, at + 8 * 16);
                const i16x8 v = {v0[0], v0[1], v0[2], v0[3], v1[0], v1[1], v1[2], v1[3]};
                xt[plane] = __builtin_bit_cast(i32x4, v);
            }
#pragma unroll
            for (int i = 0; i < RB; ++i) {
                const i32x4 bh = lds_load_16B(a, N::a_at(k, i, 0) + lane * 16u);
                const i32x4 bl = lds_load_16B(a, N::a_at(k, i, 1) + lane * 16u);
                acc[i] = mfma3(xt[0], xt[1], bh, bl, acc[i]);
            }
        }
        // a X from the same image, added last: it decides the small singular values
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const i32x4 hi = lds_load_16B(x, N::x_at(2 * wave + s, i, 0) + lane * 16u);
                const i32x4 lo = lds_load_16B(x, N::x_at(2 * wave + s, i, 1) + lane * 16u);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    acc[i][8 * s + 2 * u] = q.x_scale * (acc[i][8 * s + 2 * u] + q.linear * (f16_lo((uint32_t)hi[u]) + f16_lo((uint32_t)lo[u])));
                    acc[i][8 * s + 2 * u + 1] = q.x_scale * (acc[i][8 * s + 2 * u + 1] + q.linear * (f16_hi((uint32_t)hi[u]) + f16_hi((uint32_t)lo[u])));
                }
            }
        __syncthreads();                                // all have read the chunk
        if constexpr (LAST) {
            if (chunk + 1 < last) load_chunk(chunk + 1);
            const int64_t c0 = (int64_t)chunk * CHUNK + 32 * wave + 4 * lhi;
#pragma unroll
            for (int i = 0; i < RB; ++i) {
                const int64_t row = 32 * i + l32;
#pragma unroll
                for (int g = 0; g < 4; ++g)
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const int64_t col = c0 + 8 * g + t;
                        const int64_t gr = q.tall ? col : row, gc = q.tall ? row : col;
                        if (gr >= q.p.m || gc >= q.p.n) continue;
                        const int64_t at = ((int64_t)b * q.p.m + gr) * q.p.n + gc;
                        const float v = acc[i][4 * g + t];
                        if (q.p.out_dtype == kOutF32) ((float*)q.p.out)[at] = v;
                        else if (q.p.out_dtype == kOutBf16) ((uint16_t*)q.p.out)[at] = (uint16_t)pack_bf16x2(v, 0.0f);
                        else ((uint16_t*)q.p.out)[at] = (uint16_t)pack_f16x2(v, 0.0f);
                    }
            }
        } else {
            char* const to = q.x_out + ((int64_t)b * q.chunks + chunk) * N::X_BYTES;
#pragma unroll
            for (int i = 0; i < RB; ++i)
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = acc[i][8 * s + e];
                    i32x4 hi, lo;
                    split_eight(v, hi, lo);
                    const uint32_t at = N::x_at(2 * wave + s, i, 0) + lane * 16u;
                    lds_store_16B(x, at, hi);
                    lds_store_16B(x, at + 1024u, lo);
                    *(gbl_i32x4*)(to + at) = hi;
                    *(gbl_i32x4*)(to + at + 1024u) = lo;
                }
            __syncthreads();
            add_gram<RB>(x, wave, lane, part);
            if (chunk + 1 < last) {
                __syncthreads();                        // all have read the image
                load_chunk(chunk + 1);
            }
        }
    }
    if constexpr (!LAST) store_part<RB>(q, b, group, wave, lane, part);
}

// Adds up many parts of A, in their order: 16 bytes a thread.
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
void launch(const NewtonParams& p, const NewtonPlan& plan, const float* co, hipStream_t stream) {
    const dim3 grid((uint32_t)plan.groups, (uint32_t)p.batch);
    const int floats = RB * RB * 1024;
    NarrowParams q = {};
    q.p = p;
    q.groups = plan.groups;
    q.chunks = plan.chunks;
    q.per_group = plan.per_group;
    q.tall = plan.tall ? 1 : 0;
    q.x_out = p.x[0];
    q.parts_out = (float*)p.a;
    if (p.dtype == kOutBf16) hipLaunchKernelGGL((narrow_first_kernel<RB, kOutBf16>), grid, dim3(NT), 0, stream, q);
    else if (p.dtype == kOutF16) hipLaunchKernelGGL((narrow_first_kernel<RB, kOutF16>), grid, dim3(NT), 0, stream, q);
    else hipLaunchKernelGGL((narrow_first_kernel<RB, kOutF32>), grid, dim3(NT), 0, stream, q);
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
        const float c = newton_c(co + 3 * s);
        q.x_in = p.x[s & 1];
        q.x_out = p.x[(s + 1) & 1];
        q.a_scale = kAScale / (kXScale * kXScale);
        q.b_scale = c * (kBScale / (kAScale * kAScale));
        q.b_linear = c != 0.0f ? co[3 * s + 1] / c * kAScale : 0.0f;
        q.x_scale = (last ? 1.0f / kXScale : 1.0f) / kBScale;
        q.linear = co[3 * s] * kBScale;
        if (last) hipLaunchKernelGGL((narrow_step_kernel<RB, true>), grid, dim3(NT), 0, stream, q);
        else hipLaunchKernelGGL((narrow_step_kernel<RB, false>), grid, dim3(NT), 0, stream, q);
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
    // a workgroup of one chunk each until they are two rounds of the chip's 256 compute units
    const int64_t total = (int64_t)plan->chunks * batch;
    plan->per_group = (int32_t)(total <= 512 ? 1 : (total + 511) / 512);
    plan->groups = (plan->chunks + plan->per_group - 1) / plan->per_group;
    plan->x_bytes = (size_t)batch * plan->chunks * SLICES * rb * 2048;
    plan->a_bytes = (size_t)2 * batch * plan->groups * rb * rb * 4096;
    plan->b_bytes = (size_t)batch * rb * rb * 4096;
    plan->total = plan->parts_bytes + 2 * plan->x_bytes + plan->a_bytes + plan->b_bytes;
}

void launch_newton_narrow(const NewtonParams& p, const NewtonPlan& plan, const float* coefficients, hipStream_t stream) {
    launch_newton_norm(p, stream);
    if (plan.r == 64) launch<2>(p, plan, coefficients, stream);
    else launch<4>(p, plan, coefficients, stream);
}

}  // namespace kgw
