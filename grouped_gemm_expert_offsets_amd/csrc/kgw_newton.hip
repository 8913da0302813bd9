// Newton-Schulz orthogonalisation of a batch of matrices (gfx950), the update of a
// weight gradient:
//
//     X_0 = G / (|G|_F + eps)                     (transposed when m > n, so r <= c)
//     A = X X^T,   B = b A + c A A,   X <- a X + B X,   `steps` times
//
// The iterate is held as two fp16 planes, X = (hi + lo) / 2^(13 - e): hi is X rounded to 11 bits, lo
// the remainder rounded again, 22 bits together, so the linear term a X, which multiplies
// small singular values by a at every step, keeps those.  The products run on the matrix cores in fp16
// with fp32 sums:
//   one product each (results rounded to bf16): A = hi hi^T, B from fp16 A, B hi.  The
//     operands' rounding (2^-12) enters only through B X, which is small where the singular values are, and
//     leaves 0.3e-3 (4096 x 7168, power law) to 1.8e-3 (129 x 129, normal) of the result's norm beside bf16's own
//     rounding of 1.66e-3: 1.69e-3 to 2.45e-3 in all.  bf16 operands would leave 4e-3 .. 2e-2.
//   three products each (fp32 and fp16 results, bf16 ones where asked for): every matrix as hi + lo, hi hi + hi lo + lo hi;
//     the dropped lo lo is 2^-24 of the product.  1e-6 .. 1e-5, what fp32 arithmetic leaves.
// Powers of two keep the planes inside fp16's range, chosen for every matrix and step from a bound 2^e on its singular
// values (step_scales()): 1 for the first iterate, less where eps outweighs the norm, then the largest value the
// step's polynomial takes up to there.  Where bounds say too little (kBoundLoss) A's norm is measured in every step, by two
// more launches.
//
// A and A A are symmetric: only tiles on and below the diagonal are computed and their mirror
// images written along, which leaves 3 r^2 c + r^3 multiply-adds of a step's 4 r^2 c + 2 r^3 over two.
//
// What bounds it: 8 x 7168 x 4096 takes 16.7 ms to bf16 (17.2 TFLOP with the halves counted, 1.03 PFLOP/s;
// the library's 8192^3 fp16 product runs at 1.09 here) and 39 ms to fp32 (1.32 PFLOP/s).  There it is the
// card's power: the matrix cores are busy 60 to 76% of the time at 1.6 GHz, and with matrices of zeros,
// whose products cost less energy, the same launches take 14.4 and 28.3 ms.  Small ones are bound by
// their 17 launches and by one tile's way through K: 4 x 256 x 512 to fp32 125 us.
//
// Sides up to 128 take the kernels of kgw_newton_narrow.hip.
#include "kgw_newton_device.h"

namespace kgw {
namespace {

constexpr int NT = 256;
static_assert(kNewtonSlabs <= NT, "one workgroup clears the counters");

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

// Eight consecutive elements of one row of a stored matrix, as one or two planes of halves.
template <bool TWO>
__device__ __forceinline__ void store_planes(const float (&v)[8], uint16_t* out, int64_t lo_off) {
    i32x4 h, l;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const HalfPair p = split_pair(v[2 * u], v[2 * u + 1]);
        h[u] = (int)p.hi;
        if constexpr (TWO) l[u] = (int)p.lo;
    }
    *(gbl_i32x4*)out = h;
    if constexpr (TWO) *(gbl_i32x4*)(out + lo_off) = l;
}

// ----------------------------------------------------------------------------
// |G|_F and the first iterate
// ----------------------------------------------------------------------------
// Sum of squares of this workgroup's share of one matrix, in 64 bits: gradients may be so large or
// small that their squares leave fp32's range.  Bound by HBM: 93 us for 8 x 7168 x 4096 bf16, 5.1 TB/s.
template <int DT>
__global__ __launch_bounds__(NT) void newton_norm_kernel(NewtonParams p) {
    __shared__ double sums[NT / 64];
    const int tid = threadIdx.x, b = blockIdx.y;
    const uint32_t per_row = (uint32_t)((p.n + 7) / 8);
    const int64_t pieces = p.m * (int64_t)per_row;
    double s = 0.0;
#pragma unroll 2
    for (int64_t i = (int64_t)blockIdx.x * NT + tid; i < pieces; i += (int64_t)p.num_parts * NT) {
        const int64_t row = i >> 32 ? i / per_row : (uint32_t)i / per_row;
        float v[8];
        load_eight<DT>(p, b, row, 8 * (i - row * per_row), v);
#pragma unroll
        for (int u = 0; u < 8; ++u) s += (double)v[u] * (double)v[u];
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d);
    if ((tid & 63) == 0) sums[tid >> 6] = s;
    __syncthreads();
    if (p.arrived && blockIdx.x == 0 && b == 0 && tid < kNewtonSlabs) p.arrived[tid] = 0;
    if (tid == 0) p.parts[(int64_t)b * kNewtonParts + blockIdx.x] = (sums[0] + sums[1]) + (sums[2] + sums[3]);
}

// One 64 x 64 tile of the padded first iterate.  Bound by HBM: reads 2 bytes an element and writes 4,
// 262 us for 8 x 7168 x 4096 bf16, 5.4 TB/s; transposed through LDS it takes as long.
template <int DT, bool SPLIT, bool TALL>
__global__ __launch_bounds__(NT) void newton_first_kernel(NewtonParams p, NewtonCoefficients co, int64_t R, int64_t C) {
    __shared__ float tile[TALL ? 64 : 1][65];
    const int b = blockIdx.z, i0 = threadIdx.x >> 3, q = threadIdx.x & 7;
    const int64_t r0 = (int64_t)blockIdx.y * 64, c0 = (int64_t)blockIdx.x * 64;
    const bool writes = blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 64;
    if (writes) write_unit_scales(p, co, b);
    float v[2][8];
#pragma unroll
    for (int u = 0; u < 2; ++u) load_eight<DT>(p, b, (TALL ? c0 : r0) + i0 + 32 * u, (TALL ? r0 : c0) + 8 * q, v[u]);
    const FirstScale scale = first_scale(p, b);
    if constexpr (TALL) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e) tile[8 * q + e][i0 + 32 * u] = v[u][e];
        __syncthreads();
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[u][e] = tile[i0 + 32 * u][8 * q + e];
    }
    uint16_t* const x = (uint16_t*)p.x[0] + (int64_t)b * R * C * (SPLIT ? 2 : 1);
    const int64_t lo_off = SPLIT ? 32 : (int64_t)p.batch * R * C;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[u][e] = scale.of(v[u][e]);
        store_planes<true>(v[u], x + element<SPLIT>(r0 + i0 + 32 * u, c0 + 8 * q, C), lo_off);
    }
    if (writes) write_scales(p, co, b, scale);
}

// Scales measured on A, for coefficients whose bounds say too little (kBoundLoss): the sum of squares of A's high plane in
// parts, and from them the step's scales.
template <bool SPLIT>
__global__ __launch_bounds__(NT) void newton_measure_kernel(NewtonParams p, int64_t R, int32_t parts) {
    __shared__ double sums[NT / 64];
    const int tid = threadIdx.x, b = blockIdx.y;
    const uint16_t* const a = (const uint16_t*)p.a + (int64_t)b * R * R * (SPLIT ? 2 : 1);
    const int per_row = (int)(R / 8);
    double s = 0.0;
    for (int64_t i = (int64_t)blockIdx.x * NT + tid; i < R * per_row; i += (int64_t)parts * NT) {
        const int64_t row = i / per_row;
        const i32x4 x = *(const gbl_i32x4*)(a + element<SPLIT>(row, 8 * (i - row * per_row), R));
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const double lo = f16_lo((uint32_t)x[u]), hi = f16_hi((uint32_t)x[u]);
            s += lo * lo + hi * hi;
        }
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d);
    if ((tid & 63) == 0) sums[tid >> 6] = s;
    __syncthreads();
    if (tid == 0) p.parts[(int64_t)b * kNewtonParts + blockIdx.x] = (sums[0] + sums[1]) + (sums[2] + sums[3]);
}
__global__ __launch_bounds__(64) void newton_scales_kernel(NewtonParams p, NewtonCoefficients co, int32_t step, int32_t parts) {
    const int b = blockIdx.x;
    double s = 0.0;
    for (int i = threadIdx.x; i < parts; i += 64) s += p.parts[(int64_t)b * kNewtonParts + i];
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d);
    SingularBound bound = measured_bound(s, p.planes[(int64_t)(step & 1) * p.batch + b]);
    const StepScales r = step_scales(bound, co.v + 3 * step, step + 1 == p.steps);
    if (threadIdx.x == 0) {
        p.scales[(int64_t)b * kNewtonMaxSteps + step] = r;
        p.planes[(int64_t)(~step & 1) * p.batch + b] = bound.plane;
    }
}

// ----------------------------------------------------------------------------
// the products
// ----------------------------------------------------------------------------
enum NewtonProduct { kGram, kSquare, kUpdate, kLast };   // kLast: the last update, which writes the result
__device__ __forceinline__ float as_uniform(float x) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, x)));
}
constexpr bool updates(NewtonProduct k) { return k == kUpdate || k == kLast; }

struct NewtonGemm {
    const char* left;       // (batch, R, K) rows of the product
    const char* right;      // gram, square: left again; update: the iterate (batch, K, C)
    char* out;              // gram: A; square: B; update: the next iterate
    void* result;           // last update: (batch, m, n) of result_dtype
    int64_t m, n;
    int32_t result_dtype, tall;
    const StepScales* scales;  // of this step, every kNewtonMaxSteps-th one: out = scale * (product + linear * (square: A;
                               // update: the iterate)); gram: kGramScale * product
    int64_t rows, cols, k;  // padded sizes of the product
    int32_t batch, tiles_m, tiles_n;
    int32_t items;          // workgroups with work
    int32_t whole;          // the first of them: one tile each; the others a quarter of one
    int32_t tiles;          // of 256 x 256 in all matrices
    int32_t strips;         // quarters of one matrix beside its tiles
    int32_t parts;          // workgroups that share a tile's K (small tiles of the symmetric products)
    float* slabs;           // their sums, one tile each
    uint32_t* arrived;      // per tile, zero between launches
    int32_t num_xcds;
};

// Item of workgroup bid of `items`: workgroups are dealt to the XCDs in turn, and one XCD's get a
// contiguous run of items, so that the tiles it works on at a time share panels in its L2.
__device__ __forceinline__ int item_of(int bid, int items, int num_xcds) {
    const int each = items / num_xcds, more = items - each * num_xcds, x = bid % num_xcds;
    return x * each + min(x, more) + bid / num_xcds;
}

// The update's tiles come in columns of this many rows of tiles; all of one group walk K alike, so that
// they share the iterate's panels in L2 (each starting behind its own rows cost 4% of the update).
constexpr int kRowGroup = 4;
template <bool SPLIT, NewtonProduct KIND>
__device__ __forceinline__ int turn_of(const NewtonGemm& p, int tm, int tile) {
    if (!SPLIT || !updates(KIND)) return 0;
    const int rows = tile == 256 ? kRowGroup : 1;
    const int end = min((tm / rows + 1) * rows, p.tiles_m);
    return end == p.tiles_m ? 0 : end * tile / 32;
}

// Tile `index` of a product with tiles_m x tiles_n tiles a matrix: all of them (update), or those on
// and below the diagonal.
template <NewtonProduct KIND>
__device__ __forceinline__ void tile_of(const NewtonGemm& p, int index, int& b, int& tm, int& tn) {
    const int per = updates(KIND) ? p.tiles_m * p.tiles_n : p.tiles_m * (p.tiles_m + 1) / 2;
    b = index / per;
    const int local = index - b * per;
    if constexpr (updates(KIND)) {
        tile_coords(local, p.tiles_m, p.tiles_n, kRowGroup, tm, tn);
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

// Eight consecutive elements of the result, those inside it: `row`, `col` behind the wave's row0, col0, which
// make the address's uniform part.
template <int DT>
__device__ __forceinline__ void store_result(const NewtonGemm& p, const float (&v)[8], int b, int64_t row0, int64_t col0,
                                             int row, int col) {
    const int left = (int)(p.n - col0) - col;           // sizes are at most 2^20
    if (row >= (int)(p.m - row0) || left <= 0) return;
    const int64_t at0 = ((int64_t)b * p.m + row0) * p.n + col0;
    const uint32_t at = (uint32_t)row * (uint32_t)p.n + (uint32_t)col;
    if constexpr (DT == kOutF32) {
        float* const to = (float*)p.result + at0 + at;
        if (left >= 8) {
            ((__attribute__((address_space(1))) Floats4*)to)[0].v = f32x4{v[0], v[1], v[2], v[3]};
            ((__attribute__((address_space(1))) Floats4*)to)[1].v = f32x4{v[4], v[5], v[6], v[7]};
        } else {
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (u < left) to[u] = v[u];
        }
    } else {
        uint16_t* const to = (uint16_t*)p.result + at0 + at;
        i32x4 w;
#pragma unroll
        for (int u = 0; u < 4; ++u) w[u] = (int)pack_half2<DT>(v[2 * u], v[2 * u + 1]);
        if (left >= 8) {
            ((__attribute__((address_space(1))) Halves8*)to)->v = w;
        } else {
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (u < left) to[u] = (uint16_t)(((uint32_t)w[u >> 1] >> (16 * (u & 1))) & 0xFFFFu);
        }
    }
}

// Puts this workgroup's sums down beside those of the other parts of its tile's K.  The last one to arrive adds
// all of them up, in the order of the parts whoever is last, and goes on with the tile (true).  No one
// waits: a workgroup that is not the last is done.
//
// The parts of a tile may run on different dies, whose L2 caches do not see each other's stores.  The sums
// therefore go out and come back as device-scope accesses, which are performed beyond those caches; a store
// counts as done (vmcnt) only there, so waiting for the own stores before counting the arrival is all the
// release that is needed.  A fence would write back each die's whole L2 for every workgroup: with 216
// workgroups of 64 KiB it made a product of 35 us take 57.
template <int WAVES, int NBM, int NBN>
__device__ bool join_parts(const NewtonGemm& p, char* smem, int tile, int part, int wave, int lane,
                           f32x16 (&acc)[NBN][NBM]) {
    constexpr int WAVE = NBM * NBN * 1024;              // floats of one wave
    float* const tile_slabs = p.slabs + (int64_t)tile * p.parts * (WAVES * WAVE) + wave * WAVE + lane;
    float* const own = tile_slabs + part * (WAVES * WAVE);
#pragma unroll
    for (int j = 0; j < NBN; ++j)
#pragma unroll
        for (int i = 0; i < NBM; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                __hip_atomic_store(own + ((j * NBM + i) * 16 + e) * 64, acc[j][i][e], __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("" ::: "memory");
    wait_vmcnt<0>();
    barrier_no_fence();                                 // every wave's sums are down
    uint32_t* const last = (uint32_t*)smem;
    if (threadIdx.x == 0)
        *last = __hip_atomic_fetch_add(p.arrived + tile, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                        (uint32_t)p.parts - 1u
                    ? 1u
                    : 0u;
    __syncthreads();
    const bool is_last = *last != 0;
    __syncthreads();                                    // smem is free again
    if (!is_last) return false;
    if (threadIdx.x == 0) __hip_atomic_store(p.arrived + tile, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
    for (int j = 0; j < NBN; ++j)
#pragma unroll
        for (int i = 0; i < NBM; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[j][i][e] = 0.0f;
    for (int w = 0; w < p.parts; ++w) {
        const float* const from = tile_slabs + w * (WAVES * WAVE);
#pragma unroll
        for (int j = 0; j < NBN; ++j)
#pragma unroll
            for (int i = 0; i < NBM; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    acc[j][i][e] += __hip_atomic_load(from + ((j * NBM + i) * 16 + e) * 64, __ATOMIC_RELAXED,
                                                      __HIP_MEMORY_SCOPE_AGENT);
    }
    return true;
}

// One TILE x TILE tile at rows m0 and columns n0 of matrix b.  A stage of the K loop is a 128-byte line
// of every row of the left tile (64 halves of K, or 32 of both planes) and as many bytes of the right
// one, in a ring of SLOTS.  Left tiles, and the right ones of the symmetric products, are read as
// K-contiguous rows with 16-byte chunk q of row i in slot q ^ ((i >> 1) & 7); the iterate's rows (K
// across them) through the transposing reads, chunk q of row k in slot q ^ 4 (k & 3).  Both keep every
// read free of bank conflicts.
//
// A stage is four (six) groups of matrix products; each group's fragments are read while the group before
// multiplies.  Before the last group every read of the stage is done, so the barrier that hands the
// slot over stands there, and the next stage's first fragments and the loads that refill the
// ring go out under the last group's products.
template <int TILE, int WAVES, int SLOTS, bool SPLIT, bool JOIN, NewtonProduct KIND>
__device__ __forceinline__ void newton_tile(const NewtonGemm& p, char* smem, int b, int64_t m0, int64_t n0, int turn,
                                            int tile = 0, int part = 0) {
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
    const int64_t ldr = (updates(KIND) ? p.cols : p.k) * (SPLIT ? 4 : 2);       // of a right row
    const char* const left = p.left + ((int64_t)b * p.rows + m0) * ldl;
    const char* const right = updates(KIND) ? p.right + (int64_t)b * p.k * ldr + n0 * (SPLIT ? 4 : 2)
                                              : p.right + ((int64_t)b * p.rows + n0) * ldr;

    float scale = kGramScale, linear = 0.0f;
    if constexpr (KIND != kGram) {
        const float* const at = (const float*)(p.scales + (int64_t)b * kNewtonMaxSteps) + (updates(KIND) ? 2 : 0);
        scale = as_uniform(at[0]);
        linear = as_uniform(at[1]);
    }

    uint32_t l_off[LOADS], r_off[LOADS];
#pragma unroll
    for (int t = 0; t < LOADS; ++t) {
        const int row = (wave * LOADS + t) * 8 + (lane >> 3);
        const uint32_t chunk = (uint32_t)((lane & 7) ^ ((row >> 1) & 7));
        l_off[t] = (uint32_t)row * (uint32_t)ldl + chunk * 16u;
        if constexpr (updates(KIND)) {
            const int at = (wave * LOADS + t) * 64 + lane;
            const int krow = at / CPR;
            r_off[t] = (uint32_t)krow * (uint32_t)ldr + (uint32_t)((at % CPR) ^ (((krow & 3) << 2) & (CPR - 1))) * 16u;
        } else {
            r_off[t] = (uint32_t)row * (uint32_t)ldr + chunk * 16u;
        }
    }
    const int all_stages = (int)(p.k / KSTAGE);
    const int first_stage = JOIN ? all_stages * part / p.parts : 0;
    const int stages = JOIN ? all_stages * (part + 1) / p.parts - first_stage : all_stages;
    const int64_t r_step = updates(KIND) ? KSTAGE * ldr : 128;
    // Three products: the update walks K from stage `turn` on, so that its linear term comes late (fold()).
    // Parts of K: the stages from first_stage on (never both).
    auto place_of = [&](int s) __attribute__((always_inline)) {
        return !updates(KIND) ? first_stage + s : s + turn < stages ? s + turn : s + turn - stages;
    };
    // Slot n % SLOTS takes the n-th operand stage, left and right in turn.  Load t of slot `slot` with
    // operand stage n; past the last one an empty range (no memory is read).
    auto load_one = [&](int n, int slot, int t) __attribute__((always_inline)) {
        const uint32_t dst = lds0 + (uint32_t)(slot * STAGE + (wave * LOADS + t) * 1024);
        const uint32_t range = (n >> 1) < stages ? 0xFFFFFFFFu : 0u;
        const int at = place_of(n >> 1);
        if (n & 1) dma_16B(rsrc_words(right + at * r_step, range), r_off[t], dst);
        else dma_16B(rsrc_words(left + (int64_t)at * 128, range), l_off[t], dst);
    };

    // fragment q (0..3) of a stage: one product: K = 16 q ..; three: plane q >> 1, K = 16 (q & 1) ..
    const uint32_t l_row = (uint32_t)(wm * WTM + l32) * 128u, r_row = (uint32_t)(wn * WTN + l32) * 128u;
    const int sw = (l32 >> 1) & 7;
    const int kr = 8 * (g16 >> 1) + (i16 >> 2);
    const int cq = 2 * (g16 & 1) + ((i16 & 3) >> 1);
    auto read_left = [&](int slot, int q, int i) __attribute__((always_inline)) {
        return lds_load_16B(lds + slot * STAGE, l_row + (uint32_t)i * 4096u + (uint32_t)(((2 * q + lhi) ^ sw) << 4));
    };
    auto read_right = [&](int slot, int q, int j) __attribute__((always_inline)) {
        const lds_char* const base = lds + slot * STAGE;
        if constexpr (updates(KIND)) {
            const int chunk = SPLIT ? (wn * NBN + j) * 8 + (q >> 1) * 4 + cq : wn * (WTN / 8) + 4 * j + cq;
            const uint32_t at = (uint32_t)((SPLIT ? 16 * (q & 1) : 16 * q) + kr) * (uint32_t)ROWB +
                                (uint32_t)((chunk ^ (((i16 >> 2) << 2) & (CPR - 1))) << 4) + (uint32_t)(i16 & 1) * 8u;
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

    // The linear term's matrix passes through LDS as an operand of the product: the stages over
    // the tile's own rows (update: the iterate, right) or columns (square: A, left) hold the tile itself, and each lane
    // adds its elements to its sums from there.  a X decides the small singular values, and every
    // product summed after it rounds it once more: where the result is to be that exact, the tiles of a group of rows
    // start behind the group's own rows and meet them last.
    auto fold = [&](int s, int slot) __attribute__((always_inline)) {
        const int d = KSTAGE * place_of(s) - (int)(updates(KIND) ? m0 : n0);
        if (d < 0 || d >= TILE) return;
        const lds_char* const base = lds + slot * STAGE;
#pragma unroll
        for (int e = 0; e < KSTAGE / 32; ++e) {
            const int at = d + 32 * e;
            if (at / (updates(KIND) ? WTM : WTN) != (updates(KIND) ? wm : wn)) continue;
            const int block = at % (updates(KIND) ? WTM : WTN) / 32;
            each<PRODUCTS>([&](auto k) __attribute__((always_inline)) {
                constexpr int j = k / NBM, i = k % NBM;
                if (block != (updates(KIND) ? i : j)) return;
                // The empty asm statements differ from block to block: the compiler would otherwise merge
                // the branches' code and reach the sums through pointers, in scratch memory.
                asm volatile("; block %0" ::"n"(k.value));
#pragma unroll
                for (int g = 0; g < 4; ++g)
#pragma unroll
                    for (int plane = 0; plane < (SPLIT ? 2 : 1); ++plane) {
                        uint32_t from;
                        if constexpr (updates(KIND)) {
                            const int krow = 32 * e + l32;
                            const int chunk = SPLIT ? (wn * NBN + j) * 8 + plane * 4 + g : wn * (WTN / 8) + 4 * j + g;
                            from = (uint32_t)(krow * ROWB + ((chunk ^ (((krow & 3) << 2) & (CPR - 1))) << 4));
                        } else {
                            const int chunk = SPLIT ? plane * 4 + g : 4 * e + g;
                            from = l_row + (uint32_t)i * 4096u + (uint32_t)((chunk ^ sw) << 4);
                        }
                        const i32x2 x = lds_load_8B(base, from + (uint32_t)lhi * 8u);
                        acc[j][i][4 * g] += linear * f16_lo((uint32_t)x[0]);
                        acc[j][i][4 * g + 1] += linear * f16_hi((uint32_t)x[0]);
                        acc[j][i][4 * g + 2] += linear * f16_lo((uint32_t)x[1]);
                        acc[j][i][4 * g + 3] += linear * f16_hi((uint32_t)x[1]);
                    }
                asm volatile("; block %0" ::"n"(k.value));
            });
        }
    };

    struct Left { i32x4 v[NBM]; };
    struct Right { i32x4 v[NBN]; };
    // All products of one group; `other(k)` goes out after product k.
    auto group = [&](const Left& l, const Right& r, auto other) __attribute__((always_inline)) {
        each<PRODUCTS>([&](auto k) __attribute__((always_inline)) {
            constexpr int j = k / NBM, i = k % NBM;
            acc[j][i] = mfma_f16_32x32x16(r.v[j], l.v[i], acc[j][i]);
            __builtin_amdgcn_sched_barrier(0);
            other(k);
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    // Those of `n` things that go out after product k, as evenly as they come.
    auto share = [](auto k, auto n, auto one) __attribute__((always_inline)) {
        each<n>([&](auto t) __attribute__((always_inline)) {
            if constexpr (t * PRODUCTS / n == k) one(t);
        });
    };
    auto read_both = [&](int lslot, int rslot, int q, Left& l, Right& r, auto t) __attribute__((always_inline)) {
        if constexpr (t < NBM) l.v[t] = read_left(lslot, q, t);
        else r.v[t - NBM] = read_right(rslot, q, t - NBM);
    };
    constexpr std::integral_constant<int, NBM + NBN> BOTH{};
    constexpr std::integral_constant<int, NBM> LEFTS{};
    constexpr std::integral_constant<int, NBN> RIGHTS{};
    constexpr int GROUPS = SPLIT ? 6 : 4;
    // The stage's reads are done: wait for the next one's loads (of the SLOTS - 4 operand stages after it some
    // may still be on their way) and hand its slots over.
    auto hand_over = [&]() __attribute__((always_inline)) {
        wait_lgkmcnt0();
        wait_vmcnt<(SLOTS - 4) * LOADS>();
        barrier_no_fence();
        __builtin_amdgcn_sched_barrier(0);
    };

#pragma unroll
    for (int n = 0; n < SLOTS - 2; ++n)
#pragma unroll
        for (int t = 0; t < LOADS; ++t) load_one(n, n, t);
    wait_vmcnt<(SLOTS - 4) * LOADS>();
    barrier_no_fence();
    asm volatile("" ::"s"(scale), "s"(linear));         // both are there: the loop's waits count LDS reads alone
    Left l0, l1;
    Right r0, r1;
    each<BOTH>([&](auto t) __attribute__((always_inline)) { read_both(0, 1, 0, l0, r0, t); });
    int lslot = 0, rslot = 1;                           // of this stage
    int freed = SLOTS - 2;                              // the two slots handed over last, the second one next to it
    for (int s = 0; s < stages; ++s) {
        const int lnext = lslot + 2 < SLOTS ? lslot + 2 : lslot + 2 - SLOTS;
        const int rnext = rslot + 2 < SLOTS ? rslot + 2 : rslot + 2 - SLOTS;
        const int freed1 = freed + 1 < SLOTS ? freed + 1 : 0;
        // Under group g: the loads of its share of the two freed slots ...
        auto loads = [&](auto g, auto k) __attribute__((always_inline)) {
            each<2 * LOADS>([&](auto t) __attribute__((always_inline)) {
                if constexpr (t * (GROUPS - 1) * PRODUCTS / (2 * LOADS) == g * PRODUCTS + k)
                    load_one(2 * s + SLOTS - 2 + t / LOADS, t / LOADS ? freed1 : freed, t % LOADS);
            });
        };
        // ... and the next group's fragments
        auto both = [&](auto g, int ls, int rs, int q, Left& l, Right& r) __attribute__((always_inline)) {
            return [&, g, ls, rs, q](auto k) __attribute__((always_inline)) {
                share(k, BOTH, [&](auto t) __attribute__((always_inline)) { read_both(ls, rs, q, l, r, t); });
                loads(g, k);
            };
        };
        constexpr std::integral_constant<int, 0> G0{};
        constexpr std::integral_constant<int, 1> G1{};
        constexpr std::integral_constant<int, 2> G2{};
        constexpr std::integral_constant<int, 3> G3{};
        constexpr std::integral_constant<int, 4> G4{};
        constexpr std::integral_constant<int, 5> G5{};
        if constexpr (KIND != kGram) fold(s, updates(KIND) ? rslot : lslot);
        if constexpr (!SPLIT) {
            group(l0, r0, both(G0, lslot, rslot, 1, l1, r1));
            group(l1, r1, both(G1, lslot, rslot, 2, l0, r0));
            group(l0, r0, both(G2, lslot, rslot, 3, l1, r1));
            hand_over();
            group(l1, r1, both(G3, lnext, rnext, 0, l0, r0));
        } else {
            Left low_l;
            Right low_r;
            auto rights = [&](auto g, int q) __attribute__((always_inline)) {
                return [&, g, q](auto k) __attribute__((always_inline)) {
                    share(k, RIGHTS, [&](auto t) __attribute__((always_inline)) { low_r.v[t] = read_right(rslot, q, t); });
                    loads(g, k);
                };
            };
            auto lefts = [&](auto g, int q) __attribute__((always_inline)) {
                return [&, g, q](auto k) __attribute__((always_inline)) {
                    share(k, LEFTS, [&](auto t) __attribute__((always_inline)) { low_l.v[t] = read_left(lslot, q, t); });
                    loads(g, k);
                };
            };
            group(l0, r0, rights(G0, 2));
            group(l0, low_r, lefts(G1, 2));
            group(low_l, r0, both(G2, lslot, rslot, 1, l1, r1));
            group(l1, r1, rights(G3, 3));
            group(l1, low_r, lefts(G4, 3));
            hand_over();
            group(low_l, r1, both(G5, lnext, rnext, 0, l0, r0));
        }
        freed = lslot;
        lslot = lnext;
        rslot = rnext;
    }
    wait_lgkmcnt0();
    wait_vmcnt<0>();
    barrier_no_fence();

    if constexpr (JOIN) {
        // the sums stay in one kind of registers: the compiler would otherwise move them to the other kind and back
        // in every stage, for the stores below
#pragma unroll
        for (int j = 0; j < NBN; ++j)
#pragma unroll
            for (int i = 0; i < NBM; ++i) asm volatile("" : "+v"(acc[j][i]));
        if (!join_parts<WAVES, NBM, NBN>(p, smem, tile, part, wave, lane, acc)) return;
    }

    // acc[j][i][4g + t] is the sum at row 32 i + l32 and column 32 j + 8 g + 4 lhi + t of the wave's
    // part.  It goes out through LDS, 32 rows at a time, so that every store writes whole runs of a row: once as it
    // is and, for a tile below the diagonal, once transposed.
    constexpr bool TWO = SPLIT || updates(KIND);      // both planes are kept
    constexpr bool LOW = !SPLIT && updates(KIND);     // the iterate's low plane was no operand: added here
    const int64_t lo_off = SPLIT ? 32 : (int64_t)p.batch * p.rows * p.cols;
    const int64_t matrix = (int64_t)b * p.rows * p.cols * (SPLIT ? 2 : 1);
    uint16_t* const out = (uint16_t*)p.out + matrix;
    const uint16_t* const low = (const uint16_t*)p.right + matrix + lo_off;
    const float low_scale = linear * scale;
    const int64_t row_w = m0 + wm * WTM, col_w = n0 + wn * WTN;
    lds_char* const mine = lds + wave * (SLOTS * STAGE / WAVES);
    static_assert(32 * (WTM > WTN ? WTM : WTN) * 4 <= SLOTS * STAGE / WAVES, "the image fits the wave's share of LDS");
    // the wave's own LDS accesses keep their order; this keeps the compiler from changing it
    auto in_order = [] { asm volatile("" ::: "memory"); };
    // Rows 32 i .. of the part as they are, or (turned) columns 32 j .. as rows.
    auto write_rows = [&](int i) __attribute__((always_inline)) {
        in_order();
#pragma unroll
        for (int j = 0; j < NBN; ++j)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const f32x4 v = {acc[j][i][4 * g], acc[j][i][4 * g + 1], acc[j][i][4 * g + 2], acc[j][i][4 * g + 3]};
                lds_store_16B(mine, image_at<WTN>(l32, 8 * j + 2 * g + lhi), __builtin_bit_cast(i32x4, v));
            }
        in_order();
    };
    auto write_turned = [&](int j) __attribute__((always_inline)) {
        in_order();
#pragma unroll
        for (int i = 0; i < NBM; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g)
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const uint32_t at = image_at<WTM>(8 * g + 4 * lhi + t, 8 * i + (l32 >> 2)) + (l32 & 3) * 4u;
                    *reinterpret_cast<__attribute__((address_space(3))) float*>(mine + at) = acc[j][i][4 * g + t];
                }
        in_order();
    };
    // Each lane's eight elements of the image's rows: store(r, n, v) with the row r of the first lane in store n.
    auto read_rows = [&](auto width, auto store) __attribute__((always_inline)) {
        constexpr int W = decltype(width)::value, LPR = W / 8, RPI = 64 / LPR;
        each<32 / RPI>([&](auto n) __attribute__((always_inline)) {
            const int r = n * RPI + lane / LPR, c = lane % LPR;
            const f32x4 u = __builtin_bit_cast(f32x4, lds_load_16B(mine, image_at<W>(r, 2 * c)));
            const f32x4 w = __builtin_bit_cast(f32x4, lds_load_16B(mine, image_at<W>(r, 2 * c + 1)));
            float v[8] = {u[0], u[1], u[2], u[3], w[0], w[1], w[2], w[3]};
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] *= scale;
            store(n * RPI, n, v);
        });
    };
    // Element (row0 + the lane's row, col0 + the lane's columns) of a stored matrix: a uniform base and the
    // lane's own 32-bit offset.
    const int64_t row_step = p.cols * (SPLIT ? 2 : 1);
    auto lane_row = [&](auto width) { return lane / (decltype(width)::value / 8); };
    auto lane_col = [&](auto width) { return 8 * (lane % (decltype(width)::value / 8)); };
    auto lane_at = [&](auto width) { return (uint32_t)element<SPLIT>(lane_row(width), lane_col(width), p.cols); };
    const std::integral_constant<int, WTN> across;
    const std::integral_constant<int, WTM> turned;
    auto result_at = [&](int64_t row0, int64_t col0, int row, int col, const float (&v)[8]) __attribute__((always_inline)) {
        if constexpr (!SPLIT) {
            store_result<kOutBf16>(p, v, b, row0, col0, row, col);
        } else {
            if (p.result_dtype == kOutF16) store_result<kOutF16>(p, v, b, row0, col0, row, col);
            else if (p.result_dtype == kOutBf16) store_result<kOutBf16>(p, v, b, row0, col0, row, col);
            else store_result<kOutF32>(p, v, b, row0, col0, row, col);
        }
    };

    if (KIND == kLast && p.tall) {
        // The last step of a matrix taken transposed: its result is the transpose.  The low plane comes through LDS:
        // read from memory as the sums lie, 8 bytes of 32 rows at a time, it made this launch take 2109 us
        // instead of 1921 (8 x 7168 x 4096 to bf16).
        if constexpr (LOW) {
            constexpr int CHUNKS = WTN / 8;             // 16-byte chunks of a row; chunk q in slot q ^ low_sw(row)
            auto low_sw = [](int row) { return (row >> 1) & (CHUNKS - 1); };
            static_assert(WTM * WTN * 2 <= SLOTS * STAGE / WAVES, "the part's low plane fits the wave's share of LDS");
#pragma unroll
            for (int t = 0; t < WTM * CHUNKS / 64; ++t) {
                const int at = t * 64 + lane, row = at / CHUNKS;
                const uint32_t off = (uint32_t)row * (uint32_t)(p.cols * 2) + (uint32_t)(((at % CHUNKS) ^ low_sw(row)) << 4);
                dma_16B(rsrc_words((const char*)(low + row_w * p.cols + col_w), 0xFFFFFFFFu), off,
                        lds0 + (uint32_t)(wave * (SLOTS * STAGE / WAVES) + t * 1024));
            }
            wait_vmcnt<0>();
            in_order();
#pragma unroll
            for (int i = 0; i < NBM; ++i)
#pragma unroll
                for (int j = 0; j < NBN; ++j)
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const i32x2 x = lds_load_8B(mine, (uint32_t)((32 * i + l32) * WTN * 2 +
                                                                     (((4 * j + g) ^ low_sw(l32)) << 4) + lhi * 8));
                        acc[j][i][4 * g] += linear * f16_lo((uint32_t)x[0]);
                        acc[j][i][4 * g + 1] += linear * f16_hi((uint32_t)x[0]);
                        acc[j][i][4 * g + 2] += linear * f16_lo((uint32_t)x[1]);
                        acc[j][i][4 * g + 3] += linear * f16_hi((uint32_t)x[1]);
                    }
        }
#pragma unroll
        for (int j = 0; j < NBN; ++j) {
            write_turned(j);
            read_rows(turned, [&](int r, int, const float (&v)[8]) __attribute__((always_inline)) {
                result_at(col_w + 32 * j + r, row_w, lane_row(turned), lane_col(turned), v);
            });
        }
        return;
    }
    constexpr int PIECES = WTN / 16;                    // of eight elements a lane in 32 rows
    const uint32_t at_across = lane_at(across), at_turned = lane_at(turned);
    i32x4 lows[2][PIECES];                              // 32 rows ahead of their use
    auto load_low = [&](auto i) __attribute__((always_inline)) {
        if constexpr (LOW)
            each<PIECES>([&](auto n) __attribute__((always_inline)) {
                const uint16_t* const from = low + (row_w + 32 * i + n * (512 / WTN)) * p.cols + col_w;
                lows[i & 1][n] = *(const gbl_i32x4*)(from + at_across);
            });
    };
    load_low(std::integral_constant<int, 0>{});
    each<NBM>([&](auto i) __attribute__((always_inline)) {
        if constexpr (i + 1 < NBM) load_low(std::integral_constant<int, i + 1>{});
        write_rows(i);
        read_rows(across, [&](int r, auto n, float (&v)[8]) __attribute__((always_inline)) {
            const int64_t row = row_w + 32 * i + r;
            if constexpr (LOW) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    v[2 * u] += low_scale * f16_lo((uint32_t)lows[i & 1][n][u]);
                    v[2 * u + 1] += low_scale * f16_hi((uint32_t)lows[i & 1][n][u]);
                }
            }
            if constexpr (KIND == kLast) result_at(row, col_w, lane_row(across), lane_col(across), v);
            else store_planes<TWO>(v, out + row * row_step + col_w * (SPLIT ? 2 : 1) + at_across, lo_off);
        });
    });
    if (!updates(KIND) && m0 != n0) {
        each<NBN>([&](auto j) __attribute__((always_inline)) {
            write_turned(j);
            read_rows(turned, [&](int r, int, const float (&v)[8]) __attribute__((always_inline)) {
                const int64_t row = col_w + 32 * j + r;
                store_planes<TWO>(v, out + row * row_step + row_w * (SPLIT ? 2 : 1) + at_turned, lo_off);
            });
        });
    }
}

// Quarter `index`: those of the tiles past p.whole, then the 128-wide strips at the ends of odd sizes (of every
// matrix in turn: down the right side, then along the bottom; along the bottom only for the symmetric products).
template <NewtonProduct KIND>
__device__ __forceinline__ void quarter_of(const NewtonGemm& p, int index, int& b, int64_t& m0, int64_t& n0) {
    const int cut = p.tiles - p.whole;
    if (index < 4 * cut) {
        int tm, tn;
        tile_of<KIND>(p, p.whole + (index >> 2), b, tm, tn);
        m0 = (int64_t)tm * 256 + (index & 1) * 128;
        n0 = (int64_t)tn * 256 + ((index >> 1) & 1) * 128;
        return;
    }
    const int per = p.strips;
    const int e = index - 4 * cut;
    b = e / per;
    int at = e - b * per;
    const int rows = (int)(p.rows / 128);
    const bool right = updates(KIND) && (p.cols & 128);
    if (right && at < rows) {
        m0 = (int64_t)at * 128;
        n0 = p.cols - 128;
    } else {
        if (right) at -= rows;
        m0 = p.rows - 128;
        n0 = (int64_t)at * 128;
    }
}

constexpr int kBigWaves = 8;

// 256 x 256 tiles; the items past p.whole are quarters of one.  Eight waves of 128 x 64: a wave's sums
// take half its registers and two waves a SIMD cover each other's waits (four waves of 128 x 128 need fewer LDS
// reads, but X X^T of 8 x 4096 x 7168 took 1184 us instead of 1046).  Now, one product: X X^T 904 us, A A 532,
// B X 1820 (1.06 PFLOP/s), the last one 1921 transposed and 1766 not; power bounds them (see the top).
template <bool SPLIT, NewtonProduct KIND>
__global__ __launch_bounds__(64 * kBigWaves, kBigWaves / 4) void newton_big_kernel(NewtonGemm p) {
    __shared__ __attribute__((aligned(1024))) char smem[5 * 256 * 128];
    const int bid = blockIdx.x;
    int b, tm, tn, turn;
    if (bid < p.whole) {
        tile_of<KIND>(p, item_of(bid, p.whole, p.num_xcds), b, tm, tn);
        turn = turn_of<SPLIT, KIND>(p, tm, 256);
        newton_tile<256, kBigWaves, 5, SPLIT, false, KIND>(p, smem, b, (int64_t)tm * 256, (int64_t)tn * 256, turn);
    } else {
        int64_t m0, n0;
        quarter_of<KIND>(p, bid - p.whole, b, m0, n0);
        if (!updates(KIND) && n0 > m0) return;         // the mirror image of another quarter
        turn = turn_of<SPLIT, KIND>(p, (int)(m0 / 256), 256);
        newton_tile<128, kBigWaves, 10, SPLIT, false, KIND>(p, smem, b, m0, n0, turn);
    }
}

// Small tiles: two workgroups a CU with SLOTS slots each (80 KiB), or one with twice as many.
// JOIN: p.parts of them share a tile's K.
// A 128-edged tile alone on its CU has eight waves, so that one multiplies while another waits for LDS:
// 8 x 512 x 2048 235 -> 227 us, 2 x 1024 x 4096 327 -> 318, 3 x 1777 x 1000 502 -> 497, 2048 x 2048 345 -> 349; two
// such tiles are as good with four each (27 x 1352 x 1072 1475 us, eight 1540).
template <int TILE, bool TWO>
constexpr int kSmallWaves = TILE == 128 && !TWO ? 8 : 4;
template <int TILE, bool TWO, bool JOIN, bool SPLIT, NewtonProduct KIND>
__global__ __launch_bounds__((64 * kSmallWaves<TILE, TWO>), 2) void newton_small_kernel(NewtonGemm p) {
    constexpr int SLOTS = (TWO ? 5 : 10) * (128 / TILE);
    __shared__ __attribute__((aligned(1024))) char smem[SLOTS * TILE * 128];
    const int item = item_of(blockIdx.x, p.items, p.num_xcds);
    const int tile = JOIN ? item / p.parts : item;
    int b, tm, tn;
    tile_of<KIND>(p, tile, b, tm, tn);
    newton_tile<TILE, kSmallWaves<TILE, TWO>, SLOTS, SPLIT, JOIN, KIND>(p, smem, b, (int64_t)tm * TILE, (int64_t)tn * TILE,
                                             turn_of<SPLIT, KIND>(p, tm, TILE), tile, JOIN ? item - tile * p.parts : 0);
}

template <int TILE, bool SPLIT, NewtonProduct KIND>
void launch_small(NewtonGemm g, int tiles, hipStream_t stream) {
    // Few tiles and a long K: workgroups share a tile's K.  Joining costs a 64-edged tile about as much a part as
    // two stages, so about sqrt(stages / 2) parts are best (1 x 200 x 7000: 418 -> 190 us); for a
    // 128-edged one it pays from 24 stages a part on (56 stages in two: 35 -> 29 us, 32 stages: 27 -> 30 us).
    const int64_t stages = g.k / (SPLIT ? 32 : 64);
    int64_t parts = 1;
    if (!updates(KIND)) {
        if (TILE == 64) while (stages > 16 && 2 * (parts + 1) * (parts + 1) <= stages) ++parts;
        else parts = stages / 24;
        if (parts > kNewtonSlabs / tiles) parts = kNewtonSlabs / tiles;
    }
    g.parts = parts > 1 ? (int32_t)parts : 1;
    g.items = tiles * g.parts;
    const dim3 grid((uint32_t)g.items);
    constexpr uint32_t alone = 64 * kSmallWaves<TILE, false>, paired = 64 * kSmallWaves<TILE, true>;
    if constexpr (!updates(KIND)) {
        if (g.parts > 1) {
            hipLaunchKernelGGL((newton_small_kernel<TILE, false, true, SPLIT, KIND>), grid, dim3(alone), 0,
                           stream, g);
            return;
        }
    }
    if (g.items > kNewtonSlabs)
        hipLaunchKernelGGL((newton_small_kernel<TILE, true, false, SPLIT, KIND>), grid, dim3(paired), 0,
                           stream, g);
    else
        hipLaunchKernelGGL((newton_small_kernel<TILE, false, false, SPLIT, KIND>), grid, dim3(alone), 0,
                           stream, g);
}

// Time of what follows the whole rounds of 256 x 256 tiles, in tiles' times: `rest` tiles and `edges` quarters of
// the strips.  A quarter takes 0.36 of a tile's time.  Either the rest stays whole, with quarters on the
// CUs it leaves, or it is taken in quarters too.
double rest_kept(int64_t rest, int64_t edges, int64_t cus) {
    const double beside = rest ? (double)(cus - rest) / 0.36 : 0.0;
    const double more = (double)edges > beside ? ((double)edges - beside) / (double)cus : 0.0;
    return (rest ? 1.0 : 0.0) + 0.36 * (double)(int64_t)(more + 0.999);
}
double rest_in_quarters(int64_t rest, int64_t edges, int64_t cus) { return 0.36 * (double)((4 * rest + edges + cus - 1) / cus); }

// Estimated time of one step with tiles of 256 or 128, in K values of one 256 x 256 tile.  Two 128 x 128
// tiles on a CU take 0.55 of its time, one alone 0.36.  The model puts 8 x 4096 x 2048 9% behind with 128
// (measured: 10%), 16 x 700 x 2000 16% ahead (20%), 27 x 1352 x 1072 7% ahead (10%).
double step_cost(int64_t batch, int64_t r, int64_t c, int tile) {
    constexpr int64_t cus = 256;
    const int64_t R = (r + 127) / 128, C = (c + 127) / 128;
    auto cost = [&](int64_t big, int64_t edges, int64_t small) {
        if (tile == 256) {
            const int64_t rest = big % cus;
            const double kept = rest_kept(rest, edges, cus), cut = rest_in_quarters(rest, edges, cus);
            return (double)(big / cus) + (cut < kept ? cut : kept);
        }
        const int64_t rest = small % (2 * cus);
        return 0.55 * (double)(small / (2 * cus)) + (rest > cus ? 0.55 : rest ? 0.36 : 0.0);
    };
    const int64_t r2 = R / 2, c2 = C / 2;
    const double square = cost(batch * r2 * (r2 + 1) / 2, R % 2 ? batch * R : 0, batch * R * (R + 1) / 2);
    const int64_t right = C % 2 ? R : 0;
    const double update = cost(batch * r2 * c2, batch * (right + (R % 2 ? C - (right ? 1 : 0) : 0)), batch * R * C);
    return square * (double)(c + r) + update * (double)r;
}

template <bool SPLIT, NewtonProduct KIND>
void launch_product(NewtonGemm g, int tile, int num_cus, hipStream_t stream) {
    g.tiles_m = (int32_t)(g.rows / tile);
    g.tiles_n = (int32_t)(g.cols / tile);
    const int tiles = g.batch * (updates(KIND) ? g.tiles_m * g.tiles_n : g.tiles_m * (g.tiles_m + 1) / 2);
    g.parts = 1;
    if (tile == 256) {
        const int rows = (int)(g.rows / 128), cols = (int)(g.cols / 128);
        const int right = updates(KIND) && cols % 2 ? rows : 0;
        g.strips = right + (rows % 2 ? cols - (right ? 1 : 0) : 0);
        g.tiles = tiles;
        const int rest = tiles % num_cus, edges = g.batch * g.strips;
        g.whole = rest_in_quarters(rest, edges, num_cus) < rest_kept(rest, edges, num_cus) ? tiles - rest : tiles;
        g.items = g.whole + 4 * (tiles - g.whole) + edges;
        hipLaunchKernelGGL((newton_big_kernel<SPLIT, KIND>), dim3((uint32_t)g.items), dim3(64 * kBigWaves), 0,
                           stream, g);
    } else {
        if (tile == 128) launch_small<128, SPLIT, KIND>(g, tiles, stream);
        else launch_small<64, SPLIT, KIND>(g, tiles, stream);
    }
}

template <bool SPLIT>
void launch_steps(const NewtonParams& p, const NewtonPlan& plan, const NewtonCoefficients& co, int num_cus, int num_xcds,
                  hipStream_t stream) {
    NewtonGemm g = {};
    g.batch = p.batch;
    g.slabs = p.slabs;
    g.arrived = p.arrived;
    g.num_xcds = num_xcds;
    g.rows = plan.r;
    g.m = p.m;
    g.n = p.n;
    g.result_dtype = p.out_dtype;
    g.tall = plan.tall ? 1 : 0;
    for (int s = 0; s < p.steps; ++s) {
        const char* const x = p.x[s & 1];
        g.scales = p.scales + s;
        g.cols = plan.r;
        g.k = plan.c;
        g.left = g.right = x;
        g.out = p.a;
        launch_product<SPLIT, kGram>(g, plan.tile, num_cus, stream);
        if (co.measured) {
            const int64_t share = (plan.r * plan.r + 8191) / 8192;
            const int32_t parts = (int32_t)(share < kNewtonParts ? share : kNewtonParts);
            hipLaunchKernelGGL((newton_measure_kernel<SPLIT>), dim3((uint32_t)parts, (uint32_t)p.batch), dim3(NT), 0, stream, p,
                               plan.r, parts);
            hipLaunchKernelGGL(newton_scales_kernel, dim3((uint32_t)p.batch), dim3(64), 0, stream, p, co, s, parts);
        }
        g.k = plan.r;
        g.left = g.right = p.a;
        g.out = p.b;
        launch_product<SPLIT, kSquare>(g, plan.tile, num_cus, stream);
        g.cols = plan.c;
        g.left = p.b;
        g.right = x;
        g.out = p.x[(s + 1) & 1];
        g.result = p.out;
        if (s + 1 == p.steps) launch_product<SPLIT, kLast>(g, plan.tile, num_cus, stream);
        else launch_product<SPLIT, kUpdate>(g, plan.tile, num_cus, stream);
    }
}

template <bool SPLIT, bool TALL>
void launch_all(const NewtonParams& p, const NewtonPlan& plan, const NewtonCoefficients& co, int num_cus, int num_xcds,
                hipStream_t stream) {
    launch_newton_norm(p, stream);
    const dim3 tiles((uint32_t)(plan.c / 64), (uint32_t)(plan.r / 64), (uint32_t)p.batch);
    auto first = [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        hipLaunchKernelGGL((newton_first_kernel<DT, SPLIT, TALL>), tiles, dim3(NT), 0, stream, p, co, plan.r, plan.c);
    };
    if (p.dtype == kOutBf16) first(std::integral_constant<int, kOutBf16>{});
    else if (p.dtype == kOutF16) first(std::integral_constant<int, kOutF16>{});
    else first(std::integral_constant<int, kOutF32>{});
    launch_steps<SPLIT>(p, plan, co, num_cus, num_xcds, stream);
}

}  // namespace

void launch_newton_norm(const NewtonParams& p, hipStream_t stream) {
    const dim3 grid((uint32_t)p.num_parts, (uint32_t)p.batch);
    if (p.dtype == kOutBf16) hipLaunchKernelGGL((newton_norm_kernel<kOutBf16>), grid, dim3(NT), 0, stream, p);
    else if (p.dtype == kOutF16) hipLaunchKernelGGL((newton_norm_kernel<kOutF16>), grid, dim3(NT), 0, stream, p);
    else hipLaunchKernelGGL((newton_norm_kernel<kOutF32>), grid, dim3(NT), 0, stream, p);
}

NewtonPlan newton_plan(int32_t batch, int64_t m, int64_t n, bool split) {
    NewtonPlan plan = {};
    const int64_t r = m < n ? m : n, c = m < n ? n : m;
    plan.tall = m > n;
    plan.parts_bytes = ((size_t)batch * kNewtonParts * sizeof(double) + 1023) / 1024 * 1024;
    plan.scales_bytes = (size_t)batch * (kNewtonMaxSteps * sizeof(StepScales) + 2 * sizeof(int32_t));
    plan.narrow = r <= kNarrowMax;
    if (plan.narrow) {
        newton_narrow_plan(batch, r, c, &plan);
        return plan;
    }
    plan.split = split;
    // 64-edged tiles while 128-edged ones would leave a quarter of the CUs idle in the update (their number: 2 x 1024 x
    // 1024, 128 of them: 171 against 194 us; 3 x 900 x 900 to fp32, 192: 340 against 364; 1700 x 1700, 196:
    // 286 against 283, to fp32 537 against 513); above, what step_cost() puts lower of 256 and 128.
    auto tiles = [&](int64_t edge) { return ((r + edge - 1) / edge) * ((c + edge - 1) / edge) * batch; };
    plan.tile = tiles(128) <= 192 ? 64 : r >= 256 && step_cost(batch, r, c, 256) < step_cost(batch, r, c, 128) ? 256 : 128;
    const int64_t edge = plan.tile == 64 ? 64 : 128;    // an odd half tile at an end is taken in quarters
    plan.r = (r + edge - 1) / edge * edge;
    plan.c = (c + edge - 1) / edge * edge;
    plan.x_bytes = (size_t)batch * plan.r * plan.c * 4;
    plan.a_bytes = (size_t)batch * plan.r * plan.r * (plan.split ? 4 : 2);
    plan.b_bytes = plan.a_bytes;
    // sums of parts of K (kNewtonSlabs of them at most, one a workgroup) and their counters
    plan.slab_bytes = plan.tile == 256 ? 0 : (size_t)kNewtonSlabs * (plan.tile * plan.tile * 4 + 4);
    plan.total = plan.parts_bytes + 2 * plan.x_bytes + plan.a_bytes + plan.b_bytes + plan.slab_bytes + plan.scales_bytes;
    return plan;
}

hipError_t launch_newton(const NewtonParams& p, const NewtonPlan& plan, const float* coefficients, int num_cus,
                         int num_xcds, hipStream_t stream) {
    NewtonCoefficients co = {};
    for (int i = 0; i < 3 * p.steps; ++i) co.v[i] = coefficients[i];
    const float ratio = 1.0f / __builtin_sqrtf((float)(p.m < p.n ? p.m : p.n));
    SingularBound bound = unit_bound(ratio);
    for (int s = 0; s < p.steps; ++s) {
        if (!(bound.ratio >= ratio * kBoundLoss)) co.measured = 1;
        co.unit[s] = step_scales(bound, co.v + 3 * s, s + 1 == p.steps);
    }
    if (plan.narrow) {
        launch_newton_narrow(p, plan, co, stream);
    } else if (plan.split) {
        if (plan.tall) launch_all<true, true>(p, plan, co, num_cus, num_xcds, stream);
        else launch_all<true, false>(p, plan, co, num_cus, num_xcds, stream);
    } else {
        if (plan.tall) launch_all<false, true>(p, plan, co, num_cus, num_xcds, stream);
        else launch_all<false, false>(p, plan, co, num_cus, num_xcds, stream);
    }
    return hipGetLastError();
}

}  // namespace kgw
