// Weight gradients from 8-bit token rows (gfx950): out[e] (=|+=) A[begin:end, :]^T B[begin:end, :] over the rows of expert e,
// A e4m3 with one power of two for every 128 values of a row, B the same or bf16.
//
// The scale of an A value changes with the token, along the contracted axis, so neither a scaled MFMA nor a conversion of whole
// fragments can take it.  Each value becomes bf16 with its scale folded in -- exactly: e4m3 times a power of two -- on its
// way into LDS, once for a tile, and the bf16 MFMA (32x32x16, fp32 sums) does the rest.
//
// One workgroup of four waves has an output tile of (64 FM) x (64 FN), each wave a quarter of it, computed transposed
// (a lane ends up holding four consecutive N values of one output row).  A K step is 32 tokens.  Global memory comes in
// through registers, 8 values a lane and load, three steps ahead; wave w takes token rows 8w .. 8w+7 of every step.  In step s:
//   first half    MFMAs of the step's first 16 tokens, the fragment reads of its last 16, and the conversion of step
//                 s+2's values into LDS (a ring of three steps, rows of tokens as bf16);
//   second half   MFMAs of the last 16 tokens, the fragment reads of step s+1's first 16, and the loads of step s+5
//                 into the registers that the conversion has freed.
// One barrier a step publishes step s+1 and frees the slot of step s-1.  Fragments come by transposing reads
// (ds_read_b64_tr_b16); 16-byte chunk q of token row k lies at q ^ swizzle(k), so that the four rows of a read lie in
// different banks.  Loads of steps past an expert's range go to an empty buffer range (zeros, no traffic).
//
// The matrix cores bound the large tile: 32 experts of 7168 x 4096, 264320 tokens, B in 8 bits, bf16 results, 11.7 ms (1.32
// PFLOP/s, of the 1.37 that a library bf16 product of 8192^3 reaches on this card), cores busy 64% at 1.97 GHz, no LDS bank
// conflicts; 8 experts of 4096 x 2048, 32768 tokens, B bf16, 441 us (1.25).  With fp32 results the large tile's loop does not
// fit its registers (12 spilled for B in 8 bits, 32 for bf16): 8 experts 454 and 478 us, the 32 experts with 262144 tokens 12.3 and
// 13.1 ms (bf16 results: 12.0 and 12.0).  Staging through registers and LDS is for the conversion, once for a
// value and tile; direct loads with the conversion from LDS to LDS before took 12.7 ms.  The small tiles are bound by a
// step's length and the rounds of compute units: 5 experts of 1040 x 776, 5760 tokens, 24 us (315 tiles of 128; a wave issues in
// 45% of its cycles, waits in 32% for data or the others, in 23% for its turn, and has the matrix core for 21%).
#include <type_traits>

#include "kgw_device.h"
#include "kgw_internal.h"
#include "kgw_schedule.h"
#include "kgw_tile_io.h"

namespace kgw {
namespace {

constexpr int NT = 256;
constexpr int BK = 32;
constexpr int SLOTS = 3, SETS = 3;

// The same value in scalar registers (of a value that all lanes agree on).
__device__ __forceinline__ int64_t scalar(int64_t v) {
    return (int64_t)(((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32) |
                     (uint32_t)__builtin_amdgcn_readfirstlane((int)v));
}

// One operand's way into LDS for a tile of T columns: rows of T values, T / 8 lanes a row.
template <int T, bool EIGHT>
struct Staging {
    static constexpr int PER = T / 8;                       // lanes of a row
    static constexpr int ROWS = 64 / PER;                   // token rows of a load
    static constexpr int LOADS = 8 / ROWS;                  // of a wave's 8 rows
    static constexpr int ITEMS = LOADS + (EIGHT ? 1 : 0);   // with the scales
    static constexpr int STAGE = BK * T * 2;
    struct Raw {
        i32x4 wide[EIGHT ? 1 : LOADS];
        i32x2 codes[EIGHT ? LOADS : 1];
        i32x2 scales;                                       // of the wave's 8 tokens, for the lane's columns
    };
    uint32_t voff, row_step, sc_voff;
    const char* base;                                       // the tile's columns at the range's first token
    const uint8_t* scales;
    int64_t step_bytes;

    __device__ static constexpr int swizzle(int k) { return T == 64 ? 4 * ((k >> 1) & 1) : 4 * (k & 3); }

    // stride: columns of the whole operand; c0: the tile's first; valid: its columns that exist (a multiple of 8).
    __device__ __forceinline__ void init(const void* src, const uint8_t* sc, int64_t stride, int64_t tokens, int64_t begin,
                                         int64_t c0, int valid, int wave, int lane) {
        constexpr int SIZE = EIGHT ? 1 : 2;
        const int q = lane & (PER - 1);
        base = (const char*)scalar((int64_t)src + (begin * stride + c0) * SIZE);
        // lanes past the last column read the last ones again; they only feed outputs that are never stored
        voff = (uint32_t)(8 * wave + lane / PER) * (uint32_t)(stride * SIZE) + (uint32_t)(min(8 * q, valid - 8) * SIZE);
        row_step = (uint32_t)(ROWS * stride * SIZE);
        step_bytes = scalar(BK * stride * SIZE);
        if constexpr (EIGHT) {
            scales = (const uint8_t*)scalar((int64_t)sc + (c0 >> 7) * tokens + begin);
            sc_voff = (uint32_t)(min(8 * q, valid - 8) >> 7) * (uint32_t)tokens + (uint32_t)(8 * wave);
            // (c0 is a multiple of 64: a tile of 64 columns lies in one block, and the shift above counts from c0's block)
        }
    }
    // Load i of step x: rows of codes or values, the last one the scales.
    __device__ __forceinline__ void load(int x, int i, bool live, Raw& r) const {
        const uint32_t bytes = (uint32_t)__builtin_amdgcn_readfirstlane(live ? -1 : 0);
        if (i < LOADS) {
            const __amdgpu_buffer_rsrc_t s = make_rsrc((const void*)scalar((int64_t)base + x * step_bytes), bytes);
            const int at = (int)(voff + (uint32_t)i * row_step);
            if constexpr (EIGHT) r.codes[i] = __builtin_amdgcn_raw_buffer_load_b64(s, at, 0, 0);
            else r.wide[i] = __builtin_amdgcn_raw_buffer_load_b128(s, at, 0, 0);
        } else {
            r.scales = __builtin_amdgcn_raw_buffer_load_b64(make_rsrc((const void*)scalar((int64_t)scales + x * BK), bytes), (int)sc_voff, 0, 0);
        }
    }
    // Writes load i's rows to the stage at `to` as bf16.
    __device__ __forceinline__ void store(lds_char* to, int i, int wave, int lane, const Raw& r) const {
        const int q = lane & (PER - 1), in = i * ROWS + lane / PER, k = 8 * wave + in;
        i32x4 v;
        if constexpr (EIGHT) {
            const uint32_t word = (uint32_t)(in < 4 ? r.scales[0] : r.scales[1]);
            v = cvt_e4m3x8_bf16(r.codes[i], e8m0_scale_operand(__builtin_amdgcn_ubfe(word, (uint32_t)(8 * (in & 3)), 8)));
        } else {
            v = r.wide[i];
        }
        lds_store_16B(to, (uint32_t)(k * T * 2 + ((q ^ swizzle(k)) << 4)), v);
    }
};

// Fragments of one operand, `N` blocks of 32 columns by 16 tokens: two transposed halves of 4-token groups each.
template <int N>
struct Frag {
    i16x4 lo[N], hi[N];
};
template <int T, int N>
struct FragReader {
    uint32_t at[N];
    __device__ __forceinline__ void init(int half, int lane) {
        const int g16 = lane >> 4, i16 = lane & 15;
        const int k = 8 * (g16 >> 1) + (i16 >> 2);          // + 4 in the upper half: the same swizzle for T = 64 and others
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int q = 4 * (half * N + j) + 2 * (g16 & 1) + ((i16 & 3) >> 1);
            at[j] = (uint32_t)(k * T * 2 + ((q ^ Staging<T, false>::swizzle(k)) << 4) + (i16 & 1) * 8);
        }
    }
    // Block j, half h (0 lo, 1 hi) of the 16 tokens `ks` of a stage.
    __device__ __forceinline__ void read(const lds_char* stage, int ks, int j, int h, Frag<N>& f) const {
        const i16x4 v = lds_read_tr16(stage, at[j] + (uint32_t)((16 * ks + 4 * h) * T * 2));
        if (h) f.hi[j] = v;
        else f.lo[j] = v;
    }
};
__device__ __forceinline__ i32x4 join(i16x4 lo, i16x4 hi) {
    const i16x8 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    return __builtin_bit_cast(i32x4, v);
}

// A wave's (32 FM) x (32 FN) part of a small tile, through `stage` (4 KiB FN of LDS of its own), 32 rows at a time, with
// the layout of store_wave_tile_staged: acc[j][i][4g + t] is row 32i + (lane & 31), column 32j + 8g + 4 (lane >> 5) + t.
// All of the wave's LDS accesses are complete at the end, also where nothing is stored.
template <int OUT, int FM, int FN>
__device__ __forceinline__ void store_small_tile(const GroupedParams& p, int e, int64_t mb, int64_t nb, int lane,
                                                 const f32x16 (&acc)[FN][FM], lds_char* stage) {
    constexpr int ESIZE = OUT == kOutF32 ? 4 : 2, COLS = 16 / ESIZE;      // columns of a lane's 16 bytes
    constexpr int PER = 32 * FN / COLS, ROWS = 64 / PER, CHUNKS = 8 * FN; // lanes of a row; rows of a store; chunks of a row
    gbl_char* const obase = (gbl_char*)expert_output<OUT>(p, e);
    const int l32 = lane & 31, lhi = lane >> 5, col = lane & (PER - 1);
    const int64_t n = nb + COLS * col;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int c = 8 * j + 2 * g + lhi;
                const f32x4 w = {acc[j][i][4 * g], acc[j][i][4 * g + 1], acc[j][i][4 * g + 2], acc[j][i][4 * g + 3]};
                lds_store_16B(stage, (uint32_t)(l32 * CHUNKS * 16 + ((c ^ (l32 & (CHUNKS - 1))) << 4)), __builtin_bit_cast(i32x4, w));
            }
#pragma unroll
        for (int u = 0; u < 32 / ROWS; ++u) {
            const int r = u * ROWS + lane / PER;
            const int64_t m = mb + 32 * i + r;
            float v[COLS];
#pragma unroll
            for (int h = 0; h < COLS / 4; ++h) {
                const f32x4 w = __builtin_bit_cast(f32x4, lds_load_16B(stage, (uint32_t)(r * CHUNKS * 16 + (((COLS / 4 * col + h) ^ (r & (CHUNKS - 1))) << 4))));
#pragma unroll
                for (int t = 0; t < 4; ++t) v[4 * h + t] = w[t];
            }
            if (m >= p.hidden || n >= p.n) continue;        // n is a multiple of 8: whole pieces
            gbl_i32x4* const to = (gbl_i32x4*)(obase + (m * p.n + n) * ESIZE);
            if (p.accumulate) {
                const i32x4 old = __builtin_nontemporal_load(to);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    if constexpr (OUT == kOutF32) {
                        v[t] += __builtin_bit_cast(f32x4, old)[t];
                    } else {
                        v[2 * t] += half_lo<OUT>((uint32_t)old[t]);
                        v[2 * t + 1] += half_hi<OUT>((uint32_t)old[t]);
                    }
                }
            }
            i32x4 out;
            if constexpr (OUT == kOutF32) {
                const f32x4 w = {v[0], v[1], v[2], v[3]};
                out = __builtin_bit_cast(i32x4, w);
            } else {
                out = i32x4{(int)pack_half2<OUT>(v[0], v[1]), (int)pack_half2<OUT>(v[2], v[3]),
                            (int)pack_half2<OUT>(v[4], v[5]), (int)pack_half2<OUT>(v[6], v[7])};
            }
            __builtin_nontemporal_store(out, to);
        }
    }
    asm volatile("" ::: "memory");
    wait_lgkmcnt0();
}

template <int F>
constexpr int kGroups = F == 4 ? 1 : F == 2 ? 2 : 4;       // workgroups that share a CU

template <int OUT, int F, bool B8>
__global__ __launch_bounds__(NT, kGroups<F>) void wgrad_rows8_kernel(GroupedParams p) {
    constexpr int T = 64 * F;                               // the tile's edge
    using StageA = Staging<T, true>;
    using StageB = Staging<T, B8>;
    constexpr int STAGE = StageA::STAGE;
    constexpr int RING = 2 * SLOTS * STAGE;                 // A's ring, then B's
    constexpr int OUTPUT = F == 4 ? 4 * 32768 : 4 * 4096 * F;
    constexpr int BLOCKS = F * F;                           // MFMAs of half a step
    __shared__ __attribute__((aligned(1024))) char smem[RING > OUTPUT ? RING : OUTPUT];
    lds_char* tiles = (lds_char*)smem;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave & 1, wn = wave >> 1;
    const int64_t H = p.hidden, N = p.n;
    FragReader<T, F> reader_a, reader_b;
    reader_a.init(wm, lane);
    reader_b.init(wn, lane);
    const int TT = p.tiles_m * p.tiles_n;
    Schedule sched(p, tiles, tid);
    for (int item = sched.next(); item >= 0; item = sched.next()) {
        const int ec = item / TT;
        const int local = item - ec * TT;
        const int e = sched.expert(ec);
        const int c = ec - (sched.dyn ? ec : e * p.split);
        const int eo = c * p.num_experts + e;
        if (p.out_ptrs && !p.out_ptrs[eo]) {
            sched.claim_next();
            continue;
        }
        int tm, tn;
        tile_coords(local, p.tiles_m, p.tiles_n, p.group_m, tm, tn);
        const int64_t m0 = (int64_t)tm * T, n0 = (int64_t)tn * T;
        const TokenRange range = token_range(p, e, c);
        const int32_t begin = range.begin & ~(2 * BK - 1);  // whole 64-token units
        const int ksteps = __builtin_amdgcn_readfirstlane(((range.end - begin) / (2 * BK)) * 2);
        if (ksteps <= 0) {
            sched.claim_next();
            if (!p.accumulate) zero_slab_part<OUT, NT>(p, eo, local, TT, tid);
            continue;
        }
        StageA sa;
        StageB sb;
        sa.init(p.A, p.sfa, H, p.tokens_sum, begin, m0, (int)min<int64_t>(T, H - m0), wave, lane);
        sb.init(p.B, p.sfb, N, p.tokens_sum, begin, n0, (int)min<int64_t>(T, N - n0), wave, lane);

        f32x16 acc[F][F];
#pragma unroll
        for (int j = 0; j < F; ++j)
#pragma unroll
            for (int i = 0; i < F; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[j][i][r] = 0.0f;
        typename StageA::Raw ra[SETS];
        typename StageB::Raw rb[SETS];
        constexpr int LOADS = StageA::ITEMS + StageB::ITEMS, STORES = StageA::LOADS + StageB::LOADS;
        // in order: each operand's scales before its codes are needed, so first
        auto load_item = [&](int set, int x, int i) __attribute__((always_inline)) {
            if (i < StageA::ITEMS) sa.load(x, StageA::ITEMS - 1 - i, x < ksteps, ra[set]);
            else sb.load(x, StageB::ITEMS - 1 - (i - StageA::ITEMS), x < ksteps, rb[set]);
        };
        auto store_item = [&](int set, int slot, int i) __attribute__((always_inline)) {
            if (i < StageA::LOADS) sa.store(tiles + slot * STAGE, StageA::LOADS - 1 - i, wave, lane, ra[set]);
            else sb.store(tiles + (SLOTS + slot) * STAGE, StageB::LOADS - 1 - (i - StageA::LOADS), wave, lane, rb[set]);
        };
        Frag<F> fa[2], fb[2];                               // of the step's first and last 16 tokens
        // read i of 4 F, two of a block, in the order in which the MFMAs need the blocks: A 0, B 0, the rest of A, of B
        auto read_item = [&](int slot, int ks, int i) __attribute__((always_inline)) {
            const int block = i >> 1, h = i & 1;
            if (block == 1 || block > F) reader_b.read(tiles + (SLOTS + slot) * STAGE, ks, block == 1 ? 0 : block - F, h, fb[ks]);
            else reader_a.read(tiles + slot * STAGE, ks, block == 0 ? 0 : block - 1, h, fa[ks]);
        };
#pragma unroll
        for (int x = 0; x < SETS; ++x)
#pragma unroll
            for (int i = 0; i < LOADS; ++i) load_item(x, x, i);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int i = 0; i < STORES; ++i) store_item(x, x, i);
#pragma unroll
            for (int i = 0; i < LOADS; ++i) load_item(x, x + SETS, i);
        }
        asm volatile("" ::: "memory");
        wait_lgkmcnt0();
        barrier_no_fence();
#pragma unroll
        for (int i = 0; i < 4 * F; ++i) read_item(0, 0, i);

        // Step s, R = s mod 3 (slots and register sets are constants).
        auto half = [&](auto rc, int s, auto last) __attribute__((always_inline)) {
            constexpr int R = decltype(rc)::value, SET = (R + 2) % 3;
            constexpr bool LAST = decltype(last)::value;
            constexpr int READS = 4 * F, WORK = LAST ? LOADS : STORES;
#pragma unroll
            for (int k = 0; k < BLOCKS; ++k) {
                // Reads: one an MFMA in the large tile, whose waves have their SIMDs alone; ahead of the last MFMAs in the
                // smaller ones, where an MFMA that waits costs more (2048 x 2048 x 2048: 24.0 us, spread evenly 26.0).
                constexpr int FIRST = F == 2 ? BLOCKS / 2 : BLOCKS;
                if (k < FIRST) {
#pragma unroll
                    for (int i = k * READS / FIRST; i < (k + 1) * READS / FIRST; ++i)
                        read_item(LAST ? (R + 1) % 3 : R, LAST ? 0 : 1, i);
                }
                acc[k / F][k % F] = mfma_bf16_32x32x16(join(fb[LAST].lo[k / F], fb[LAST].hi[k / F]),
                                                       join(fa[LAST].lo[k % F], fa[LAST].hi[k % F]), acc[k / F][k % F]);
#pragma unroll
                for (int i = k * WORK / BLOCKS; i < (k + 1) * WORK / BLOCKS; ++i) {
                    if constexpr (LAST) load_item(SET, s + 5, i);
                    else store_item(SET, SET, i);
                }
                if constexpr (BLOCKS > 1) __builtin_amdgcn_sched_barrier(0);
            }
        };
        auto body = [&](auto rc, int s) __attribute__((always_inline)) {
            // Step s+1's values are written and step s-1's slot is read: LDS works in order, and only step s's first
            // fragments were asked for after that.
            asm volatile("" ::: "memory");
            wait_lgkmcnt<(4 * F < 15 ? 4 * F : 15)>();
            barrier_no_fence();
            half(rc, s, std::false_type{});
            half(rc, s, std::true_type{});
        };
        int s = 0;
        for (; s + 3 <= ksteps; s += 3) {
            body(std::integral_constant<int, 0>{}, s);
            body(std::integral_constant<int, 1>{}, s + 1);
            body(std::integral_constant<int, 2>{}, s + 2);
        }
        if (s < ksteps) {
            body(std::integral_constant<int, 0>{}, s);
            if (s + 1 < ksteps) body(std::integral_constant<int, 1>{}, s + 1);
        }
        wait_lgkmcnt0();
        barrier_no_fence();
        sched.claim_next();
        if constexpr (F == 4)
            store_wave_tile_staged<OUT>(p, eo, m0 + wm * 128, n0 + wn * 128, lane, acc, tiles + wave * 32768);
        else
            store_small_tile<OUT, F, F>(p, eo, m0 + wm * 32 * F, n0 + wn * 32 * F, lane, acc, tiles + wave * (4096 * F));
        barrier_no_fence();
    }
}

template <int F, bool B8>
void launch_tile(const GroupedParams& p, int out_kind, int grid, hipStream_t stream) {
    if (out_kind == kOutBf16) hipLaunchKernelGGL((wgrad_rows8_kernel<kOutBf16, F, B8>), dim3(grid), dim3(NT), 0, stream, p);
    else if (out_kind == kOutF16) hipLaunchKernelGGL((wgrad_rows8_kernel<kOutF16, F, B8>), dim3(grid), dim3(NT), 0, stream, p);
    else hipLaunchKernelGGL((wgrad_rows8_kernel<kOutF32, F, B8>), dim3(grid), dim3(NT), 0, stream, p);
}

}  // namespace

hipError_t launch_wgrad_fp8_rows(const GroupedParams& p, int out_kind, int tile, int grid, hipStream_t stream) {
    if (tile == 256) p.sfb ? launch_tile<4, true>(p, out_kind, grid, stream) : launch_tile<4, false>(p, out_kind, grid, stream);
    else if (tile == 128) p.sfb ? launch_tile<2, true>(p, out_kind, grid, stream) : launch_tile<2, false>(p, out_kind, grid, stream);
    else p.sfb ? launch_tile<1, true>(p, out_kind, grid, stream) : launch_tile<1, false>(p, out_kind, grid, stream);
    return hipGetLastError();
}

}  // namespace kgw
