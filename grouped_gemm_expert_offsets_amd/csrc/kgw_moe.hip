// Tokens sorted by expert and brought back (gfx950): the routing step around the grouped
// products, which take rows grouped by expert with every group padded to a multiple of
// 128 or 256 rows.
//
//   sort            ids (T, k) -> per-expert counts, inclusive aligned offsets, the row of
//                   every assignment and the assignment of every row (a stable counting sort)
//   permute         out[row_of[t][j]] = x[t], every other row zero
//   unpermute       out[t] = sum_j w[t][j] * y[row_of[t][j]]
//   unpermute grad  dy[row_of[t][j]] = w[t][j] * dout[t], every other row zero;
//                   dw[t][j] = <dout[t], y[row_of[t][j]]>
//
// permute and the gradient walk the tokens, not the rows: a token's row is read once and
// written (or used) k times, so the reads are T rows and not T * k.  Rows move in 16-byte
// pieces at element alignment (gfx950 takes 16-byte global accesses at any element-aligned
// address), so odd row lengths and unaligned views need no path of their own; the last
// H % (16 / element size) elements of a row move one by one.  Sums are fp32, in the order of
// j (unpermute) or a fixed tree over the row (dw), so results do not depend on scheduling.
//
// The row kernels are bound by HBM.  On this card a large copy moves 4.9 TB/s and a fill 6.9;
// 32768 x 8 tokens, 7168 bf16:
//   permute          4.29 GB  786 us  5.4 TB/s (7/8 of it writes)
//   unpermute        4.23 GB  739 us  5.7 TB/s
//   unpermute grad   8.05 GB 1560 us  5.1 TB/s
// Small ones are bound by the launch: 4099 x 6 tokens of 1001 fp32 take 8.1 us, their 41 MB from the
// Infinity Cache.
#include <type_traits>

#include "kgw_device.h"
#include "kgw_layer.h"

namespace kgw {
namespace {

// ----------------------------------------------------------------------------
// sort
// ----------------------------------------------------------------------------
constexpr int SORT_NT = 1024;
constexpr int SORT_WAVES = SORT_NT / 64;
// Assignments a lane that one workgroup ranks at a time.  Up to 2048 assignments one workgroup does it all (2048 to 256
// experts: 7.1 us, two launches 7.7; 4096 in two rounds 10.4, two launches 7.6).  Beyond, one a lane
// makes more workgroups (32768 to 64 experts: 7.6 us, with two 8.5) until each has several rounds: 131072 to 256
// experts 11.2 us with one, 10.9 with two.
constexpr int64_t kSortAlone = 2 * SORT_NT;
constexpr int sort_per_lane(int64_t assignments) { return assignments > kSortAlone && assignments <= kMoeSortShort ? 1 : 2; }

// Expert of assignment i, or -1 when it is not one of the num_experts held here.
template <class ID>
__device__ __forceinline__ int expert_of(const ID* ids, int64_t i, int num_experts) {
    const ID v = ids[i];
    return v >= 0 && v < (ID)num_experts ? (int)v : -1;
}

// Fills src_of[0 .. rows) with -1 (rows of no assignment), the workgroups' shares in turn.
__device__ __forceinline__ void clear_src(const MoeSortParams& p) {
    const i32x4 none = {-1, -1, -1, -1};
    const int64_t quads = p.src_aligned ? p.rows >> 2 : 0;
    const int64_t step = (int64_t)gridDim.x * SORT_NT;
    const int64_t at = (int64_t)blockIdx.x * SORT_NT + threadIdx.x;
    for (int64_t q = at; q < quads; q += step) ((gbl_i32x4*)p.src_of)[q] = none;
    for (int64_t r = 4 * quads + at; r < p.rows; r += step) p.src_of[r] = -1;
}

// Workgroup b's assignments [b * chunk, (b + 1) * chunk) counted by expert into hist[b][.].  Bound by
// latencies: 3.0 us for 262144 assignments (2 MB of ids).
template <class ID>
__global__ __launch_bounds__(SORT_NT) void moe_count_kernel(MoeSortParams p) {
    __shared__ int count[kMoeMaxExperts];
    const int tid = threadIdx.x, E = p.num_experts;
    for (int e = tid; e < E; e += SORT_NT) count[e] = 0;
    __syncthreads();
    const int64_t first = (int64_t)blockIdx.x * p.chunk;
    const int64_t last = min(p.assignments, first + p.chunk);
    for (int64_t i = first + tid; i < last; i += SORT_NT) {
        const int e = expert_of((const ID*)p.ids, i, E);
        if (e >= 0) atomicAdd(&count[e], 1);         // integer sums: their order changes nothing
    }
    clear_src(p);
    __syncthreads();
    for (int e = tid; e < E; e += SORT_NT) p.hist[(int64_t)blockIdx.x * E + e] = count[e];
}

// Ranks and places the assignments.  Each workgroup sums the others' counts for itself (at
// most kMoeSortGroups rows of E counts, from L2), which costs less than a launch or a chain of
// waits between workgroups.  Within a wave the lanes of one expert find each other by
// ballots over the bits of the id; a lane's rank is the number of earlier such lanes, and the
// wave's own row of 16-bit counters carries the ranks on.  ALONE: one workgroup does it all,
// with no counts from a first launch.  Bound by latencies: 7.2 us for 262144 assignments to 32 experts
// (128 workgroups), 5.8 us for 512 to 256 (one).
template <class ID, int PER_LANE, bool ALONE>
__global__ __launch_bounds__(SORT_NT) void moe_place_kernel(MoeSortParams p) {
    constexpr int SUB = SORT_NT * PER_LANE;
    __shared__ uint16_t wave_count[SORT_WAVES * kMoeMaxExperts];   // [wave][expert], at most SUB
    __shared__ int base[kMoeMaxExperts];                           // next row of every expert
    __shared__ int total[kMoeMaxExperts];
    __shared__ int wave_sum[SORT_WAVES];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, E = p.num_experts;
    const int64_t first = (int64_t)blockIdx.x * p.chunk;
    const int64_t last = min(p.assignments, first + p.chunk);

    // totals and the sums of the workgroups before this one
    for (int e = tid; e < E; e += SORT_NT) {
        base[e] = 0;
        total[e] = 0;
    }
    if constexpr (ALONE) clear_src(p);
    __syncthreads();
    if constexpr (ALONE) {
        for (int64_t i = first + tid; i < last; i += SORT_NT) {
            const int e = expert_of((const ID*)p.ids, i, E);
            if (e >= 0) atomicAdd(&total[e], 1);
        }
    } else {
        // SORT_NT / E' threads share an expert's column (E' = E up to a power of two)
        int width = 1;
        while (width < E && width < SORT_NT) width <<= 1;
        const int part = tid / width, parts = SORT_NT / width;
        for (int e = tid & (width - 1); e < E; e += width) {
            int before = 0, all = 0;
#pragma unroll 4
            for (int b = part; b < p.groups; b += parts) {
                const int c = p.hist[(int64_t)b * E + e];
                all += c;
                if (b < (int)blockIdx.x) before += c;
            }
            atomicAdd(&total[e], all);
            atomicAdd(&base[e], before);
        }
    }
    __syncthreads();

    // exclusive scan of the padded totals: two consecutive experts a thread
    int padded[2], sum = 0;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int e = 2 * tid + u;
        padded[u] = e < E ? (total[e] + p.alignment - 1) / p.alignment * p.alignment : 0;
        sum += padded[u];
    }
    int scan = sum;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(scan, d);
        if (lane >= d) scan += v;
    }
    if (lane == 63) wave_sum[wave] = scan;
    __syncthreads();
    int start = scan - sum;
    for (int w = 0; w < wave; ++w) start += wave_sum[w];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int e = 2 * tid + u;
        if (e < E) {
            base[e] += start;
            if (blockIdx.x == 0) {
                p.counts[e] = total[e];
                p.offsets[e] = (int)min<int64_t>((int64_t)start + padded[u], p.rows);
            }
        }
        start += padded[u];
    }

    for (int64_t sub = first; sub < last; sub += SUB) {
        for (int i = tid; i < SORT_WAVES * E; i += SORT_NT) wave_count[i] = 0;
        __syncthreads();
        // each wave ranks PER_LANE runs of 64 consecutive assignments
        int expert[PER_LANE], rank[PER_LANE];
        uint16_t* const mine = wave_count + wave * E;
#pragma unroll
        for (int u = 0; u < PER_LANE; ++u) {
            const int64_t i = sub + (wave * PER_LANE + u) * 64 + lane;
            expert[u] = i < last ? expert_of((const ID*)p.ids, i, E) : -1;
        }
#pragma unroll
        for (int u = 0; u < PER_LANE; ++u) {
            const int e = expert[u];
            rank[u] = 0;
            if (sub + (wave * PER_LANE + u) * 64 >= last) continue;
            uint64_t peers = __ballot(e >= 0);
            for (int bit = 0; bit < p.id_bits; ++bit) {
                const uint64_t ones = __ballot((e >> bit) & 1);
                peers &= (e >> bit) & 1 ? ones : ~ones;
            }
            const int earlier = __popcll(peers & ((1ull << lane) - 1));
            int seen = 0;
            if (e >= 0) seen = mine[e];
            rank[u] = seen + earlier;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // the reads above come before the write below
            if (e >= 0 && earlier == 0) mine[e] = (uint16_t)(seen + __popcll(peers));
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
        __syncthreads();
        // exclusive sums over the waves; the sub-chunk's count stays in total[]
        for (int e = tid; e < E; e += SORT_NT) {
            int run = 0;
#pragma unroll
            for (int w = 0; w < SORT_WAVES; ++w) {
                const int c = wave_count[w * E + e];
                wave_count[w * E + e] = (uint16_t)run;
                run += c;
            }
            total[e] = run;
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < PER_LANE; ++u) {
            const int64_t i = sub + (wave * PER_LANE + u) * 64 + lane;
            if (i >= last) continue;
            int row = -1;
            if (expert[u] >= 0) {
                row = base[expert[u]] + mine[expert[u]] + rank[u];
                if (row >= p.rows) row = -1;             // past the caller's rows: dropped
                else p.src_of[row] = (int)i;
            }
            p.row_of[i] = row;
        }
        __syncthreads();
        for (int e = tid; e < E; e += SORT_NT) base[e] += total[e];
        // (the next round's first barrier orders these sums before their next use)
    }
}

// ----------------------------------------------------------------------------
// rows
// ----------------------------------------------------------------------------
constexpr int ROW_NT = kMoeRowThreads;
constexpr int ROW_WAVES = ROW_NT / 64;
constexpr int PAD_ROWS = 2;      // rows whose source one wave looks up before zeroing the empty ones (33024 rows of 7168 bf16, nearly
                                 // all empty: 16 take 96 us, 4 91, 2 89.4, 1 89; 262144 copied ones 789 with 2, 794 with 1)

// 16 bytes at element alignment.
typedef i32x4 Piece2 __attribute__((aligned(2)));
typedef i32x4 Piece4 __attribute__((aligned(4)));
template <int DT>
struct Elem {
    static constexpr int size = DT == kOutF32 ? 4 : 2;
    static constexpr int per = 16 / size;                 // elements of a piece
    using Piece = std::conditional_t<DT == kOutF32, Piece4, Piece2>;
    using Raw = std::conditional_t<DT == kOutF32, uint32_t, uint16_t>;
};
template <int DT>
__device__ __forceinline__ i32x4 load_piece(const char* p) {
    return *(const __attribute__((address_space(1))) typename Elem<DT>::Piece*)p;
}
template <int DT>
__device__ __forceinline__ void store_piece(char* p, i32x4 v) {
    *(__attribute__((address_space(1))) typename Elem<DT>::Piece*)p = v;
}
// The same past the caches' retention, for what is used once (see kStreamBytes).
template <int DT, bool STREAM>
__device__ __forceinline__ i32x4 load_once(const char* p) {
    if constexpr (STREAM) return __builtin_nontemporal_load((const __attribute__((address_space(1))) typename Elem<DT>::Piece*)p);
    else return load_piece<DT>(p);
}
template <int DT>
__device__ __forceinline__ void store_once(char* p, i32x4 v) {
    __builtin_nontemporal_store(v, (__attribute__((address_space(1))) typename Elem<DT>::Piece*)p);
}
template <int DT>
__device__ __forceinline__ void unpack(i32x4 v, float (&f)[Elem<DT>::per]) {
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        if constexpr (DT == kOutF32) {
            f[h] = __builtin_bit_cast(f32x4, v)[h];
        } else {
            f[2 * h] = half_lo<DT>((uint32_t)v[h]);
            f[2 * h + 1] = half_hi<DT>((uint32_t)v[h]);
        }
    }
}
template <int DT>
__device__ __forceinline__ i32x4 pack(const float (&f)[Elem<DT>::per]) {
    i32x4 v;
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        if constexpr (DT == kOutF32) v[h] = __builtin_bit_cast(int, f[h]);
        else v[h] = (int)pack_half2<DT>(f[2 * h], f[2 * h + 1]);
    }
    return v;
}
template <int DT>
__device__ __forceinline__ float load_one(const char* p) {
    if constexpr (DT == kOutF32) return *(const float*)p;
    else return half_lo<DT>((uint32_t)*(const uint16_t*)p);
}
template <int DT>
__device__ __forceinline__ void store_one(char* p, float f) {
    if constexpr (DT == kOutF32) *(float*)p = f;
    else *(uint16_t*)p = (uint16_t)pack_half2<DT>(f, 0.0f);
}

// Zeroes the rows without a source among rows [PAD_ROWS * g, PAD_ROWS * (g + 1)), one wave.
template <int DT>
__device__ __forceinline__ void zero_empty_rows(const MoeRowsParams& p, char* out, int64_t g, int lane) {
    const int64_t r0 = g * PAD_ROWS;
    const int64_t r = r0 + lane;
    const bool empty = lane < PAD_ROWS && r < p.rows && p.src_of[r] < 0;
    uint64_t mask = __ballot(empty);
    const int64_t pieces = p.hidden / Elem<DT>::per;
    const int tail = (int)(p.hidden - pieces * Elem<DT>::per);
    const i32x4 z = {0, 0, 0, 0};
    while (mask) {
        const int i = __builtin_ctzll(mask);
        mask &= mask - 1;
        char* row = out + (r0 + i) * p.hidden * Elem<DT>::size;
        for (int64_t c = lane; c < pieces; c += 64) store_piece<DT>(row + 16 * c, z);
        if (lane < tail) *(typename Elem<DT>::Raw*)(row + 16 * pieces + lane * Elem<DT>::size) = 0;
    }
}

// One wave moves SEG pieces a lane of one token's row to the token's rows; the waves past the
// tokens' zero the empty rows.  512 rows of 33024 copied and the others zeroed: 87 us, 5.4 TB/s.
constexpr int SEG = 2;
template <int DT>
__global__ __launch_bounds__(ROW_NT) void moe_permute_kernel(MoeRowsParams p) {
    using El = Elem<DT>;
    const int lane = threadIdx.x & 63;
    const int64_t item = (int64_t)blockIdx.x * ROW_WAVES + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (item >= p.items) {
        zero_empty_rows<DT>(p, (char*)p.out, item - p.items, lane);
        return;
    }
    const int64_t t = item / p.segments;
    const int64_t c0 = (item - t * p.segments) * (64 * SEG) + lane;
    const int64_t pieces = p.hidden / El::per;
    const char* src = (const char*)p.in + t * p.ld_in * El::size;
    i32x4 v[SEG];
#pragma unroll
    for (int u = 0; u < SEG; ++u)
        if (c0 + 64 * u < pieces) v[u] = load_piece<DT>(src + 16 * (c0 + 64 * u));
    // the row's last elements go with its first segment
    const int tail = (int)(p.hidden - pieces * El::per);
    const bool has_tail = c0 < tail;
    typename El::Raw last = 0;
    const int64_t tail_at = 16 * pieces + c0 * El::size;
    if (has_tail) last = *(const typename El::Raw*)(src + tail_at);
    for (int j = 0; j < p.topk; ++j) {
        const int row = p.row_of[t * p.topk + j];
        if (row < 0 || row >= p.rows) continue;
        char* dst = (char*)p.out + (int64_t)row * p.hidden * El::size;
#pragma unroll
        for (int u = 0; u < SEG; ++u)
            if (c0 + 64 * u < pieces) store_piece<DT>(dst + 16 * (c0 + 64 * u), v[u]);
        if (has_tail) *(typename El::Raw*)(dst + tail_at) = last;
    }
}

// One wave sums USEG pieces a lane of one token's rows, four rows' loads on their way at a time (one
// piece a lane, or four, were slower).
constexpr int USEG = 2;
template <int DT, bool WEIGHTED, bool STREAM>
__global__ __launch_bounds__(ROW_NT) void moe_unpermute_kernel(MoeRowsParams p) {
    using El = Elem<DT>;
    const int lane = threadIdx.x & 63;
    const int64_t item = (int64_t)blockIdx.x * ROW_WAVES + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (item >= p.items) return;
    const int64_t t = item / p.segments;
    const int64_t c0 = (item - t * p.segments) * (64 * USEG) + lane;
    const int64_t pieces = p.hidden / El::per;
    const int tail = (int)(p.hidden - pieces * El::per);
    const bool has_tail = c0 < tail;
    const int64_t tail_at = 16 * pieces + c0 * El::size;
    float acc[USEG][El::per];
#pragma unroll
    for (int u = 0; u < USEG; ++u)
#pragma unroll
        for (int q = 0; q < El::per; ++q) acc[u][q] = 0.0f;
    float last = 0.0f;
#pragma unroll 4
    for (int j = 0; j < p.topk; ++j) {
        const int row = p.row_of[t * p.topk + j];
        if (row < 0 || row >= p.rows) continue;
        const float w = WEIGHTED ? p.weights[t * p.topk + j] : 1.0f;
        const char* src = (const char*)p.in + (int64_t)row * p.ld_in * El::size;
#pragma unroll
        for (int u = 0; u < USEG; ++u)
            if (c0 + 64 * u < pieces) {
                float f[El::per];
                unpack<DT>(load_once<DT, STREAM>(src + 16 * (c0 + 64 * u)), f);
#pragma unroll
                for (int q = 0; q < El::per; ++q) acc[u][q] += WEIGHTED ? w * f[q] : f[q];
            }
        if (has_tail) last += w * load_one<DT>(src + tail_at);
    }
    char* dst = (char*)p.out + t * p.hidden * El::size;
#pragma unroll
    for (int u = 0; u < USEG; ++u)
        if (c0 + 64 * u < pieces) store_once<DT>(dst + 16 * (c0 + 64 * u), pack<DT>(acc[u]));
    if (has_tail) store_one<DT>(dst + tail_at, last);
}

// One workgroup a token: its dout row stays in registers (GSEG pieces a thread; longer rows are
// read again for every j) while its k rows of y are read, reduced against it and the k rows of dy
// written.  The workgroups past the tokens' zero the empty rows of dy.  A wave a token would need no LDS
// for the dot products but four times the registers for the row; a workgroup moves 5.6 TB/s (16384 x 2
// tokens, 4096 bf16: 0.69 GB in 122 us).
constexpr int GSEG = 4;
template <int DT, bool STREAM>
__global__ __launch_bounds__(ROW_NT) void moe_unpermute_grad_kernel(MoeRowsParams p) {
    using El = Elem<DT>;
    __shared__ float part[ROW_WAVES];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t t = blockIdx.x;
    if (t >= p.items) {
        zero_empty_rows<DT>(p, (char*)p.out, (t - p.items) * ROW_WAVES + wave, lane);
        return;
    }
    const int64_t pieces = p.hidden / El::per;
    const int tail = (int)(p.hidden - pieces * El::per);
    const int64_t tail_at = 16 * pieces + tid * El::size;
    const char* dsrc = (const char*)p.in + t * p.ld_in * El::size;
    const bool once = pieces <= GSEG * ROW_NT;
    i32x4 d[GSEG];
#pragma unroll
    for (int u = 0; u < GSEG; ++u)
        if (tid + u * ROW_NT < pieces) d[u] = load_piece<DT>(dsrc + 16 * (int64_t)(tid + u * ROW_NT));
    const float dlast = tid < tail ? load_one<DT>(dsrc + tail_at) : 0.0f;
    for (int j = 0; j < p.topk; ++j) {
        const int row = p.row_of[t * p.topk + j];
        if (row < 0 || row >= p.rows) {
            if (tid == 0) p.dweights[t * p.topk + j] = 0.0f;
            continue;
        }
        const float w = p.weights[t * p.topk + j];
        const char* ysrc = (const char*)p.y + (int64_t)row * p.ld_y * El::size;
        char* dst = (char*)p.out + (int64_t)row * p.hidden * El::size;
        float dot = 0.0f;
        for (int64_t c0 = tid; c0 < pieces; c0 += GSEG * ROW_NT) {
            i32x4 y[GSEG];
#pragma unroll
            for (int u = 0; u < GSEG; ++u)
                if (c0 + u * ROW_NT < pieces) {
                    y[u] = load_once<DT, STREAM>(ysrc + 16 * (c0 + u * ROW_NT));
                    if (!once) d[u] = load_piece<DT>(dsrc + 16 * (c0 + u * ROW_NT));
                }
#pragma unroll
            for (int u = 0; u < GSEG; ++u)
                if (c0 + u * ROW_NT < pieces) {
                    float fd[El::per], fy[El::per];
                    unpack<DT>(d[u], fd);
                    unpack<DT>(y[u], fy);
#pragma unroll
                    for (int q = 0; q < El::per; ++q) {
                        dot += fd[q] * fy[q];
                        fd[q] *= w;
                    }
                    store_once<DT>(dst + 16 * (c0 + u * ROW_NT), pack<DT>(fd));
                }
        }
        if (tid < tail) {
            dot += dlast * load_one<DT>(ysrc + tail_at);
            store_one<DT>(dst + tail_at, w * dlast);
        }
#pragma unroll
        for (int s = 32; s > 0; s >>= 1) dot += __shfl_xor(dot, s);
        __syncthreads();
        if (lane == 0) part[wave] = dot;
        __syncthreads();
        if (tid == 0) p.dweights[t * p.topk + j] = (part[0] + part[1]) + (part[2] + part[3]);
    }
}

template <class ID>
void launch_sort(const MoeSortParams& p, hipStream_t stream) {
    if (p.groups == 1) {
        hipLaunchKernelGGL((moe_place_kernel<ID, 2, true>), dim3(1), dim3(SORT_NT), 0, stream, p);
        return;
    }
    hipLaunchKernelGGL((moe_count_kernel<ID>), dim3(p.groups), dim3(SORT_NT), 0, stream, p);
    if (sort_per_lane(p.assignments) == 1)
        hipLaunchKernelGGL((moe_place_kernel<ID, 1, false>), dim3(p.groups), dim3(SORT_NT), 0, stream, p);
    else
        hipLaunchKernelGGL((moe_place_kernel<ID, 2, false>), dim3(p.groups), dim3(SORT_NT), 0, stream, p);
}

// Pieces of a row, at least one so that a short row's tail has a wave.
int64_t row_segments(int64_t hidden, int dt, int per_lane) {
    const int64_t pieces = hidden * (dt == kOutF32 ? 4 : 2) / 16;
    return pieces <= 64 * per_lane ? 1 : (pieces + 64 * per_lane - 1) / (64 * per_lane);
}

// Waves of one token's row; the gradient has a workgroup a token.
int64_t segments_of(int op, int dt, int64_t hidden) {
    return op == kMoePermute ? row_segments(hidden, dt, SEG) : op == kMoeUnpermute ? row_segments(hidden, dt, USEG) : 1;
}

// Rows of y beyond this are read past the caches' retention: twice the 256 MB Infinity Cache, so they cannot be in it
// from whoever wrote them.  3.8 GB: 784 -> 739 us (unpermute), 1576 -> 1552 us (gradient); but 268 MB, half of which
// is still there: 62 -> 68 us, and 33 MB 11.9 -> 14.5 us.  Sums and gradients are always written that way (826 -> 784 us,
// 77 -> 62 us); permute's copies are not (805 -> 826 us).
constexpr int64_t kStreamBytes = (int64_t)512 << 20;

template <int DT>
void launch_rows(MoeRowsParams p, int op, hipStream_t stream) {
    const bool stream_rows = p.rows * p.hidden * Elem<DT>::size > kStreamBytes;
    p.segments = segments_of(op, DT, p.hidden);
    p.items = p.tokens * p.segments;
    const dim3 grid((uint32_t)moe_rows_grid(op, DT, p.tokens, p.rows, p.hidden));
    auto run = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(ROW_NT), 0, stream, p); };
    if (op == kMoePermute) {
        run(moe_permute_kernel<DT>);
    } else if (op == kMoeUnpermute) {
        if (p.weights) stream_rows ? run(moe_unpermute_kernel<DT, true, true>) : run(moe_unpermute_kernel<DT, true, false>);
        else stream_rows ? run(moe_unpermute_kernel<DT, false, true>) : run(moe_unpermute_kernel<DT, false, false>);
    } else {
        stream_rows ? run(moe_unpermute_grad_kernel<DT, true>) : run(moe_unpermute_grad_kernel<DT, false>);
    }
}

}  // namespace

int64_t moe_rows_grid(int op, int dtype, int64_t tokens, int64_t rows, int64_t hidden) {
    const int64_t pad_waves = op == kMoeUnpermute ? 0 : (rows + PAD_ROWS - 1) / PAD_ROWS;
    if (op == kMoeUnpermuteGrad) return tokens + (pad_waves + ROW_WAVES - 1) / ROW_WAVES;
    return (tokens * segments_of(op, dtype, hidden) + pad_waves + ROW_WAVES - 1) / ROW_WAVES;
}

void moe_sort_plan(int64_t assignments, int32_t* groups, int64_t* chunk) {
    const int64_t sub = SORT_NT * sort_per_lane(assignments);
    int64_t g = assignments <= kSortAlone ? 1 : (assignments + sub - 1) / sub;
    if (g > kMoeSortGroups) g = kMoeSortGroups;
    const int64_t per = (assignments + g - 1) / g;
    *chunk = (per + sub - 1) / sub * sub;
    *groups = (int32_t)g;
}

hipError_t launch_moe_sort(const MoeSortParams& p, bool wide_ids, hipStream_t stream) {
    if (wide_ids) launch_sort<int64_t>(p, stream);
    else launch_sort<int32_t>(p, stream);
    return hipGetLastError();
}

hipError_t launch_moe_rows(const MoeRowsParams& p, int op, int dtype, hipStream_t stream) {
    if (dtype == kOutBf16) launch_rows<kOutBf16>(p, op, stream);
    else if (dtype == kOutF16) launch_rows<kOutF16>(p, op, stream);
    else launch_rows<kOutF32>(p, op, stream);
    return hipGetLastError();
}

}  // namespace kgw
