// The router of a mixture-of-experts layer (gfx950): each token's experts and weights from its scores, the counts
// of every expert, the balance loss and the gradients of all of it.
//
//   u = exp(score - top) or sigmoid(score)           p = u / sum u
//   ids: the k largest scores, ties to the lowest index     weights = p (sigmoid: u) at ids, or u / sum of the chosen
//   N tokens take part, expert e has c_e assignments:  slope_e = E c_e / (k N^2),  loss = sum over t, e of slope_e p_te
//
// which is 1 when experts are used alike, and is differentiated through p alone (slope is constant: counts have no
// gradient).  With push_e = dloss slope_e and the chosen experts' dw_j (times `scale`):
//
//   softmax   ds_e = p_e (push_e - sum p push) + { p_j dw_j - p_e sum p_j dw_j
//                                                { q_j (dw_j - sum q dw)   at the chosen only, q = u / sum of the chosen
//   sigmoid   ds_e = u_e (1 - u_e) [(push_e - sum p push) / sum u + the chosen's part]
//
// A row of E scores is held by L lanes (4 to 64), V to a lane, so that a wave takes 64 / L tokens at once and sums and
// maxima over a row stay in registers.  The scores are read once, in pieces of four at element alignment.
//
// Vector instructions bound the forward kernel where there are many tokens (top-k needs several per score), launches and
// the call's issue elsewhere.  Measured, MI355X: 32768 x 256 fp32, top 8 of sigmoids, 17.8 us and 5.7 us for the sums
// of the workgroups' parts (its bytes, 36 MB, take 7 us); 64 x 256 in one workgroup and launch 7.8 us; 5003 x 61 bf16 5.2 and
// 4.1 us; fp32 softmax, top 8: 32768 x 32 7.6 and 3.9 us, 20000 x 512 26 and 7.4, 65536 x 512 49 and 7.8, 16384 x 2048 79 and 19;
// given ids: 32768 x 256 11.8 and 6.7 us, 32768 x 32 6.7 and 4.1, 16384 x 2048 34 and 20.
// Gradient: 32768 x 32 fp32 5.9 us, 16411 x 256 fp16 7.0 us (17.6 MB from the Infinity Cache: 2.5 TB/s).
#include <type_traits>

#include "kgw_layer.h"
#include "kgw_row_io.h"

namespace kgw {
namespace {

constexpr int NT = 256;                // of the gradient's workgroups
constexpr float kTiny = 1e-20f;        // keeps the sums of sigmoids that underflow away from zero
constexpr float kNone = -__builtin_inff();

// Expert of piece q, place c of lane `sub`; and of value i = 4 q + c, less the lane's part 4 sub.
template <int L>
__device__ __forceinline__ int expert_at(int q, int c, int sub) { return 4 * (q * L + sub) + c; }
template <int L>
__device__ __forceinline__ constexpr int slot_of(int i) { return 4 * L * (i >> 2) + (i & 3); }

// The pieces of a row of E as they are read: no branch a piece, lanes past the end read the row's last piece, and a last
// piece of fewer than four is read from the row's end.
template <int DT, int L, int Q>
__device__ __forceinline__ void load_pieces(const char* row, int E, int sub, float (&x)[4 * Q]) {
    constexpr int S = RowElem<DT>::size;
    if (L > 4 || E >= 4) {                                 // (only the smallest shape has rows of fewer)
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            float f[4];
            load4<DT>(row + (int64_t)min(expert_at<L>(q, 0, sub), E - 4) * S, f);
#pragma unroll
            for (int c = 0; c < 4; ++c) x[4 * q + c] = f[c];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4 * Q; ++i) x[i] = 0.0f;
#pragma unroll
        for (int c = 0; c < 3; ++c)
            if (c < E) x[c] = load_elem<DT>(row + c * S);
    }
}
// Moves a last piece down to its place; `none` past the row's end and where the row is not live.
template <int L, int Q>
__device__ __forceinline__ void place_pieces(int E, bool live, int sub, float none, float (&x)[4 * Q]) {
    if (L > 4 || E >= 4) {
        const int over = -E & 3;                           // uniform: by how much the last piece was moved
        if (over) {
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const int e = expert_at<L>(q, 0, sub);
                const bool moved = e < E && e + 4 > E;
                const float f1 = x[4 * q + 1], f2 = x[4 * q + 2], f3 = x[4 * q + 3];
                x[4 * q] = moved ? (over == 1 ? f1 : over == 2 ? f2 : f3) : x[4 * q];
                x[4 * q + 1] = moved ? (over == 1 ? f2 : over == 2 ? f3 : none) : f1;
                x[4 * q + 2] = moved ? (over == 1 ? f3 : none) : f2;
                x[4 * q + 3] = moved ? none : f3;
            }
        }
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const bool in = live && expert_at<L>(q, 0, sub) < E;
#pragma unroll
            for (int c = 0; c < 4; ++c) x[4 * q + c] = in ? x[4 * q + c] : none;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4 * Q; ++i) x[i] = live && sub == 0 && i < E ? x[i] : none;
    }
}

// A token's scores as they are read (a token past the last one is read as the last).
template <int DT, int L, int Q>
__device__ __forceinline__ void load_scores(const RouteParams& p, int64_t t, int sub, float (&x)[4 * Q]) {
    load_pieces<DT, L, Q>((const char*)p.scores + min(t, p.tokens - 1) * p.ld * RowElem<DT>::size, p.experts, sub, x);
}

// Whole numbers in the order of the scores (-0 as 0; NaN, which is never chosen, as -inf), and back.
__device__ __forceinline__ int order_of(float x) {
    const int v = __builtin_bit_cast(int, fmaxf(x + 0.0f, kNone));
    return v ^ ((v >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float score_of(int order) {
    return __builtin_bit_cast(float, order ^ ((order >> 31) & 0x7FFFFFFF));
}
constexpr int kNoOrder = (int)0x807FFFFF;              // of -inf

template <int V>
__device__ __forceinline__ int max_of(const int (&x)[V]) {
    int m = x[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = max(m, x[i]);
    return m;
}

// How many of the other lanes of 16 come before this one: a larger order, or the same one and a lower expert (rare but for
// 16-bit scores, so looked at only where a wave has any).
template <int N = 1>
__device__ __forceinline__ int larger_of(int order, bool& tie) {
    if constexpr (N == 16) {
        return 0;
    } else {
        const int other = lane_dpp<0x120 + N>(order);      // row rotation
        tie = tie || other == order;
        return (other > order ? 1 : 0) + larger_of<N + 1>(order, tie);
    }
}
template <int N = 1>
__device__ __forceinline__ int tied_before(int order, int e) {
    if constexpr (N == 16) {
        return 0;
    } else {
        const int other = lane_dpp<0x120 + N>(order), oe = lane_dpp<0x120 + N>(e);
        return (other == order && oe < e ? 1 : 0) + tied_before<N + 1>(order, e);
    }
}
__device__ __forceinline__ int rank_of(int order, int e, bool counts) {
    bool tie = false;
    int rank = larger_of(order, tie);
    if (__any(tie && counts)) rank += tied_before(order, e);
    return rank;
}

// u of every score and their sum; a row without any allowed expert has zeros (NaN where a score is NaN).
template <bool SIGMOID>
__device__ __forceinline__ float share_of(float x, float top) {
    if constexpr (SIGMOID) return sigmoid_of(x);
    else return exp2_of((x - top) * kLog2e);
}
// 1 - u of a sigmoid u without a second exponential: e / (1 + e) with e = exp(-x), held below 2^125 so that neither it nor
// u is lost (u is within 2^-125 of the sigmoid then).  -inf has u = 0.
__device__ __forceinline__ float other_share(float x, float& u) {
    const float e = fminf(exp2_of(-kLog2e * x), 0x1p125f);               // (a NaN score: the sum of u is NaN)
    u = x == kNone ? 0.0f : x != x ? x : reciprocal(1.0f + e);
    return e * reciprocal(1.0f + e);
}
__device__ __forceinline__ float finite_top(float top) { return top == kNone ? 0.0f : top; }

__device__ __forceinline__ int64_t given_id(const RouteParams& p, int64_t i) {
    return p.id_bytes == 8 ? ((const int64_t*)p.given)[i] : (int64_t)((const int32_t*)p.given)[i];
}

__device__ __forceinline__ float slope_of(const RouteParams& p, int count, int tokens) {
    const float n = (float)tokens;
    return tokens > 0 ? (float)count * ((float)p.experts / (float)p.topk) / (n * n) : 0.0f;
}

// One pass over the scores.  Every workgroup leaves its sums of p, its counts and its tokens in p.part; a single
// workgroup writes counts, slope and loss itself.
// GIVEN: the caller's ids.
template <int DT, int L, int Q, int THREADS, bool GIVEN>
__global__ __launch_bounds__(THREADS) void route_kernel(RouteParams p) {
    constexpr int V = 4 * Q, ROWS = THREADS / L;           // tokens at a time
    constexpr int MOST = L * V < kRouteMaxTopk ? L * V : kRouteMaxTopk;
    constexpr int WAVES = THREADS / 64;
    __shared__ float sums[WAVES][L * V];
    __shared__ int count[L * V];
    __shared__ int sel[ROWS][2][MOST + 1];                 // a row's chosen experts, and their scores' order
    __shared__ int taking[WAVES];
    __shared__ float dots[WAVES];
    const int tid = threadIdx.x, sub = tid & (L - 1), row = tid / L, lane = tid & 63, wave = tid >> 6;
    const int E = p.experts, K = p.topk;
    const bool sigmoid = p.sigmoid != 0;
    for (int e = tid; e < E; e += THREADS) count[e] = 0;
    __syncthreads();
    float psum[V];
#pragma unroll
    for (int i = 0; i < V; ++i) psum[i] = 0.0f;
    int took = 0;
    for (int64_t first = (int64_t)blockIdx.x * ROWS; first < p.tokens; first += (int64_t)gridDim.x * ROWS) {
        const int64_t t = first + row;
        const bool there = t < p.tokens;
        const bool live = there && (!p.mask || p.mask[t]);
        float x[V];
        load_scores<DT, L, Q>(p, t, sub, x);
        place_pieces<L, Q>(E, live, sub, kNone, x);
        int order[V];
#pragma unroll
        for (int i = 0; i < V; ++i) order[i] = order_of(x[i]);
        const int mine = max_of(order);                    // the largest of the lane, and of the row
        int best = lanes_max<L>(mine);
        const float top = best == kNoOrder ? 0.0f : score_of(best);
        float sum = 0.0f;
        if (sigmoid) {
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] = share_of<true>(x[i], top);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] = share_of<false>(x[i], top);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) sum += x[i];
        sum = lanes_sum<L>(sum);
        const bool part = best != kNoOrder || sum != 0.0f; // (a NaN sum of a row without an allowed expert: seen in the loss)
        const float inverse = part ? reciprocal(sigmoid ? sum + kTiny : sum) : 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) psum[i] += x[i] * inverse;
        took += part && sub == 0 ? 1 : 0;
        // weights of the chosen, of which this lane has u (0: none) of `held`; sums go over the row's lanes
        auto factor = [&](float held) __attribute__((always_inline)) {
            const float chosen = lanes_sum<L>(held);
            float per = sigmoid ? 1.0f : inverse;
            if (p.renormalize) per = sigmoid ? reciprocal(chosen + kTiny) : (chosen > 0.0f ? reciprocal(chosen) : 0.0f);
            return per * p.scale;
        };
        // (beside `from`: the row's largest score, or that of the chosen)
        auto share = [&](float x, float from) __attribute__((always_inline)) { return sigmoid ? share_of<true>(x, from) : share_of<false>(x, from); };
        auto leave = [&](int j, int id, float u, float per) __attribute__((always_inline)) {
            p.ids[t * K + j] = id;
            p.weights[t * K + j] = id >= 0 ? u * per : 0.0f;
            if (id >= 0) atomicAdd(&count[id], 1);         // integer sums: their order changes nothing
        };
        if constexpr (L == 16 && !GIVEN) {
            // The k-th largest of the 16 lanes' maxima (or less, where they tie) bounds the chosen from below; what
            // reaches it is seldom more than 16 scores.  They go to a lane each, through LDS, and every lane counts those
            // before its own.
            if (K <= 16) {
                int bound = mine, least = best;
                for (int j = 1; j < K; ++j) {
                    bound = bound == least ? kNoOrder : bound;
                    least = lanes_max<L>(bound);
                }
                least = max(least, kNoOrder + 1);
                int n = 0;
#pragma unroll
                for (int i = 0; i < V; ++i) n += order[i] >= least ? 1 : 0;
                const int total = lanes_sum<L>(n);
                if (!__any(total > 16)) {
                    int at = n;                            // inclusive sums over the lanes
                    at += __builtin_amdgcn_update_dpp(0, at, 0x111, 0xF, 0xF, true);
                    at += __builtin_amdgcn_update_dpp(0, at, 0x112, 0xF, 0xF, true);
                    at += __builtin_amdgcn_update_dpp(0, at, 0x114, 0xF, 0xF, true);
                    at += __builtin_amdgcn_update_dpp(0, at, 0x118, 0xF, 0xF, true);
                    at -= n;
                    int e4 = 4 * sub, from = least;        // (neither V sums nor V comparisons are to be kept for here)
                    asm volatile("" : "+v"(e4), "+v"(from));
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const bool keep = order[i] >= from;              // the others go where nobody looks
                        int* const to = &sel[row][0][keep ? at : MOST];
                        to[0] = slot_of<L>(i) + e4;
                        to[MOST + 1] = order[i];
                        at += keep ? 1 : 0;
                    }
                    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // a row's lanes are of one wave
                    const int id = sub < total ? sel[row][0][sub] : 1 << 30;
                    const int key = sub < total ? sel[row][1][sub] : kNoOrder;
                    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // the next token's writes come after
                    const int rank = rank_of(key, id, sub < total);
                    const bool taken = sub < total && rank < K;
                    const float u = taken ? share(score_of(key), top) : 0.0f;
                    const float per = factor(u);
                    if (there && taken) leave(rank, id, u, per);
                    if (there && sub >= total && sub < K) leave(sub, -1, 0.0f, 0.0f);
                    continue;
                }
            }
        }
        if constexpr (GIVEN) {
            for (int j = sub; j < K; j += L) {
                int id = -1;
                float s = kNone;
                if (live) {
                    const int64_t v = given_id(p, t * K + j);
                    if (v >= 0 && v < E) {
                        s = load_elem<DT>((const char*)p.scores + (t * p.ld + v) * RowElem<DT>::size);
                        id = s > kNone ? (int)v : -1;
                    }
                }
                sel[row][0][j] = id;
                sel[row][1][j] = order_of(s);
            }
        } else {
            // the largest score, its lowest index, and that one taken out, k times
            for (int j = 0; j < K; ++j) {
                if (j) best = lanes_max<L>(max_of(order));
                int id = 1 << 30;
#pragma unroll
                for (int i = V - 1; i >= 0; --i) id = order[i] == best ? slot_of<L>(i) : id;
                id = lanes_min<L>(id + 4 * sub);
                const int slot = id - 4 * sub;
#pragma unroll
                for (int i = 0; i < V; ++i) order[i] = slot_of<L>(i) == slot ? kNoOrder : order[i];
                if (sub == 0) {
                    sel[row][0][j] = best > kNoOrder ? id : -1;
                    sel[row][1][j] = best;
                }
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        float from = top;
        if constexpr (GIVEN) {
            // The caller's need not have the row's largest score, beside which their shares may all vanish: those that are
            // made to sum to one go by the largest of their own.
            if (p.renormalize && !sigmoid) {
                int most = kNoOrder;
                for (int j = sub; j < K; j += L) most = max(most, sel[row][1][j]);
                most = lanes_max<L>(most);
                from = most == kNoOrder ? 0.0f : score_of(most);
            }
        }
        float held = 0.0f;
        for (int j = sub; j < K; j += L)
            if (sel[row][0][j] >= 0) held += share(score_of(sel[row][1][j]), from);
        const float per = factor(held);
        if (there)
            for (int j = sub; j < K; j += L) leave(j, sel[row][0][j], share(score_of(sel[row][1][j]), from), per);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    // the wave's tokens, then the waves in turn
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float v = psum[i];
#pragma unroll
        for (int d = L; d < 64; d <<= 1) v += __shfl_xor(v, d);
        if (lane < L) sums[wave][expert_at<L>(i >> 2, i & 3, sub)] = v;
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) took += __shfl_xor(took, d);
    if (lane == 0) taking[wave] = took;
    __syncthreads();
    int tokens = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) tokens += taking[w];
    float dot = 0.0f;
    for (int e = tid; e < E; e += THREADS) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) v += sums[w][e];
        if (gridDim.x == 1) {
            const float slope = slope_of(p, count[e], tokens);
            p.counts[e] = count[e];
            p.slope[e] = slope;
            dot += slope * v;
        } else {
            p.part[(int64_t)blockIdx.x * E + e] = {v, __builtin_bit_cast(float, count[e])};
        }
    }
    if (gridDim.x == 1) {
        dot = lanes_sum<64>(dot);
        if (lane == 0) dots[wave] = dot;
        __syncthreads();
        if (tid == 0) {
            float v = 0.0f;
            for (int w = 0; w < WAVES; ++w) v += dots[w];
            *p.loss = v;
        }
    } else if (tid == 0) {
        p.tokens_part[blockIdx.x] = tokens;
        if (blockIdx.x == 0) *p.arrived = 0;
    }
}

// Adds the workgroups' parts: 16 experts a workgroup, 64 runs of the parts.  The last workgroup to arrive adds the losses
// of all, in their order.
constexpr int FINISH = 1024, COLUMNS = 16;
__global__ __launch_bounds__(FINISH) void route_finish_kernel(RouteParams p) {
    __shared__ float sums[FINISH / 64][COLUMNS];
    __shared__ int counts[FINISH / 64][COLUMNS];
    __shared__ int taking[FINISH / 64];
    __shared__ float slopes[COLUMNS];
    __shared__ int last;
    const int tid = threadIdx.x, column = tid & (COLUMNS - 1), run = tid / COLUMNS, E = p.experts;
    const int e = blockIdx.x * COLUMNS + column;
    int took = 0;
    for (int g = tid; g < p.groups; g += FINISH) took += p.tokens_part[g];
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) took += __shfl_xor(took, d);
    if ((tid & 63) == 0) taking[tid >> 6] = took;
    float v = 0.0f;
    int c = 0;
    if (e < E) {
#pragma unroll 8
        for (int g = run; g < p.groups; g += FINISH / COLUMNS) {
            const RoutePart part = p.part[(int64_t)g * E + e];
            const float counted = part[1];                 // (a bit cast of a vector's element would take its first)
            v += part[0];
            c += __builtin_bit_cast(int, counted);
        }
    }
#pragma unroll
    for (int d = COLUMNS; d < 64; d <<= 1) {
        v += __shfl_xor(v, d);
        c += __shfl_xor(c, d);
    }
    if ((tid & 63) < COLUMNS) {
        sums[tid >> 6][column] = v;
        counts[tid >> 6][column] = c;
    }
    __syncthreads();
    // a wave has four runs of every column, which it adds across its lanes; then 16 waves' are left
    if (tid < COLUMNS) {
        int tokens = 0;
#pragma unroll
        for (int w = 0; w < FINISH / 64; ++w) tokens += taking[w];
        v = 0.0f;
        c = 0;
#pragma unroll
        for (int r = 0; r < FINISH / 64; ++r) {
            v += sums[r][column];
            c += counts[r][column];
        }
        const float slope = slope_of(p, c, tokens);
        if (e < E) {
            p.counts[e] = c;
            p.slope[e] = slope;
        }
        slopes[column] = e < E ? slope * v : 0.0f;
    }
    __syncthreads();
    if (tid == 0) {
        float dot = 0.0f;
        for (int k = 0; k < COLUMNS; ++k) dot += slopes[k];
        __hip_atomic_store(p.dots + blockIdx.x, dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        last = __hip_atomic_fetch_add(p.arrived, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == (int)gridDim.x - 1;
        if (last) {
            dot = 0.0f;
            for (int b = 0; b < (int)gridDim.x; ++b)
                dot += __hip_atomic_load(p.dots + b, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            *p.loss = dot;
        }
    }
}

// The gradient: one token a row of lanes.  The chosen experts' own terms are added to the row in LDS.
template <int DT, int L, int Q, bool SIGMOID>
__global__ __launch_bounds__(NT) void route_grad_kernel(RouteParams p) {
    constexpr int V = 4 * Q, ROWS = NT / L;
    __shared__ __attribute__((aligned(16))) float grad[ROWS][L * V];
    const int tid = threadIdx.x, sub = tid & (L - 1), row = tid / L;
    const int E = p.experts, K = p.topk;
    const int64_t t = (int64_t)blockIdx.x * ROWS + row;
    const bool there = t < p.tokens;
    const bool live = there && (!p.mask || p.mask[t]);
    float x[V];
    load_scores<DT, L, Q>(p, t, sub, x);
    place_pieces<L, Q>(E, live, sub, kNone, x);
    float push[V];
#pragma unroll
    for (int i = 0; i < V; ++i) push[i] = 0.0f;
    if (p.dloss) {
        const float dloss = *p.dloss;
        load_pieces<kOutF32, L, Q>((const char*)p.slope, E, sub, push);
        place_pieces<L, Q>(E, true, sub, 0.0f, push);
#pragma unroll
        for (int i = 0; i < V; ++i) push[i] *= dloss;
    }
    float best = x[0];
#pragma unroll
    for (int i = 1; i < V; ++i) best = fmaxf(best, x[i]);
    best = lanes_max<L>(best);
    const float top = finite_top(best);
    float u[V], sum = 0.0f, pushed = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if constexpr (SIGMOID) x[i] = other_share(x[i], u[i]);           // 1 - u is all that is left to know of x
        else u[i] = share_of<false>(x[i], top);
        sum += u[i];
        pushed += u[i] * push[i];
    }
    sum = lanes_sum<L>(sum);
    pushed = lanes_sum<L>(pushed);
    const bool part = best != kNone || sum != 0.0f;
    const float inverse = part ? reciprocal(SIGMOID ? sum + kTiny : sum) : 0.0f;
    pushed *= inverse;
    // sums over the chosen
    float chosen = 0.0f, weighed = 0.0f;
    auto pick = [&](int j, int& id, float& s, float& dw) __attribute__((always_inline)) {
        id = -1;
        s = kNone;
        dw = 0.0f;
        if (live) {
            const int64_t v = given_id(p, t * K + j);
            if (v >= 0 && v < E) {
                s = load_elem<DT>((const char*)p.scores + (t * p.ld + v) * RowElem<DT>::size);
                if (s > kNone) {
                    id = (int)v;
                    dw = p.dweights ? p.dweights[t * K + j] * p.scale : 0.0f;
                }
            }
        }
    };
    int id0 = -1;
    float s0 = kNone, dw0 = 0.0f;                          // the lane's first; a lane has more where K > L
    if (sub < K) pick(sub, id0, s0, dw0);
    float from = top;                                      // as in the forward pass
    if (!SIGMOID && p.renormalize) {
        float most = id0 >= 0 ? s0 : kNone;
        for (int j = sub + L; j < K; j += L) {
            int id;
            float s, dw;
            pick(j, id, s, dw);
            most = id >= 0 ? fmaxf(most, s) : most;
        }
        from = finite_top(lanes_max<L>(most));
    }
    for (int j = sub; j < K; j += L) {
        int id = id0;
        float s = s0, dw = dw0;
        if (j != sub) pick(j, id, s, dw);
        if (id >= 0) {
            const float v = share_of<SIGMOID>(s, from);
            chosen += v;
            weighed += v * dw;
        }
    }
    chosen = lanes_sum<L>(chosen);
    weighed = lanes_sum<L>(weighed);
    float per = SIGMOID ? 1.0f : inverse, less = 0.0f, all = pushed;
    if (p.renormalize) {
        per = SIGMOID ? reciprocal(chosen + kTiny) : (chosen > 0.0f ? reciprocal(chosen) : 0.0f);
        less = weighed * per;
    } else if (!SIGMOID) {
        all += weighed * inverse;
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        f32x4 d;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int i = 4 * q + c;
            d[c] = (push[i] - all) * (u[i] * inverse);
            if constexpr (SIGMOID) d[c] *= x[i];
            // zero, not zero times something: for a masked token and a score of -inf whatever is infinite or NaN elsewhere
            d[c] = u[i] != 0.0f ? d[c] : 0.0f;
        }
        *(f32x4*)&grad[row][expert_at<L>(q, 0, sub)] = d;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    for (int j = sub; j < K; j += L) {
        int id = id0;
        float s = s0, dw = dw0;
        if (j != sub) pick(j, id, s, dw);
        if (id >= 0) {
            float d = share_of<SIGMOID>(s, from) * per * (dw - less);
            if constexpr (SIGMOID) d *= sigmoid_of(-s);
            atomicAdd(&grad[row][id], d);                    // adds up where a token names an expert twice
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (!there) return;
    char* out = (char*)p.dscores + t * E * RowElem<DT>::size;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int e = expert_at<L>(q, 0, sub);
        const f32x4 d = *(const f32x4*)&grad[row][e];
        const float f[4] = {d[0], d[1], d[2], d[3]};
        if (e + 4 <= E) {
            store4<DT>(out + (int64_t)e * RowElem<DT>::size, f);
        } else {
#pragma unroll
            for (int c = 0; c < 3; ++c)
                if (e + c < E) store_elem<DT>(out + (int64_t)(e + c) * RowElem<DT>::size, f[c]);
        }
    }
}

// Calls f(lanes of a row, pieces of a lane) with the smallest pair that holds `experts`.
template <class F>
void with_shape(int experts, F f) {
    if (experts <= 32) f(std::integral_constant<int, 4>(), std::integral_constant<int, 2>());
    else if (experts <= 64) f(std::integral_constant<int, 8>(), std::integral_constant<int, 2>());
    else if (experts <= 128) f(std::integral_constant<int, 16>(), std::integral_constant<int, 2>());
    else if (experts <= 256) f(std::integral_constant<int, 16>(), std::integral_constant<int, 4>());
    else if (experts <= 512) f(std::integral_constant<int, 16>(), std::integral_constant<int, 8>());
    else if (experts <= 1024) f(std::integral_constant<int, 64>(), std::integral_constant<int, 4>());
    else f(std::integral_constant<int, 64>(), std::integral_constant<int, 8>());
}
template <class F>
void with_dtype(int dtype, F f) {
    if (dtype == kOutF32) f(std::integral_constant<int, kOutF32>());
    else if (dtype == kOutBf16) f(std::integral_constant<int, kOutBf16>());
    else f(std::integral_constant<int, kOutF16>());
}

}  // namespace

// Workgroups of 1024 threads where all of a CU's waves then have tokens, or where one takes all of them in a round (one
// launch); of 256 between these, so that more CUs have some, and where the ids are given and there is little to do.  Lanes
// of 32 scores need 207 registers, of which 1024 threads leave them 128: 512 then (65536 x 512 97 -> 60 us, 16384 x 2048 112 -> 97,
// 64 x 512 in one workgroup 18 -> 15).  Workgroups of 256 threads are at most 1024, past 512 experts 512: the second launch
// reads a part of every expert for each of them (4096 x 2048 45 us, with 1024 of them 49; 4096 x 1024 27 and 28; 3000 x 700 24 and 23;
// only many tokens with given ids do better with more: 65536 x 1024 95 and 70).
template <int Q>
constexpr int kWide = Q == 8 ? 512 : 1024;
RoutePlan route_plan(int64_t tokens, int experts, bool given) {
    RoutePlan plan;
    int lanes = 64, wide = 1024;
    with_shape(experts, [&](auto l, auto q) {
        lanes = decltype(l)::value;
        wide = kWide<decltype(q)::value>;
    });
    const int64_t threads = tokens * lanes;
    const bool one = !given && threads <= 1024;
    plan.threads = one || (!given && threads > 1024 * kRouteGroups) ? wide : 256;
    const int64_t wanted = one ? 1 : (threads + plan.threads - 1) / plan.threads;
    const int64_t most = plan.threads == wide ? kRouteGroups : experts <= 512 ? 4 * kRouteGroups : 2 * kRouteGroups;
    plan.groups = (int)(wanted < 1 ? 1 : wanted < most ? wanted : most);
    plan.finish = (experts + COLUMNS - 1) / COLUMNS;
    plan.words = plan.groups == 1 ? 0 : (size_t)plan.groups * (2 * experts + 1) + plan.finish + 1;
    return plan;
}

hipError_t launch_route(const RouteParams& p, int dtype, hipStream_t stream) {
    const RoutePlan plan = route_plan(p.tokens, p.experts, p.given != nullptr);
    with_shape(p.experts, [&](auto l, auto q) {
        with_dtype(dtype, [&](auto dt) {
            constexpr int L = decltype(l)::value, Q = decltype(q)::value, DT = decltype(dt)::value;
            const dim3 grid((unsigned)plan.groups);
            if (p.given) hipLaunchKernelGGL((route_kernel<DT, L, Q, 256, true>), grid, dim3(256), 0, stream, p);
            else if (plan.threads == kWide<Q>) hipLaunchKernelGGL((route_kernel<DT, L, Q, kWide<Q>, false>), grid, dim3(kWide<Q>), 0, stream, p);
            else hipLaunchKernelGGL((route_kernel<DT, L, Q, 256, false>), grid, dim3(256), 0, stream, p);
        });
    });
    if (plan.groups > 1)
        hipLaunchKernelGGL(route_finish_kernel, dim3((unsigned)plan.finish), dim3(FINISH), 0, stream, p);
    return hipGetLastError();
}

hipError_t launch_route_grad(const RouteParams& p, int dtype, bool sigmoid, hipStream_t stream) {
    with_shape(p.experts, [&](auto l, auto q) {
        with_dtype(dtype, [&](auto dt) {
            constexpr int L = decltype(l)::value, Q = decltype(q)::value, DT = decltype(dt)::value, ROWS = NT / L;
            const dim3 grid((unsigned)((p.tokens + ROWS - 1) / ROWS));
            if (sigmoid) hipLaunchKernelGGL((route_grad_kernel<DT, L, Q, true>), grid, dim3(NT), 0, stream, p);
            else hipLaunchKernelGGL((route_grad_kernel<DT, L, Q, false>), grid, dim3(NT), 0, stream, p);
        });
    });
    return hipGetLastError();
}

}  // namespace kgw
