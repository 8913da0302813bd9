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
#include <type_traits>

#include "kgw_layer.h"
#include "kgw_row_io.h"

namespace kgw {
namespace {

constexpr int NT = kRouteThreads;
constexpr float kTiny = 1e-20f;        // keeps the sums of sigmoids that underflow away from zero
constexpr float kNone = -__builtin_inff();

// Expert of piece q, place c of lane `sub`.
template <int L>
__device__ __forceinline__ int expert_at(int q, int c, int sub) { return 4 * (q * L + sub) + c; }

// A token's scores; -inf past the last expert and where the token takes no part.
template <int DT, int L, int Q>
__device__ __forceinline__ void load_scores(const RouteParams& p, int64_t t, bool live, int sub, float (&x)[4 * Q]) {
    const char* row = (const char*)p.scores + t * p.ld * RowElem<DT>::size;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int e = expert_at<L>(q, 0, sub);
        float f[4] = {kNone, kNone, kNone, kNone};
        if (live) {
            if (e + 4 <= p.experts) {
                load4<DT>(row + (int64_t)e * RowElem<DT>::size, f);
            } else {
#pragma unroll
                for (int c = 0; c < 3; ++c)
                    if (e + c < p.experts) f[c] = load_elem<DT>(row + (int64_t)(e + c) * RowElem<DT>::size);
            }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) x[4 * q + c] = f[c];
    }
}

// u of every score and their sum; a row without any allowed expert has zeros (NaN where a score is NaN).
template <bool SIGMOID>
__device__ __forceinline__ float share_of(float x, float top) {
    if constexpr (SIGMOID) return sigmoid_of(x);
    else return exp2_of((x - top) * kLog2e);
}
__device__ __forceinline__ float finite_top(float top) { return top == kNone ? 0.0f : top; }

__device__ __forceinline__ int64_t given_id(const RouteParams& p, int64_t i) {
    return p.id_bytes == 8 ? ((const int64_t*)p.given)[i] : (int64_t)((const int32_t*)p.given)[i];
}

// The sums of all workgroups' shares of the experts [16 b, 16 b + 16) and what follows from them, or (ALONE) of all
// experts from this workgroup's own.  In a fixed order.
__device__ __forceinline__ float slope_of(const RouteParams& p, int count, int tokens) {
    const float n = (float)tokens;
    return tokens > 0 ? (float)count * ((float)p.experts / (float)p.topk) / (n * n) : 0.0f;
}

// One pass over the scores.  Every workgroup leaves its sums of p, its counts and its tokens in p.part; with a single
// workgroup (ALONE) it writes counts, slope and loss itself.
template <int DT, int L, int Q, bool SIGMOID, bool ALONE>
__global__ __launch_bounds__(ALONE ? 1024 : NT) void route_kernel(RouteParams p) {
    constexpr int THREADS = ALONE ? 1024 : NT;
    constexpr int V = 4 * Q, ROWS = THREADS / L;           // tokens at a time
    constexpr int MOST = L * V < kRouteMaxTopk ? L * V : kRouteMaxTopk;
    constexpr int WAVES = THREADS / 64;
    __shared__ float sums[WAVES][L * V];
    __shared__ int count[L * V];
    __shared__ int sel_id[ROWS][MOST];
    __shared__ float sel_x[ROWS][MOST];
    __shared__ int taking[WAVES];
    __shared__ float dots[WAVES];
    const int tid = threadIdx.x, sub = tid & (L - 1), row = tid / L, lane = tid & 63, wave = tid >> 6;
    const int E = p.experts, K = p.topk;
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
        load_scores<DT, L, Q>(p, t, live, sub, x);
        float best = x[0];
#pragma unroll
        for (int i = 1; i < V; ++i) best = fmaxf(best, x[i]);
        best = lanes_max<L>(best);
        const float top = finite_top(best);
        float u[V], sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            u[i] = share_of<SIGMOID>(x[i], top);
            sum += u[i];
        }
        sum = lanes_sum<L>(sum);
        const bool part = best != kNone || sum != 0.0f;    // (a NaN sum of a row without an allowed expert: seen in the loss)
        const float inverse = part ? 1.0f / (SIGMOID ? sum + kTiny : sum) : 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) psum[i] += u[i] * inverse;
        took += part && sub == 0 ? 1 : 0;
        if (p.given) {
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
                sel_id[row][j] = id;
                sel_x[row][j] = s;
            }
        } else {
            // the largest score, its lowest index, and that one taken out, k times
            for (int j = 0; j < K; ++j) {
                if (j) {
                    best = x[0];
#pragma unroll
                    for (int i = 1; i < V; ++i) best = fmaxf(best, x[i]);
                    best = lanes_max<L>(best);
                }
                int id = 1 << 30;
#pragma unroll
                for (int i = V - 1; i >= 0; --i) id = x[i] == best ? expert_at<L>(i >> 2, i & 3, sub) : id;
                id = lanes_min<L>(id);
#pragma unroll
                for (int i = 0; i < V; ++i) x[i] = expert_at<L>(i >> 2, i & 3, sub) == id ? kNone : x[i];
                if (sub == 0) {
                    sel_id[row][j] = best > kNone ? id : -1;
                    sel_x[row][j] = best;
                }
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // a row's lanes are of one wave
        float chosen = 0.0f;
        for (int j = sub; j < K; j += L)
            if (sel_id[row][j] >= 0) chosen += share_of<SIGMOID>(sel_x[row][j], top);
        chosen = lanes_sum<L>(chosen);
        float per = SIGMOID ? 1.0f : inverse;
        if (p.renormalize) per = SIGMOID ? 1.0f / (chosen + kTiny) : (chosen > 0.0f ? 1.0f / chosen : 0.0f);
        per *= p.scale;
        if (there) {
            for (int j = sub; j < K; j += L) {
                const int id = sel_id[row][j];
                p.ids[t * K + j] = id;
                p.weights[t * K + j] = id >= 0 ? share_of<SIGMOID>(sel_x[row][j], top) * per : 0.0f;
                if (id >= 0) atomicAdd(&count[id], 1);           // integer sums: their order changes nothing
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // the reads above come before the next token's writes
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
        if constexpr (ALONE) {
            const float slope = slope_of(p, count[e], tokens);
            p.counts[e] = count[e];
            p.slope[e] = slope;
            dot += slope * v;
        } else {
            p.part[(int64_t)blockIdx.x * 2 * E + e] = v;
            ((int*)p.part)[(int64_t)blockIdx.x * 2 * E + E + e] = count[e];
        }
    }
    if constexpr (ALONE) {
        dot = lanes_sum<64>(dot);
        if (lane == 0) dots[wave] = dot;
        __syncthreads();
        if (tid == 0) {
            float v = 0.0f;
            for (int w = 0; w < WAVES; ++w) v += dots[w];
            *p.loss = v;
        }
    } else if (tid == 0) {
        ((int*)p.tokens_part)[blockIdx.x] = tokens;
        if (blockIdx.x == 0) *p.arrived = 0;
    }
}

// Adds the workgroups' parts: 16 experts a workgroup, its 256 threads 16 runs of the parts each.  The last workgroup to
// arrive adds the losses of all, in their order.
constexpr int FINISH = 256, COLUMNS = 16;
__global__ __launch_bounds__(FINISH) void route_finish_kernel(RouteParams p) {
    __shared__ float sums[FINISH];
    __shared__ int counts[FINISH];
    __shared__ int taking[FINISH / 64];
    __shared__ float slopes[COLUMNS];
    __shared__ int last;
    const int tid = threadIdx.x, column = tid & (COLUMNS - 1), run = tid / COLUMNS, E = p.experts;
    const int e = blockIdx.x * COLUMNS + column;
    int took = 0;
    for (int g = tid; g < p.groups; g += FINISH) took += ((const int*)p.tokens_part)[g];
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) took += __shfl_xor(took, d);
    if ((tid & 63) == 0) taking[tid >> 6] = took;
    float v = 0.0f;
    int c = 0;
    if (e < E) {
#pragma unroll 4
        for (int g = run; g < p.groups; g += FINISH / COLUMNS) {
            v += p.part[(int64_t)g * 2 * E + e];
            c += ((const int*)p.part)[(int64_t)g * 2 * E + E + e];
        }
    }
    sums[tid] = v;
    counts[tid] = c;
    __syncthreads();
    if (tid < COLUMNS) {
        int tokens = 0;
        for (int w = 0; w < FINISH / 64; ++w) tokens += taking[w];
        v = 0.0f;
        c = 0;
        for (int r = 0; r < FINISH / COLUMNS; ++r) {
            v += sums[r * COLUMNS + column];
            c += counts[r * COLUMNS + column];
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
    load_scores<DT, L, Q>(p, t, live, sub, x);
    float push[V];
    const float dloss = p.dloss ? *p.dloss : 0.0f;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int e = expert_at<L>(q, 0, sub);
#pragma unroll
        for (int c = 0; c < 4; ++c) push[4 * q + c] = p.dloss && e + c < E ? dloss * p.slope[e + c] : 0.0f;
    }
    float best = x[0];
#pragma unroll
    for (int i = 1; i < V; ++i) best = fmaxf(best, x[i]);
    best = lanes_max<L>(best);
    const float top = finite_top(best);
    float u[V], sum = 0.0f, pushed = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        u[i] = share_of<SIGMOID>(x[i], top);
        sum += u[i];
        pushed += u[i] * push[i];
    }
    sum = lanes_sum<L>(sum);
    pushed = lanes_sum<L>(pushed);
    const bool part = best != kNone || sum != 0.0f;
    const float inverse = part ? 1.0f / (SIGMOID ? sum + kTiny : sum) : 0.0f;
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
    for (int j = sub; j < K; j += L) {
        int id;
        float s, dw;
        pick(j, id, s, dw);
        if (id >= 0) {
            const float v = share_of<SIGMOID>(s, top);
            chosen += v;
            weighed += v * dw;
        }
    }
    chosen = lanes_sum<L>(chosen);
    weighed = lanes_sum<L>(weighed);
    float per = SIGMOID ? 1.0f : inverse, less = 0.0f, all = pushed;
    if (p.renormalize) {
        per = SIGMOID ? 1.0f / (chosen + kTiny) : (chosen > 0.0f ? 1.0f / chosen : 0.0f);
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
            if constexpr (SIGMOID) d[c] *= sigmoid_of(-x[i]);
            if (x[i] == kNone) d[c] = 0.0f;
        }
        *(f32x4*)&grad[row][expert_at<L>(q, 0, sub)] = d;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    for (int j = sub; j < K; j += L) {
        int id;
        float s, dw;
        pick(j, id, s, dw);
        if (id >= 0) {
            float d = share_of<SIGMOID>(s, top) * per * (dw - less);
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
    else if (experts <= 512) f(std::integral_constant<int, 64>(), std::integral_constant<int, 2>());
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

RoutePlan route_plan(int64_t tokens, int experts) {
    RoutePlan plan;
    int lanes = 64;
    with_shape(experts, [&](auto l, auto) { lanes = decltype(l)::value; });
    plan.rows = NT / lanes;
    const int64_t wanted = (tokens + plan.rows - 1) / plan.rows;
    plan.groups = (int)(tokens * lanes <= 1024 ? 1 : wanted < kRouteGroups ? wanted : kRouteGroups);
    plan.finish = (experts + COLUMNS - 1) / COLUMNS;
    plan.words = plan.groups == 1 ? 0 : (size_t)plan.groups * (2 * experts + 1) + plan.finish + 1;
    return plan;
}

hipError_t launch_route(const RouteParams& p, int dtype, bool sigmoid, hipStream_t stream) {
    const RoutePlan plan = route_plan(p.tokens, p.experts);
    with_shape(p.experts, [&](auto l, auto q) {
        with_dtype(dtype, [&](auto dt) {
            constexpr int L = decltype(l)::value, Q = decltype(q)::value, DT = decltype(dt)::value;
            const dim3 grid((unsigned)plan.groups);
            if (plan.groups == 1) {
                if (sigmoid) hipLaunchKernelGGL((route_kernel<DT, L, Q, true, true>), grid, dim3(1024), 0, stream, p);
                else hipLaunchKernelGGL((route_kernel<DT, L, Q, false, true>), grid, dim3(1024), 0, stream, p);
            } else {
                if (sigmoid) hipLaunchKernelGGL((route_kernel<DT, L, Q, true, false>), grid, dim3(NT), 0, stream, p);
                else hipLaunchKernelGGL((route_kernel<DT, L, Q, false, false>), grid, dim3(NT), 0, stream, p);
            }
        });
    });
    if (plan.groups > 1)
        hipLaunchKernelGGL(route_finish_kernel, dim3((unsigned)plan.finish), dim3(FINISH), 0, stream, p);
    return hipGetLastError();
}

hipError_t launch_route_grad(const RouteParams& p, int dtype, bool sigmoid, hipStream_t stream) {
    const int rows = route_plan(p.tokens, p.experts).rows;
    const dim3 grid((unsigned)((p.tokens + rows - 1) / rows));
    with_shape(p.experts, [&](auto l, auto q) {
        with_dtype(dtype, [&](auto dt) {
            constexpr int L = decltype(l)::value, Q = decltype(q)::value, DT = decltype(dt)::value;
            if (sigmoid) hipLaunchKernelGGL((route_grad_kernel<DT, L, Q, true>), grid, dim3(NT), 0, stream, p);
            else hipLaunchKernelGGL((route_grad_kernel<DT, L, Q, false>), grid, dim3(NT), 0, stream, p);
        });
    });
    return hipGetLastError();
}

}  // namespace kgw
