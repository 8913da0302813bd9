// Host/device launch contract of the operators around the grouped products: the token sort,
// permute and unpermute (kgw_moe.hip), the router (kgw_route.hip), the activation with its 8-bit checkpoint (kgw_act.hip)
// and the Newton-Schulz orthogonalisation (kgw_newton.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kgw {

// ----------------------------------------------------------------------------
// tokens sorted by expert and back (kgw_moe.hip)
// ----------------------------------------------------------------------------
constexpr int kMoeMaxExperts = 2048;    // per-wave counters of one workgroup stay in LDS
constexpr int kMoeSortGroups = 128;     // workgroups of the sort (each reads the others' counts)

struct MoeSortParams {
    const void* ids;        // (assignments,) int32 or int64
    int32_t* counts;        // (num_experts,)
    int32_t* offsets;       // (num_experts,) inclusive, aligned, at most rows
    int32_t* row_of;        // (assignments,)
    int32_t* src_of;        // (rows,)
    int32_t* hist;          // (groups, num_experts) workspace, groups > 1 only
    int64_t assignments;
    int64_t chunk;          // assignments of one workgroup
    int64_t rows;
    int32_t num_experts;
    int32_t alignment;
    int32_t groups;
    int32_t id_bits;        // bits that tell the experts apart
    int32_t src_aligned;    // src_of is 16-byte aligned
};

struct MoeRowsParams {
    const void* in;         // permute: x; unpermute: y; gradient: dout
    const void* y;          // gradient only
    void* out;              // permute: rows; unpermute: tokens; gradient: dy (contiguous)
    float* dweights;        // gradient only
    const float* weights;   // (tokens, topk) or NULL
    const int32_t* row_of;  // (tokens, topk)
    const int32_t* src_of;  // (rows,)
    int64_t ld_in, ld_y;    // row strides in elements
    int64_t tokens, rows, hidden;
    int64_t items;          // waves (permute, unpermute) or workgroups (gradient) of tokens
    int64_t segments;       // waves of one row
    int32_t topk;
};

constexpr int kMoePermute = 0, kMoeUnpermute = 1, kMoeUnpermuteGrad = 2;
constexpr int kMoeRowThreads = 256;     // of a workgroup of the row kernels

// Workgroups of the sort and the assignments of each.
constexpr int64_t kMoeSortShort = 65536;    // up to here smaller shares, so that up to 64 workgroups have one
void moe_sort_plan(int64_t assignments, int32_t* groups, int64_t* chunk);
hipError_t launch_moe_sort(const MoeSortParams& p, bool wide_ids, hipStream_t stream);
// Workgroups that launch_moe_rows() starts.
int64_t moe_rows_grid(int op, int dtype, int64_t tokens, int64_t rows, int64_t hidden);
hipError_t launch_moe_rows(const MoeRowsParams& p, int op, int dtype, hipStream_t stream);

// ----------------------------------------------------------------------------
// the router (kgw_route.hip)
// ----------------------------------------------------------------------------
constexpr int kRouteMaxTopk = 64;
constexpr int kRouteGroups = 256;       // workgroups of 1024 (or 512) threads, at most (of 256: four times as many, past 512 experts twice)

typedef float RoutePart __attribute__((ext_vector_type(2)));     // a workgroup's sum of an expert's shares, and its count

struct RouteParams {
    const void* scores;     // (tokens, experts)
    const uint8_t* mask;    // (tokens,) or NULL
    const void* given;      // (tokens, topk) ids that the caller has, or NULL; the gradient: the ids
    int32_t* ids;           // (tokens, topk)
    float* weights;         // (tokens, topk)
    int32_t* counts;        // (experts,)
    float* loss;            // (1,)
    float* slope;           // (experts,); the gradient: the caller's
    const float* dweights;  // gradient only, from here on: (tokens, topk) or NULL
    const float* dloss;     // (1,) or NULL
    void* dscores;          // (tokens, experts), contiguous
    // workspace, with more than one workgroup: every workgroup's parts (groups, experts), its tokens, the
    // finishing workgroups' parts of the loss and their counter
    RoutePart* part;
    int32_t* tokens_part;
    float* dots;
    int32_t* arrived;
    int64_t ld;             // of scores, in elements
    int64_t tokens;
    int32_t experts;
    int32_t topk;
    int32_t id_bytes;
    int32_t renormalize;
    int32_t sigmoid;        // (the gradient's kernels are told apart by it)
    int32_t groups;
    float scale;
};

struct RoutePlan {
    int threads;            // of a workgroup
    int groups;             // workgroups (1: no workspace)
    int finish;             // workgroups that add the others' parts
    size_t words;           // of workspace
};
RoutePlan route_plan(int64_t tokens, int experts, bool given);
hipError_t launch_route(const RouteParams& p, int dtype, hipStream_t stream);
hipError_t launch_route_grad(const RouteParams& p, int dtype, bool sigmoid, hipStream_t stream);

// ----------------------------------------------------------------------------
// the activation and its 8-bit checkpoint (kgw_act.hip)
// ----------------------------------------------------------------------------
struct ActParams {
    const void* h;          // (rows, inner), gated (rows, 2 inner); forward only
    const void* dy;         // (rows, inner); gradient only
    uint8_t* saved;         // e4m3 of h, contiguous (forward: NULL keeps none)
    uint8_t* saved_scales;  // (blocks of a row, rows)
    void* y;                // (rows, inner), contiguous (gradient: NULL for none)
    uint8_t* y_scales;      // y is e4m3 with these scales (NULL: y has the rows' type)
    void* dh;               // as h, contiguous; gradient only
    uint8_t* dh_scales;     // likewise
    const int32_t* offsets; // (num_experts,) or NULL: rows from the last one on are left alone
    int64_t ld_h, ld_dy;    // row strides in elements
    int64_t rows, inner;
    int32_t num_experts;
    int32_t group_rows;     // rows of a workgroup
};
int act_group_rows(int64_t rows, int64_t inner);
int64_t act_grid(int64_t rows, int64_t inner);
hipError_t launch_act(const ActParams& p, int dtype, bool gated, bool grad, hipStream_t stream);

// ----------------------------------------------------------------------------
// Newton-Schulz orthogonalisation (kgw_newton.hip)
// ----------------------------------------------------------------------------
constexpr int kNewtonMaxSteps = 64;
constexpr int kNewtonParts = 256;       // partial sums of squares per matrix, at most

constexpr int kNewtonSlabs = 256;       // workgroups that may share tiles: one for every CU

// One step of one matrix, in the planes' powers of two: B = square (A A + square_linear A), then
// X = update (B X + update_linear X).
struct alignas(16) StepScales {
    float square, square_linear, update, update_linear;
};

struct NewtonCoefficients {
    float v[3 * kNewtonMaxSteps];       // a, b, c of every step
    StepScales unit[kNewtonMaxSteps];   // the scales of a matrix whose norm is nothing beside eps
    int32_t measured;                   // the scales come from the norm of every step's A instead
};

// An upper bound on an iterate's singular values, m 2^e with m in [1, 2), and what its planes hold: it times
// 2^(13 - plane).  The largest of the singular values is at least ratio times the bound.
struct SingularBound {
    float m;
    int e, plane;
    float ratio;
};
__host__ __device__ inline SingularBound unit_bound(float ratio) { return {1.0f + 0x1p-20f, 0, 0, ratio}; }

// The scales of the step X <- a X + (b A + c A A) X for a matrix of bound s, which becomes the bound of the next.
//
// Singular values go through f(x) = x (a + b x^2 + c x^4), those of B are b x^2 + c x^4: with x = s t, u = t^2,
// their largest values for t in [0, 1] are at t = 1 or where the derivatives vanish, 5 g u^2 + 3 h u + a = 0 and
// 2 g u + h = 0 (h = b s^2, g = c s^4).  Everything is taken times 2^-q, which brings the largest of a, h and g near 1,
// so that no size of coefficients or matrix leaves fp32's range here.  B's power follows the larger of B and a: what
// a B far below a loses does not matter beside a X.
__host__ __device__ inline StepScales step_scales(SingularBound& s, const float* co, bool last) {
    const float a = co[0], b = co[1], c = co[2];
    auto exponent = [](float x) {                           // 2^exponent <= |x|; far below all others for zero
        int e = 0;
        __builtin_frexpf(x, &e);
        return x != 0.0f ? e - 1 : -100000;
    };
    auto at_most = [](float x, float y) { return x < y ? x : y; };
    auto at_least = [](float x, float y) { return x > y ? x : y; };      // y for a NaN x
    const int ea = exponent(a), eb = exponent(b) + 2 * s.e, ec = exponent(c) + 4 * s.e;
    const int q = ea > eb ? (ea > ec ? ea : ec) : (eb > ec ? eb : ec);
    const float m2 = s.m * s.m;
    const float b0 = __builtin_ldexpf(b, 2 * s.e - q), c0 = __builtin_ldexpf(c, 4 * s.e - q);
    const float al = __builtin_ldexpf(a, -q), h = b0 * m2, g = c0 * m2 * m2;
    auto inner = [&](float u) { return al + u * (h + g * u); };
    auto value = [&](float u) { return __builtin_sqrtf(u) * __builtin_fabsf(inner(u)); };
    auto inside = [&](float u, float from) { return at_most(at_least(u, from), 1.0f); };
    const float root = __builtin_sqrtf(at_least(9.0f * h * h - 20.0f * al * g, 0.0f));
    const float w = -0.5f * (3.0f * h + __builtin_copysignf(root, h));
    const float flat0 = w / (5.0f * g), flat1 = al / w, turn = -0.5f * h / g;
    const float gain = at_least(value(1.0f), at_least(value(inside(flat0, 0.0f)), value(inside(flat1, 0.0f))));
    const float in = inside(turn, 0.0f);
    const float of_b = at_least(__builtin_fabsf(h + g), __builtin_fabsf(in * (h + g * in)));
    const float largest = at_least(of_b, __builtin_fabsf(al));
    const int lg = largest > 0.0f ? exponent(largest) : 0;
    const int b_power = 8 - lg - q;                         // the planes hold B times 2^b_power
    // c A A + b A = c (A A + b / c A); a c that is nothing beside b is made 2^-60 b, which still is
    const int below = s.plane - s.e;                        // the planes' powers of two above the bound's
    const float b1 = __builtin_ldexpf(b0, 2 * below - 2 - lg);
    float c1 = __builtin_ldexpf(c0, 4 * below - 12 - lg);
    if (__builtin_fabsf(c1) <= __builtin_fabsf(b1) * 0x1p-60f) c1 = b1 * 0x1p-60f;
    StepScales r;
    r.square = c1;
    r.square_linear = c1 != 0.0f ? b1 / c1 : 0.0f;
    // the least that the largest singular value, from ratio to 1 of the bound, may become
    const float from = s.ratio * s.ratio;
    const float least = at_most(at_most(value(from), value(1.0f)),
                                at_most(value(inside(flat0, from)), value(inside(flat1, from))));
    const float p0 = inner(from), p1 = inner(1.0f), p2 = inner(inside(turn, from));
    s.ratio = p0 * p1 > 0.0f && p0 * p2 > 0.0f && gain > 0.0f ? least / gain : 0.0f;      // a zero in between: anything
    const float next = s.m * gain;
    const bool any = next > 0.0f && next < 0x1p100f;
    int e = any ? s.e + q + exponent(next) : 0;
    e = e < -2000 ? -2000 : e > 2000 ? 2000 : e;            // past fp32's range either way
    r.update = __builtin_ldexpf(1.0f, s.plane - b_power - (last ? 13 : e));
    r.update_linear = __builtin_ldexpf(a, b_power);
    s.m = any ? __builtin_ldexpf(next, -exponent(next)) : 1.0f;
    s.e = s.plane = e;
    return r;
}

// Whether the scales may follow the bounds alone: the bounds stay about as near the singular values as |G|_F is (within
// its square root of r), as they do for coefficients that bring singular values below 1 together.  Where they part (f
// grows steeply towards 1, or vanishes in between), planes made for the bound would leave the iterate too few bits.
constexpr float kBoundLoss = 1.0f / 16.0f;

struct NewtonParams {
    const void* G;          // (batch, m, n), rows contiguous
    void* out;              // (batch, m, n), contiguous
    int64_t ld, stride;     // of G, in elements
    int64_t m, n;
    int32_t batch;
    int32_t dtype, out_dtype;
    int32_t steps;
    float eps;
    // workspace
    double* parts;          // (batch, kNewtonParts), the first num_parts used
    int32_t num_parts;
    char* x[2];             // iterates, see kgw_newton.hip and kgw_newton_narrow.hip
    char* a;
    char* b;
    float* slabs;           // (kNewtonSlabs, tile, tile), small tiles only
    uint32_t* arrived;      // (kNewtonSlabs,), or NULL
    StepScales* scales;     // (batch, kNewtonMaxSteps)
    int32_t* planes;        // (2, batch): SingularBound::plane of even and odd steps, for measured scales
};

// How a batch is computed, and the layout of its workspace.
struct NewtonPlan {
    bool tall;              // m > n: the iterates hold the transposes
    bool narrow;            // short side at most kNarrowMax: kgw_newton_narrow.hip
    bool split;             // three products of 16-bit halves instead of one
    int32_t tile;           // edge of the output tiles
    int64_t r, c;           // padded sizes of the iterates, r the short side
    int32_t chunks;         // narrow: 128-column chunks of a matrix
    int32_t per_group;      // narrow: chunks of one workgroup
    int32_t groups;         // narrow: workgroups of a matrix (0: one that runs all steps)
    size_t x_bytes, a_bytes, b_bytes, parts_bytes, slab_bytes, scales_bytes, total;
};
constexpr int64_t kNarrowMax = 128;
NewtonPlan newton_plan(int32_t batch, int64_t m, int64_t n, bool split);
void newton_narrow_plan(int32_t batch, int64_t r, int64_t c, NewtonPlan* plan);
void launch_newton_norm(const NewtonParams& p, hipStream_t stream);
void launch_newton_narrow(const NewtonParams& p, const NewtonPlan& plan, const NewtonCoefficients& co, hipStream_t stream);
hipError_t launch_newton(const NewtonParams& p, const NewtonPlan& plan, const float* coefficients, int num_cus,
                         int num_xcds, hipStream_t stream);

}  // namespace kgw
