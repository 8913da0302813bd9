// Host/device launch contract of the operators around the grouped products: the token sort,
// permute and unpermute (kgw_moe.hip) and the Newton-Schulz orthogonalisation (kgw_newton.hip).
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
// Newton-Schulz orthogonalisation (kgw_newton.hip)
// ----------------------------------------------------------------------------
constexpr int kNewtonMaxSteps = 64;
constexpr int kNewtonParts = 256;       // partial sums of squares per matrix, at most

constexpr int kNewtonSlabs = 256;       // workgroups that may share tiles: one for every CU

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
};

// The factor c of one step's (a, b, c), for c A A + b A = c (A A + b / c A): one that is nothing beside b
// is made 2^-60 b, which still is.
inline float newton_c(const float* co) {
    const float least = co[1] < 0.0f ? -co[1] * 0x1p-60f : co[1] * 0x1p-60f;
    return co[2] > least || co[2] < -least ? co[2] : co[1] * 0x1p-60f;
}

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
    size_t x_bytes, a_bytes, b_bytes, parts_bytes, slab_bytes, total;
};
constexpr int64_t kNarrowMax = 128;
NewtonPlan newton_plan(int32_t batch, int64_t m, int64_t n, int32_t out_dtype);
void newton_narrow_plan(int32_t batch, int64_t r, int64_t c, NewtonPlan* plan);
void launch_newton_norm(const NewtonParams& p, hipStream_t stream);
void launch_newton_narrow(const NewtonParams& p, const NewtonPlan& plan, const float* coefficients, hipStream_t stream);
hipError_t launch_newton(const NewtonParams& p, const NewtonPlan& plan, const float* coefficients, int num_cus,
                         int num_xcds, hipStream_t stream);

}  // namespace kgw
