// C-ABI layer of the token sort, permute and unpermute: argument checks and dispatch.
// Declarations and the contract of every entry point are in include/kgw.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/kgw.h"
#include "kgw_layer.h"

namespace {

bool aligned_to(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

kgw_status_t usable_device() {
    int32_t is_gfx950 = 0;
    return kgw_device_info(nullptr, &is_gfx950, nullptr) == KGW_SUCCESS && is_gfx950 ? KGW_SUCCESS : KGW_ERROR_DEVICE;
}

int element_size(int32_t dtype) { return dtype == KGW_OUT_FP32 ? 4 : 2; }

constexpr int64_t kMaxRowTokens = (int64_t)1 << 23;

// Checks shared by the calls that move rows.
kgw_status_t check_rows(int op, int32_t dtype, int64_t tokens, int32_t topk, int64_t rows, int64_t hidden) {
    if (dtype != KGW_OUT_FP32 && dtype != KGW_OUT_BF16 && dtype != KGW_OUT_FP16) return KGW_ERROR_INVALID_VALUE;
    if (tokens < 0 || topk < 1 || rows < 0 || hidden < 0) return KGW_ERROR_INVALID_VALUE;
    if (tokens > kMaxRowTokens || topk > 65536 || tokens * (int64_t)topk > INT32_MAX || rows > INT32_MAX)
        return KGW_ERROR_UNSUPPORTED;
    if (hidden >= ((int64_t)1 << 28)) return KGW_ERROR_UNSUPPORTED;
    // HIP counts a grid's threads in 32 bits
    return kgw::moe_rows_grid(op, dtype, tokens, rows, hidden) < ((int64_t)1 << 32) / kgw::kMoeRowThreads
               ? KGW_SUCCESS
               : KGW_ERROR_UNSUPPORTED;
}

bool rows_aligned(const void* p, int32_t dtype) { return aligned_to(p, (uintptr_t)element_size(dtype)); }

kgw_status_t run_rows(const kgw::MoeRowsParams& p, int op, int32_t dtype, void* stream) {
    const kgw_status_t st = usable_device();
    if (st != KGW_SUCCESS) return st;
    return kgw::launch_moe_rows(p, op, dtype, (hipStream_t)stream) == hipSuccess ? KGW_SUCCESS : KGW_ERROR_DEVICE;
}

}  // namespace

extern "C" {

int64_t kgw_moe_rows(int64_t tokens, int32_t topk, int32_t num_experts, int32_t alignment) {
    if (tokens < 0 || topk < 1 || num_experts < 1 || alignment < 1 || tokens > INT32_MAX / topk) return -1;
    const int64_t assignments = tokens * topk;
    const int64_t used = assignments < num_experts ? assignments : num_experts;
    const int64_t rows = (assignments + used * (alignment - 1)) / alignment * alignment;
    return rows <= INT32_MAX ? rows : -1;
}

size_t kgw_moe_sort_workspace_bytes(int64_t tokens, int32_t topk, int32_t num_experts) {
    if (tokens < 0 || topk < 1 || num_experts < 1 || tokens > INT32_MAX / topk) return 0;
    const int64_t assignments = tokens * topk;
    int32_t groups, fewer;
    int64_t chunk;
    kgw::moe_sort_plan(assignments, &groups, &chunk);
    // never less than for fewer tokens, so that a workspace for the most serves all
    kgw::moe_sort_plan(assignments < kgw::kMoeSortShort ? assignments : kgw::kMoeSortShort, &fewer, &chunk);
    if (fewer > groups) groups = fewer;
    return groups > 1 ? (size_t)groups * (size_t)num_experts * sizeof(int32_t) : 0;
}

kgw_status_t kgw_moe_sort(const void* ids, int32_t id_bytes, int64_t tokens, int32_t topk, int32_t num_experts,
                          int32_t alignment, int64_t rows, int32_t* counts, int32_t* offsets, int32_t* row_of,
                          int32_t* src_of, void* workspace, size_t workspace_bytes, void* stream) {
    if (id_bytes != 4 && id_bytes != 8) return KGW_ERROR_INVALID_VALUE;
    if (tokens < 0 || topk < 1 || num_experts < 1 || alignment < 1 || rows < 0) return KGW_ERROR_INVALID_VALUE;
    if (!counts || !offsets || (tokens > 0 && (!ids || !row_of)) || (rows > 0 && !src_of))
        return KGW_ERROR_INVALID_VALUE;
    if (num_experts > kgw::kMoeMaxExperts || tokens > INT32_MAX / topk) return KGW_ERROR_UNSUPPORTED;
    // padded totals are summed in 32 bits
    if (tokens * topk + (int64_t)num_experts * alignment > INT32_MAX || rows > INT32_MAX) return KGW_ERROR_UNSUPPORTED;
    if (rows % alignment != 0) return KGW_ERROR_BAD_OFFSETS;
    if (!aligned_to(ids, (uintptr_t)id_bytes) || !aligned_to(counts, 4) || !aligned_to(offsets, 4) ||
        !aligned_to(row_of, 4) || !aligned_to(src_of, 4) || !aligned_to(workspace, 4))
        return KGW_ERROR_MISALIGNED;
    const size_t need = kgw_moe_sort_workspace_bytes(tokens, topk, num_experts);
    if (need && (!workspace || workspace_bytes < need)) return KGW_ERROR_INVALID_VALUE;
    const kgw_status_t st = usable_device();
    if (st != KGW_SUCCESS) return st;
    kgw::MoeSortParams p;
    p.ids = ids;
    p.counts = counts;
    p.offsets = offsets;
    p.row_of = row_of;
    p.src_of = src_of;
    p.hist = (int32_t*)workspace;
    p.assignments = tokens * topk;
    p.rows = rows;
    p.num_experts = num_experts;
    p.alignment = alignment;
    p.id_bits = 0;
    while ((1 << p.id_bits) < num_experts) ++p.id_bits;
    p.src_aligned = aligned_to(src_of, 16) ? 1 : 0;
    kgw::moe_sort_plan(p.assignments, &p.groups, &p.chunk);
    return kgw::launch_moe_sort(p, id_bytes == 8, (hipStream_t)stream) == hipSuccess ? KGW_SUCCESS : KGW_ERROR_DEVICE;
}

kgw_status_t kgw_moe_permute(const void* x, int64_t ld_x, int32_t dtype, const int32_t* row_of,
                             const int32_t* src_of, int64_t tokens, int32_t topk, int64_t rows, int64_t hidden,
                             void* out, void* stream) {
    const kgw_status_t st = check_rows(kgw::kMoePermute, dtype, tokens, topk, rows, hidden);
    if (st != KGW_SUCCESS) return st;
    if (rows == 0 || hidden == 0) return KGW_SUCCESS;
    if (!src_of || !out || (tokens > 0 && (!x || !row_of || ld_x < hidden))) return KGW_ERROR_INVALID_VALUE;
    if (!rows_aligned(x, dtype) || !rows_aligned(out, dtype) || !aligned_to(row_of, 4) || !aligned_to(src_of, 4))
        return KGW_ERROR_MISALIGNED;
    kgw::MoeRowsParams p = {};
    p.in = x;
    p.out = out;
    p.row_of = row_of;
    p.src_of = src_of;
    p.ld_in = ld_x;
    p.tokens = tokens;
    p.rows = rows;
    p.hidden = hidden;
    p.topk = topk;
    return run_rows(p, kgw::kMoePermute, dtype, stream);
}

kgw_status_t kgw_moe_unpermute(const void* y, int64_t ld_y, int32_t dtype, const int32_t* row_of,
                               const float* weights, int64_t tokens, int32_t topk, int64_t rows, int64_t hidden,
                               void* out, void* stream) {
    const kgw_status_t st = check_rows(kgw::kMoeUnpermute, dtype, tokens, topk, rows, hidden);
    if (st != KGW_SUCCESS) return st;
    if (tokens == 0 || hidden == 0) return KGW_SUCCESS;
    if (!row_of || !out || (rows > 0 && (!y || ld_y < hidden))) return KGW_ERROR_INVALID_VALUE;
    if (!rows_aligned(y, dtype) || !rows_aligned(out, dtype) || !aligned_to(row_of, 4) || !aligned_to(weights, 4))
        return KGW_ERROR_MISALIGNED;
    kgw::MoeRowsParams p = {};
    p.in = y;
    p.out = out;
    p.row_of = row_of;
    p.weights = weights;
    p.ld_in = ld_y;
    p.tokens = tokens;
    p.rows = rows;
    p.hidden = hidden;
    p.topk = topk;
    return run_rows(p, kgw::kMoeUnpermute, dtype, stream);
}

kgw_status_t kgw_moe_unpermute_grad(const void* dout, int64_t ld_dout, const void* y, int64_t ld_y, int32_t dtype,
                                    const int32_t* row_of, const int32_t* src_of, const float* weights,
                                    int64_t tokens, int32_t topk, int64_t rows, int64_t hidden, void* dy,
                                    float* dweights, void* stream) {
    const kgw_status_t st = check_rows(kgw::kMoeUnpermuteGrad, dtype, tokens, topk, rows, hidden);
    if (st != KGW_SUCCESS) return st;
    if (tokens == 0 && (rows == 0 || hidden == 0)) return KGW_SUCCESS;
    if (tokens > 0 && (!row_of || !weights || !dweights)) return KGW_ERROR_INVALID_VALUE;
    if (hidden > 0 && tokens > 0 && (!dout || ld_dout < hidden)) return KGW_ERROR_INVALID_VALUE;
    if (rows > 0 && (!src_of || (hidden > 0 && (!y || !dy || ld_y < hidden)))) return KGW_ERROR_INVALID_VALUE;
    if (!rows_aligned(dout, dtype) || !rows_aligned(y, dtype) || !rows_aligned(dy, dtype) || !aligned_to(row_of, 4) ||
        !aligned_to(src_of, 4) || !aligned_to(weights, 4) || !aligned_to(dweights, 4))
        return KGW_ERROR_MISALIGNED;
    kgw::MoeRowsParams p = {};
    p.in = dout;
    p.y = y;
    p.out = dy;
    p.dweights = dweights;
    p.weights = weights;
    p.row_of = row_of;
    p.src_of = src_of;
    p.ld_in = ld_dout;
    p.ld_y = ld_y;
    p.tokens = tokens;
    p.rows = rows;
    p.hidden = hidden;
    p.topk = topk;
    return run_rows(p, kgw::kMoeUnpermuteGrad, dtype, stream);
}

}  // extern "C"
