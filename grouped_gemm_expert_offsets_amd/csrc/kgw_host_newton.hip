// C-ABI layer of the Newton-Schulz orthogonalisation: argument checks and dispatch.
// Declarations and the contract of every entry point are in include/kgw.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/kgw.h"
#include "kgw_layer.h"

namespace {

// The result's type without its flag.
int32_t result_type(int32_t out_dtype) { return out_dtype & ~KGW_NEWTON_PRECISE; }

bool known_dtype(int32_t d) { return d == KGW_OUT_FP32 || d == KGW_OUT_BF16 || d == KGW_OUT_FP16; }

// Three products of 16-bit halves rather than one.
bool split(int32_t out_dtype) { return result_type(out_dtype) != KGW_OUT_BF16 || (out_dtype & KGW_NEWTON_PRECISE); }

kgw_status_t check_sizes(int32_t batch, int64_t m, int64_t n, int32_t out_dtype) {
    if (batch < 0 || m < 0 || n < 0 || !known_dtype(result_type(out_dtype))) return KGW_ERROR_INVALID_VALUE;
    // a tile's rows are addressed with 32-bit byte offsets, a grid has 16-bit y and z extents
    if (batch > 65535 || m > ((int64_t)1 << 20) || n > ((int64_t)1 << 20)) return KGW_ERROR_UNSUPPORTED;
    const int64_t r = (m < n ? m : n) + 256, c = (m < n ? n : m) + 256;
    if (r / 64 > 65535 || batch * (r / 128) * (c / 128) >= (int64_t)1 << 23) return KGW_ERROR_UNSUPPORTED;
    return KGW_SUCCESS;
}

}  // namespace

extern "C" {

size_t kgw_newton_schulz_workspace_bytes(int32_t batch, int64_t m, int64_t n, int32_t out_dtype) {
    if (check_sizes(batch, m, n, out_dtype) != KGW_SUCCESS || batch == 0 || m == 0 || n == 0) return 0;
    return kgw::newton_plan(batch, m, n, split(out_dtype)).total;
}

kgw_status_t kgw_newton_schulz(const void* G, int64_t ld, int64_t stride, int32_t dtype, int32_t batch, int64_t m,
                               int64_t n, int32_t steps, const float* coefficients, float eps, void* out,
                               int32_t out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
    if (!known_dtype(dtype) || steps < 1 || !coefficients || !(eps >= 0.0f)) return KGW_ERROR_INVALID_VALUE;
    kgw_status_t st = check_sizes(batch, m, n, out_dtype);
    if (st != KGW_SUCCESS) return st;
    if (steps > kgw::kNewtonMaxSteps) return KGW_ERROR_UNSUPPORTED;
    if (batch == 0 || m == 0 || n == 0) return KGW_SUCCESS;
    if (!G || !out || !workspace || ld < n || (batch > 1 && stride < 0)) return KGW_ERROR_INVALID_VALUE;
    if (((uintptr_t)G & (dtype == KGW_OUT_FP32 ? 3u : 1u)) || ((uintptr_t)out & (result_type(out_dtype) == KGW_OUT_FP32 ? 3u : 1u)) ||
        ((uintptr_t)workspace & 255u))
        return KGW_ERROR_MISALIGNED;
    const kgw::NewtonPlan plan = kgw::newton_plan(batch, m, n, split(out_dtype));
    if (workspace_bytes < plan.total) return KGW_ERROR_INVALID_VALUE;
    int32_t num_cus = 0, is_gfx950 = 0, num_xcds = 1;
    if (kgw_device_info(&num_cus, &is_gfx950, &num_xcds) != KGW_SUCCESS || !is_gfx950) return KGW_ERROR_DEVICE;
    kgw::NewtonParams p;
    p.G = G;
    p.out = out;
    p.ld = ld;
    p.stride = stride;
    p.m = m;
    p.n = n;
    p.batch = batch;
    p.dtype = dtype;
    p.out_dtype = result_type(out_dtype);
    p.steps = steps;
    p.eps = eps;
    char* ws = (char*)workspace;
    p.x[0] = ws;
    p.x[1] = ws + plan.x_bytes;
    p.a = ws + 2 * plan.x_bytes;
    p.b = p.a + plan.a_bytes;
    // at least 8192 elements a workgroup of the norm
    const int64_t parts = (m * n + 8191) / 8192;
    p.num_parts = (int32_t)(parts < kgw::kNewtonParts ? parts : kgw::kNewtonParts);
    p.parts = (double*)(p.b + plan.b_bytes);
    char* const slabs = p.b + plan.b_bytes + plan.parts_bytes;
    p.slabs = plan.slab_bytes ? (float*)slabs : nullptr;
    p.arrived = plan.slab_bytes ? (uint32_t*)(slabs + plan.slab_bytes - kgw::kNewtonSlabs * sizeof(uint32_t)) : nullptr;
    p.scales = (kgw::StepScales*)(slabs + plan.slab_bytes);
    p.planes = (int32_t*)(p.scales + (size_t)batch * kgw::kNewtonMaxSteps);
    return kgw::launch_newton(p, plan, coefficients, num_cus, num_xcds, (hipStream_t)stream) == hipSuccess
               ? KGW_SUCCESS
               : KGW_ERROR_DEVICE;
}

}  // extern "C"
