"""Python binding of libkgw: the K-grouped MoE weight-gradient GEMM for MI355X.

For expert e with token range [begin, end) from int32 inclusive cumulative
offsets (begin = 0 for the first expert, offsets[e-1] otherwise; end =
offsets[e]) the library computes

    Wgrad[e] = A[:, begin:end] @ B[begin:end, :]

into a dense (num_experts, hidden, n) output, overwriting it or accumulating
into it (cuDNN "Grouped GEMM + WGrad (Unified)", section "Operation").

Every function here only marshals arguments (tensor shapes, dtypes, device
pointers, the current HIP stream) and calls the C-ABI entry point of the
same name in libkgw.so; all arithmetic runs in the library's HIP kernels.
Status codes 1-4 raise ValueError, 5 raises RuntimeError (the cuDNN page,
section "Scheduling, cache, and errors", splits errors the same way).
There is no fallback: without the built library every call raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

import torch

__all__ = [
    "kgw_wgrad_bf16", "kgw_wgrad_bf16_noalloc", "kgw_wgrad_bf16_ex", "kgw_wgrad_fp8", "kgw_wgrad_fp8_native", "kgw_wgrad_fp8_ex",
    "kgw_wgrad_fp4", "FP4_TOKEN_ALIGN", "kgw_wgrad_fp8_rows",
    "kgw_quantize_fp8", "kgw_quantize_fp4", "kgw_mgrouped_bf16", "kgw_mgrouped_fp8", "kgw_workspace_bytes",
    "kgw_moe_route", "kgw_moe_route_grad", "kgw_moe_act_fp8", "kgw_moe_act_fp8_grad",
    "kgw_moe_rows", "kgw_moe_sort", "kgw_moe_permute", "kgw_moe_unpermute", "kgw_moe_unpermute_grad",
    "kgw_newton_schulz", "NEWTON_SCHULZ_COEFFICIENTS", "KGW_NEWTON_PRECISE",
    "KGW_LAYOUT_NT",
    "KGW_LAYOUT_NN",
    "KGW_A_M_MAJOR", "KGW_B_K_MAJOR", "KGW_RAGGED",
    "kgw_validate_offsets", "kgw_check_offsets", "kgw_mfma_ceiling",
    "kgw_validate_offsets_host", "kgw_status_string", "kgw_device_info", "wgrad",
    "KGW_SUCCESS", "KGW_ERROR_INVALID_VALUE", "KGW_ERROR_MISALIGNED", "KGW_ERROR_BAD_OFFSETS",
    "KGW_ERROR_UNSUPPORTED", "KGW_ERROR_DEVICE", "KGW_OUT_FP32", "KGW_OUT_BF16", "KGW_OUT_FP16",
    "KGW_SCALES_U8", "KGW_SCALES_PACKED", "KGW_SCALES_PACKED_32", "scale_shape",
    "BF16_TOKEN_ALIGN", "FP8_TOKEN_ALIGN", "library_path", "load_library",
]

KGW_SUCCESS = 0
KGW_ERROR_INVALID_VALUE = 1
KGW_ERROR_MISALIGNED = 2
KGW_ERROR_BAD_OFFSETS = 3
KGW_ERROR_UNSUPPORTED = 4
KGW_ERROR_DEVICE = 5
KGW_OUT_FP32 = 0
KGW_OUT_BF16 = 1
KGW_OUT_FP16 = 2
KGW_A_M_MAJOR = 1          # weight-gradient A stored (tokens_sum, hidden)
KGW_B_K_MAJOR = 2          # weight-gradient B stored (n, tokens_sum)
KGW_RAGGED = 4             # per-expert K-contiguous blocks back to back (with KGW_B_K_MAJOR)
KGW_LAYOUT_NT = 0          # m-grouped forward: W (E, N, K)
KGW_LAYOUT_NN = 1          # m-grouped dgrad:   W (E, K, N)
KGW_NEWTON_PRECISE = 0x100 # with an out_dtype of kgw_newton_schulz: fp32's precision for bf16 results too
KGW_SCORE_SOFTMAX = 0      # the router's shares: softmax of a token's scores
KGW_SCORE_SIGMOID = 1      # sigmoids, divided by their sum for the balance loss
KGW_ACT_SWIGLU = 0         # silu(g) * u of rows [g | u]
KGW_ACT_RELU2 = 1          # relu(h)^2
KGW_SCALES_U8 = 0          # uint8 (tokens/128, mn)
KGW_SCALES_PACKED = 1      # int32 (ceil(tokens/512), mn): four 128-token blocks per word
KGW_SCALES_PACKED_32 = 2   # int32 (tokens/128, mn): four 32-token blocks per word
BF16_TOKEN_ALIGN = 256
FP8_TOKEN_ALIGN = 128
FP4_TOKEN_ALIGN = 256

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libkgw.so")
_lib = None

# Every symbol include/kgw.h declares.
EXPORTED_SYMBOLS = ("kgw_wgrad_bf16", "kgw_wgrad_bf16_noalloc", "kgw_wgrad_bf16_ex", "kgw_wgrad_fp8", "kgw_wgrad_fp8_native",
                    "kgw_wgrad_fp8_ex", "kgw_wgrad_fp4", "kgw_quantize_fp8", "kgw_quantize_fp4", "kgw_mgrouped_bf16",
                    "kgw_mgrouped_fp8", "kgw_workspace_bytes", "kgw_validate_offsets_host", "kgw_validate_offsets", "kgw_check_offsets",
                    "kgw_mfma_ceiling", "kgw_status_string", "kgw_device_info", "kgw_moe_rows",
                    "kgw_moe_sort_workspace_bytes", "kgw_moe_sort", "kgw_moe_permute", "kgw_moe_unpermute",
                    "kgw_moe_unpermute_grad", "kgw_newton_schulz", "kgw_newton_schulz_workspace_bytes", "kgw_wgrad_fp8_rows",
                    "kgw_wgrad_fp8_rows_workspace_bytes", "kgw_moe_route_workspace_bytes", "kgw_moe_route", "kgw_moe_route_grad", "kgw_moe_act_fp8",
                    "kgw_moe_act_fp8_grad")


def load_library():
    """Load libkgw.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(library_path):
        raise RuntimeError(f"{library_path} is missing: build it with "
                           "`python -m grouped_gemm_expert_offsets_amd.build`")
    lib = ctypes.CDLL(library_path)
    p, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    lib.kgw_wgrad_bf16.restype = ctypes.c_int
    lib.kgw_wgrad_bf16.argtypes = [p, p, p, i32, i64, i64, i64, p, i32, i32, p, sz, p]
    lib.kgw_wgrad_bf16_noalloc.restype = ctypes.c_int
    lib.kgw_wgrad_bf16_noalloc.argtypes = [p, p, p, i32, i64, i64, i64, p, i32, i32, p]
    lib.kgw_wgrad_fp8.restype = ctypes.c_int
    lib.kgw_wgrad_fp8.argtypes = [p, p, p, p, p, i32, i64, i64, i64, p, i32, i32, p, sz, p]
    lib.kgw_wgrad_fp8_native.restype = ctypes.c_int
    lib.kgw_wgrad_fp8_native.argtypes = [p, p, p, p, p, i32, i64, i64, i64, p, i32, i32, p, sz, p]
    lib.kgw_wgrad_bf16_ex.restype = ctypes.c_int
    lib.kgw_wgrad_bf16_ex.argtypes = [p, p, i32, p, i32, i64, i64, i64, p, p, i32, i32, p, sz, p]
    lib.kgw_wgrad_fp8_ex.restype = ctypes.c_int
    lib.kgw_wgrad_fp8_ex.argtypes = [p, p, p, p, i32, i32, i32, p, i32, i64, i64, i64, p, p, i32, i32, p, sz, p]
    lib.kgw_wgrad_fp4.restype = ctypes.c_int
    lib.kgw_wgrad_fp4.argtypes = [p, p, p, p, p, i32, i64, i64, i64, p, p, i32, i32, p, sz, p]
    lib.kgw_mgrouped_bf16.restype = ctypes.c_int
    lib.kgw_mgrouped_bf16.argtypes = [p, p, i32, p, p, i32, i64, i64, i64, p, i32, i32, p]
    lib.kgw_mgrouped_fp8.restype = ctypes.c_int
    lib.kgw_mgrouped_fp8.argtypes = [p, p, p, p, i32, p, p, i32, i64, i64, i64, p, i32, i32, p]
    lib.kgw_quantize_fp8.restype = ctypes.c_int
    lib.kgw_quantize_fp8.argtypes = [p, i64, i64, i32, i32, p, p, p]
    lib.kgw_quantize_fp4.restype = ctypes.c_int
    lib.kgw_quantize_fp4.argtypes = [p, i64, i64, i32, i32, p, p, p]
    lib.kgw_workspace_bytes.restype = sz
    lib.kgw_workspace_bytes.argtypes = [i32, i64, i64, i64, i32]
    lib.kgw_validate_offsets_host.restype = ctypes.c_int
    lib.kgw_validate_offsets_host.argtypes = [p, i32, i64, i32, ctypes.POINTER(i32)]
    lib.kgw_validate_offsets.restype = ctypes.c_int
    lib.kgw_validate_offsets.argtypes = [p, i32, i64, i32, ctypes.POINTER(i32), p]
    lib.kgw_check_offsets.restype = ctypes.c_int
    lib.kgw_check_offsets.argtypes = [p, i32, i64, i32, p, p]
    lib.kgw_mfma_ceiling.restype = ctypes.c_int
    lib.kgw_mfma_ceiling.argtypes = [p, i64, i32, i32, i32, p, p]
    lib.kgw_moe_rows.restype = i64
    lib.kgw_moe_rows.argtypes = [i64, i32, i32, i32]
    lib.kgw_moe_sort_workspace_bytes.restype = sz
    lib.kgw_moe_sort_workspace_bytes.argtypes = [i64, i32, i32]
    lib.kgw_moe_sort.restype = ctypes.c_int
    lib.kgw_moe_sort.argtypes = [p, i32, i64, i32, i32, i32, i64, p, p, p, p, p, sz, p]
    lib.kgw_moe_permute.restype = ctypes.c_int
    lib.kgw_moe_permute.argtypes = [p, i64, i32, p, p, i64, i32, i64, i64, p, p]
    lib.kgw_moe_unpermute.restype = ctypes.c_int
    lib.kgw_moe_unpermute.argtypes = [p, i64, i32, p, p, i64, i32, i64, i64, p, p]
    lib.kgw_moe_unpermute_grad.restype = ctypes.c_int
    lib.kgw_moe_unpermute_grad.argtypes = [p, i64, p, i64, i32, p, p, p, i64, i32, i64, i64, p, p, p]
    lib.kgw_newton_schulz.restype = ctypes.c_int
    lib.kgw_newton_schulz.argtypes = [p, i64, i64, i32, i32, i64, i64, i32, ctypes.POINTER(ctypes.c_float),
                                      ctypes.c_float, p, i32, p, sz, p]
    lib.kgw_newton_schulz_workspace_bytes.restype = sz
    lib.kgw_newton_schulz_workspace_bytes.argtypes = [i32, i64, i64, i32]
    f32 = ctypes.c_float
    lib.kgw_wgrad_fp8_rows.restype = ctypes.c_int
    lib.kgw_wgrad_fp8_rows.argtypes = [p, p, p, p, p, i32, i64, i64, i64, p, p, i32, i32, p, sz, p]
    lib.kgw_wgrad_fp8_rows_workspace_bytes.restype = sz
    lib.kgw_wgrad_fp8_rows_workspace_bytes.argtypes = [i32, i64, i64, i64]
    lib.kgw_moe_route_workspace_bytes.restype = sz
    lib.kgw_moe_route_workspace_bytes.argtypes = [i64, i32, i32]
    lib.kgw_moe_route.restype = ctypes.c_int
    lib.kgw_moe_route.argtypes = [p, i64, i32, p, p, i32, i64, i32, i32, i32, i32, f32, p, p, p, p, p, p, sz, p]
    lib.kgw_moe_route_grad.restype = ctypes.c_int
    lib.kgw_moe_route_grad.argtypes = [p, i64, i32, p, p, i32, p, p, p, i64, i32, i32, i32, i32, f32, p, p]
    lib.kgw_moe_act_fp8.restype = ctypes.c_int
    lib.kgw_moe_act_fp8.argtypes = [p, i64, i32, i32, p, i32, i64, i64, p, p, p, p, p]
    lib.kgw_moe_act_fp8_grad.restype = ctypes.c_int
    lib.kgw_moe_act_fp8_grad.argtypes = [p, i64, i32, i32, p, p, p, i32, i64, i64, p, p, p, p, p]
    lib.kgw_status_string.restype = ctypes.c_char_p
    lib.kgw_status_string.argtypes = [ctypes.c_int]
    lib.kgw_device_info.restype = ctypes.c_int
    lib.kgw_device_info.argtypes = [ctypes.POINTER(i32), ctypes.POINTER(i32), ctypes.POINTER(i32)]
    _lib = lib
    return lib


def kgw_status_string(status: int) -> str:
    return load_library().kgw_status_string(int(status)).decode()


def _check(status: int, what: str):
    if status == KGW_SUCCESS:
        return
    msg = f"{what}: {kgw_status_string(status)} (status {status})"
    if status == KGW_ERROR_DEVICE:
        raise RuntimeError(msg)
    raise ValueError(msg)


def _stream_ptr(stream) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return int(s.cuda_stream)


def _workspace(E: int, hidden: int, n: int, T: int, fp8: bool, device, stream, split_k: bool):
    """Device workspace for the call (None when it runs in one pass or split_k is False)."""
    if not split_k:
        return None, 0
    nbytes = kgw_workspace_bytes(E, hidden, n, T, fp8)
    if nbytes == 0:
        return None, 0
    return _empty(nbytes, torch.uint8, device, stream), nbytes


def _empty(shape, dtype: torch.dtype, device, stream) -> torch.Tensor:
    """Memory that a call on `stream` (None: the current one) writes first.

    It has to be that stream's: a block that the allocator hands out for the current stream may
    still be in use by work queued there, which `stream` does not wait for.
    """
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    caller = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(caller)        # whose work uses the result next
    return t


def _used_on(stream, *tensors: Optional[torch.Tensor]):
    """Keeps the caller's tensors alive for the pending work of the launch stream."""
    if stream is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else int(t.data_ptr())


_OUT_CODES = {torch.float32: KGW_OUT_FP32, torch.bfloat16: KGW_OUT_BF16, torch.float16: KGW_OUT_FP16}


def _out_code(dtype: torch.dtype) -> int:
    code = _OUT_CODES.get(dtype)
    if code is None:
        raise ValueError(f"output dtype must be float32, bfloat16 or float16, got {dtype}")
    return code


def _prepare_out(out, E, hidden, n, out_dtype, accumulate, device, stream):
    if out is None:
        if accumulate:
            raise ValueError("accumulate=True needs an initialised `out`")
        return _empty((E, hidden, n), out_dtype, device, stream)
    if tuple(out.shape) != (E, hidden, n):
        raise ValueError(f"out must have shape {(E, hidden, n)}, got {tuple(out.shape)}")
    if not out.is_contiguous() or out.device != device:
        raise ValueError("out must be a contiguous tensor on the operands' device")
    return out


def _prepare_outs(outs, E, hidden, n, out_dtype, device, stream):
    """Per-expert outputs -> (list, device int64 array of their addresses, 0 for None)."""
    outs = list(outs)
    if len(outs) != E:
        raise ValueError(f"need one output (or None) per expert: {E}, got {len(outs)}")
    for t in outs:
        if t is None:
            continue
        if tuple(t.shape) != (hidden, n) or t.dtype != out_dtype or t.device != device or not t.is_contiguous():
            raise ValueError(f"each output must be a contiguous {(hidden, n)} {out_dtype} tensor on {device}")
    addrs = torch.tensor([0 if t is None else int(t.data_ptr()) for t in outs], dtype=torch.int64)
    s = torch.cuda.current_stream(device) if stream is None else stream
    with torch.cuda.stream(s):
        ptrs = addrs.to(device)
    ptrs.record_stream(s)
    return outs, ptrs


def _check_offsets(offsets: torch.Tensor, device):
    if offsets.dtype != torch.int32 or offsets.dim() != 1 or not offsets.is_contiguous():
        raise ValueError("offsets must be a contiguous 1-D int32 tensor")
    if offsets.device != device:
        raise ValueError("offsets must live on the operands' device")
    if offsets.numel() < 1:
        raise ValueError("need at least one expert")


def kgw_wgrad_bf16(A: torch.Tensor, B: torch.Tensor, offsets: torch.Tensor, out: Optional[torch.Tensor] = None,
                   *, out_dtype: torch.dtype = torch.float32, accumulate: bool = False, validate: bool = False,
                   stream=None, split_k: bool = True) -> torch.Tensor:
    """bf16 A (hidden, tokens_sum) token-contiguous, B (tokens_sum, n) row-major -> out (E, hidden, n).

    validate=True first checks the offsets on the host (one synchronising copy).  The
    workspace kgw_workspace_bytes asks for is allocated here; split_k=False passes none
    (one pass).
    """
    if A.dtype != torch.bfloat16 or B.dtype != torch.bfloat16:
        raise ValueError("kgw_wgrad_bf16 takes bfloat16 A and B")
    if A.dim() != 2 or B.dim() != 2 or A.shape[1] != B.shape[0]:
        raise ValueError(f"shape mismatch: A {tuple(A.shape)}, B {tuple(B.shape)}")
    if not (A.is_contiguous() and B.is_contiguous()):
        raise ValueError("A and B must be contiguous (A token-contiguous, B row-major)")
    device = A.device
    if B.device != device:
        raise ValueError("A and B must be on the same device")
    _check_offsets(offsets, device)
    hidden, T = A.shape
    n = B.shape[1]
    E = offsets.numel()
    if out is not None:
        out_dtype = out.dtype
    code = _out_code(out_dtype)
    out = _prepare_out(out, E, hidden, n, out_dtype, accumulate, device, stream)
    if validate:
        kgw_validate_offsets(offsets, T, BF16_TOKEN_ALIGN, stream=stream)
    ws, ws_bytes = _workspace(E, hidden, n, T, False, device, stream, split_k)
    _used_on(stream, A, B, offsets, out)
    st = load_library().kgw_wgrad_bf16(_ptr(A), _ptr(B), _ptr(offsets), E, hidden, n, T, _ptr(out), code,
                                       int(bool(accumulate)), _ptr(ws), ws_bytes, _stream_ptr(stream))
    _check(st, "kgw_wgrad_bf16")
    return out


def kgw_wgrad_bf16_noalloc(A: torch.Tensor, B: torch.Tensor, offsets: torch.Tensor, out: torch.Tensor, *,
                           accumulate: bool = False, stream=None) -> torch.Tensor:
    """kgw_wgrad_bf16 that allocates nothing, here or in the library: `out` must be given
    (its dtype selects the output type), and split-K partials use the library's fixed
    per-device scratch.  Calls that overlap in time on one device race on that scratch."""
    if A.dtype != torch.bfloat16 or B.dtype != torch.bfloat16:
        raise ValueError("kgw_wgrad_bf16_noalloc takes bfloat16 A and B")
    if A.dim() != 2 or B.dim() != 2 or A.shape[1] != B.shape[0]:
        raise ValueError(f"shape mismatch: A {tuple(A.shape)}, B {tuple(B.shape)}")
    if not (A.is_contiguous() and B.is_contiguous()):
        raise ValueError("A and B must be contiguous (A token-contiguous, B row-major)")
    if out is None:
        raise ValueError("kgw_wgrad_bf16_noalloc needs `out` (it allocates nothing)")
    device = A.device
    if B.device != device:
        raise ValueError("A and B must be on the same device")
    _check_offsets(offsets, device)
    hidden, T = A.shape
    n = B.shape[1]
    E = offsets.numel()
    code = _out_code(out.dtype)
    out = _prepare_out(out, E, hidden, n, out.dtype, accumulate, device, stream)
    _used_on(stream, A, B, offsets, out)
    st = load_library().kgw_wgrad_bf16_noalloc(_ptr(A), _ptr(B), _ptr(offsets), E, hidden, n, T, _ptr(out), code,
                                               int(bool(accumulate)), _stream_ptr(stream))
    _check(st, "kgw_wgrad_bf16_noalloc")
    return out


def kgw_wgrad_bf16_ex(A: torch.Tensor, B: torch.Tensor, offsets: torch.Tensor, *, a_major: str = "k",
                      b_major: str = "n", ragged: bool = False, hidden: Optional[int] = None,
                      n: Optional[int] = None, out: Optional[torch.Tensor] = None, outs=None,
                      out_dtype: torch.dtype = torch.float32, accumulate: bool = False, validate: bool = False,
                      stream=None, split_k: bool = True):
    """kgw_wgrad_bf16 with a choice of operand layout and output form.

    a_major "k": A is (hidden, tokens_sum) (the default); "m": A is stored (tokens_sum, hidden).
    b_major "n": B is (tokens_sum, n) (the default); "k": B is stored (n, tokens_sum).
    ragged=True (with a_major "k", b_major "k"): A and B hold per-expert blocks (hidden, n_e) and
    (n, n_e) back to back; pass them as flat buffers with `hidden` and `n`.
    `outs` is a list of num_experts (hidden, n) tensors (None skips that expert) whose addresses
    go to the device as the pointer array (returned); otherwise `out` as for kgw_wgrad_bf16.
    """
    if A.dtype != torch.bfloat16 or B.dtype != torch.bfloat16:
        raise ValueError("kgw_wgrad_bf16_ex takes bfloat16 A and B")
    if a_major not in ("k", "m") or b_major not in ("n", "k"):
        raise ValueError("a_major is 'k' or 'm', b_major is 'n' or 'k'")
    if not (A.is_contiguous() and B.is_contiguous()):
        raise ValueError("A and B must be contiguous in their declared layout")
    layout = (KGW_A_M_MAJOR if a_major == "m" else 0) | (KGW_B_K_MAJOR if b_major == "k" else 0)
    if ragged:
        if a_major != "k" or b_major != "k":
            raise ValueError("ragged input needs K-major A and B (a_major='k', b_major='k')")
        if hidden is None or n is None or hidden <= 0 or n <= 0 or A.numel() % hidden:
            raise ValueError("ragged input needs hidden and n, and A.numel() a multiple of hidden")
        layout |= KGW_RAGGED
        T = A.numel() // hidden
        if B.numel() != T * n:
            raise ValueError(f"B must hold tokens_sum * n = {T * n} elements")
    else:
        if A.dim() != 2 or B.dim() != 2:
            raise ValueError("A and B must be 2-D")
        hidden, T = A.shape if a_major == "k" else (A.shape[1], A.shape[0])
        Tb, n = B.shape if b_major == "n" else (B.shape[1], B.shape[0])
        if Tb != T:
            raise ValueError(f"shape mismatch: A {tuple(A.shape)} ({a_major}-major), B {tuple(B.shape)} ({b_major}-major)")
    device = A.device
    if B.device != device:
        raise ValueError("A and B must be on the same device")
    _check_offsets(offsets, device)
    E = offsets.numel()
    out, outs, ptrs, code = _outputs(out, outs, E, hidden, n, out_dtype, accumulate, device, stream)
    if validate:
        kgw_validate_offsets(offsets, T, BF16_TOKEN_ALIGN, stream=stream)
    ws, ws_bytes = _workspace(E, hidden, n, T, False, device, stream, split_k)
    _used_on(stream, A, B, offsets, out, *(outs or ()))
    st = load_library().kgw_wgrad_bf16_ex(_ptr(A), _ptr(B), layout, _ptr(offsets), E, hidden, n, T, _ptr(out),
                                          _ptr(ptrs), code, int(bool(accumulate)), _ptr(ws), ws_bytes,
                                          _stream_ptr(stream))
    _check(st, "kgw_wgrad_bf16_ex")
    return out if outs is None else outs


def _outputs(out, outs, E, hidden, n, out_dtype, accumulate, device, stream):
    """Resolve the dense / discrete output forms: (out, outs, pointer array, dtype code)."""
    if out is not None and outs is not None:
        raise ValueError("pass either out or outs, not both")
    if outs is not None:
        outs = list(outs)
        given = [t for t in outs if t is not None]
        if given:
            out_dtype = given[0].dtype
        code = _out_code(out_dtype)
        outs, ptrs = _prepare_outs(outs, E, hidden, n, out_dtype, device, stream)
        return None, outs, ptrs, code
    if out is not None:
        out_dtype = out.dtype
    code = _out_code(out_dtype)
    return _prepare_out(out, E, hidden, n, out_dtype, accumulate, device, stream), None, None, code


def kgw_wgrad_fp8(A: torch.Tensor, sfa: torch.Tensor, B: torch.Tensor, sfb: torch.Tensor, offsets: torch.Tensor,
                  out: Optional[torch.Tensor] = None, *, out_dtype: torch.dtype = torch.bfloat16,
                  accumulate: bool = False, validate: bool = False, stream=None, split_k: bool = True) -> torch.Tensor:
    """e4m3 A (hidden, T) with UE8M0 sfa (T/128, hidden); e4m3 B (T, n) with sfb (T/128, n)."""
    return _fp8_call("kgw_wgrad_fp8", A, sfa, B, sfb, offsets, out, out_dtype, accumulate, validate, stream,
                     split_k)


def kgw_wgrad_fp8_native(A: torch.Tensor, sfa: torch.Tensor, B: torch.Tensor, sfb: torch.Tensor,
                         offsets: torch.Tensor, out: Optional[torch.Tensor] = None, *,
                         out_dtype: torch.dtype = torch.bfloat16, accumulate: bool = False, validate: bool = False,
                         stream=None, split_k: bool = True) -> torch.Tensor:
    """kgw_wgrad_fp8 on the native scaled fp8 MFMA (faster, ~13-bit in-group alignment; see include/kgw.h)."""
    return _fp8_call("kgw_wgrad_fp8_native", A, sfa, B, sfb, offsets, out, out_dtype, accumulate, validate,
                     stream, split_k)


def kgw_wgrad_fp8_ex(A: torch.Tensor, sfa: torch.Tensor, B: torch.Tensor, sfb: torch.Tensor,
                     offsets: torch.Tensor, *, scale_format: int = KGW_SCALES_U8, native: bool = False,
                     a_major: str = "k", b_major: str = "n", ragged: bool = False, hidden: Optional[int] = None,
                     n: Optional[int] = None, out: Optional[torch.Tensor] = None, outs=None,
                     out_dtype: torch.dtype = torch.bfloat16, accumulate: bool = False, validate: bool = False,
                     stream=None, split_k: bool = True):
    """fp8 product with a scale layout (KGW_SCALES_*: uint8 per 128 tokens, packed int32 words of
    four 128-token blocks, or packed words of four 32-token blocks) and a dense `out` or discrete
    `outs` (see kgw_wgrad_bf16_ex); native=True uses the scaled fp8 MFMA.  Operand layouts as for
    kgw_wgrad_bf16_ex: a_major "k" (A is (hidden, T), the default) or "m" (A stored (T, hidden));
    b_major "n" (B is (T, n), the default) or "k" (B stored (n, T)); ragged=True (with a_major
    "k", b_major "k"): per-expert K-contiguous blocks back to back, passed as flat buffers with
    `hidden` and `n`.  Layouts other than the default take the exact path with uint8 scales;
    the scales keep their (T/128, mn) shapes."""
    if a_major not in ("k", "m") or b_major not in ("n", "k"):
        raise ValueError("a_major is 'k' or 'm', b_major is 'n' or 'k'")
    if ragged and (a_major != "k" or b_major != "k"):
        raise ValueError("ragged input needs K-major A and B (a_major='k', b_major='k')")
    return _fp8_call("kgw_wgrad_fp8_ex", A, sfa, B, sfb, offsets, out, out_dtype, accumulate, validate, stream,
                     split_k, scale_format=scale_format, native=native, outs=outs, a_m_major=a_major == "m",
                     b_k_major=b_major == "k", ragged_dims=(hidden, n) if ragged else None)


def kgw_wgrad_fp4(A: torch.Tensor, sfa: torch.Tensor, B: torch.Tensor, sfb: torch.Tensor, offsets: torch.Tensor,
                  *, out: Optional[torch.Tensor] = None, outs=None, out_dtype: torch.dtype = torch.bfloat16,
                  accumulate: bool = False, validate: bool = False, stream=None, split_k: bool = True):
    """FP4 (e2m1) operands, both token-contiguous and packed two tokens per byte: A (hidden, T/2)
    and B (n, T/2) uint8; scales one UE8M0 per 32 tokens, packed: sfa (T/128, hidden) and
    sfb (T/128, n) int32 (KGW_SCALES_PACKED_32)."""
    if A.dtype != torch.uint8 or B.dtype != torch.uint8 or A.dim() != 2 or B.dim() != 2:
        raise ValueError("kgw_wgrad_fp4 takes packed e2m1 bytes: A (hidden, T/2), B (n, T/2) uint8")
    if A.shape[1] != B.shape[1]:
        raise ValueError(f"A {tuple(A.shape)} and B {tuple(B.shape)} must hold the same token count")
    hidden, T = A.shape[0], 2 * A.shape[1]
    n = B.shape[0]
    (sa_shape, sdtype), (sb_shape, _) = (scale_shape(T, hidden, KGW_SCALES_PACKED_32),
                                         scale_shape(T, n, KGW_SCALES_PACKED_32))
    if sfa.dtype != sdtype or sfb.dtype != sdtype or tuple(sfa.shape) != sa_shape or tuple(sfb.shape) != sb_shape:
        raise ValueError(f"scales must be int32 {sa_shape} and {sb_shape}")
    for t in (A, B, sfa, sfb):
        if not t.is_contiguous():
            raise ValueError("fp4 operands and scales must be contiguous")
    device = A.device
    if any(t.device != device for t in (B, sfa, sfb)):
        raise ValueError("operands and scales must be on the same device")
    _check_offsets(offsets, device)
    E = offsets.numel()
    out, outs, ptrs, code = _outputs(out, outs, E, hidden, n, out_dtype, accumulate, device, stream)
    if validate:
        kgw_validate_offsets(offsets, T, FP4_TOKEN_ALIGN, stream=stream)
    ws, ws_bytes = _workspace(E, hidden, n, T, True, device, stream, split_k)
    _used_on(stream, A, sfa, B, sfb, offsets, out, *(outs or ()))
    st = load_library().kgw_wgrad_fp4(_ptr(A), _ptr(sfa), _ptr(B), _ptr(sfb), _ptr(offsets), E, hidden, n, T,
                                      _ptr(out), _ptr(ptrs), code, int(bool(accumulate)), _ptr(ws), ws_bytes,
                                      _stream_ptr(stream))
    _check(st, "kgw_wgrad_fp4")
    return out if outs is None else outs


def scale_shape(tokens: int, mn: int, scale_format: int) -> Tuple[Tuple[int, int], torch.dtype]:
    """Shape and dtype of the scale tensor of an operand with `tokens` tokens and mn other extent."""
    if scale_format == KGW_SCALES_U8:
        return (tokens // FP8_TOKEN_ALIGN, mn), torch.uint8
    if scale_format == KGW_SCALES_PACKED:
        return ((tokens // FP8_TOKEN_ALIGN + 3) // 4, mn), torch.int32
    if scale_format == KGW_SCALES_PACKED_32:
        return (tokens // FP8_TOKEN_ALIGN, mn), torch.int32
    raise ValueError(f"unknown scale_format {scale_format}")


def _fp8_call(name, A, sfa, B, sfb, offsets, out, out_dtype, accumulate, validate, stream, split_k,
              scale_format=KGW_SCALES_U8, native=None, outs=None, a_m_major=False, b_k_major=False,
              ragged_dims=None):
    fp8_types = (torch.uint8, torch.float8_e4m3fn)
    if A.dtype not in fp8_types or B.dtype not in fp8_types:
        raise ValueError(f"{name} takes e4m3fn (or raw uint8) A and B")
    if sfa is None or sfb is None:
        raise ValueError(f"{name} needs both scale tensors sfa and sfb")
    if ragged_dims is not None:
        hidden, n = ragged_dims
        if hidden is None or n is None or hidden <= 0 or n <= 0 or A.numel() % hidden:
            raise ValueError("ragged input needs hidden and n, and A.numel() a multiple of hidden")
        T = A.numel() // hidden
        if B.numel() != T * n:
            raise ValueError(f"B must hold tokens_sum * n = {T * n} elements")
    else:
        if A.dim() != 2 or B.dim() != 2:
            raise ValueError("A and B must be 2-D")
        hidden, T = (A.shape[1], A.shape[0]) if a_m_major else (A.shape[0], A.shape[1])
        Tb, n = (B.shape[1], B.shape[0]) if b_k_major else (B.shape[0], B.shape[1])
        if Tb != T:
            raise ValueError(f"shape mismatch: A {tuple(A.shape)}{' (stored (T, hidden))' if a_m_major else ''}, "
                             f"B {tuple(B.shape)}{' (stored (n, T))' if b_k_major else ''}")
    (sa_shape, sdtype), (sb_shape, _) = scale_shape(T, hidden, scale_format), scale_shape(T, n, scale_format)
    if sfa.dtype != sdtype or sfb.dtype != sdtype:
        raise ValueError(f"this scale format takes {sdtype} scale tensors")
    if tuple(sfa.shape) != sa_shape or tuple(sfb.shape) != sb_shape:
        raise ValueError(f"scale shapes must be {sa_shape} and {sb_shape}")
    for t in (A, B, sfa, sfb):
        if not t.is_contiguous():
            raise ValueError("fp8 operands and scales must be contiguous")
    device = A.device
    if any(t.device != device for t in (B, sfa, sfb)):
        raise ValueError("operands and scales must be on the same device")
    _check_offsets(offsets, device)
    E = offsets.numel()
    out, outs, ptrs, code = _outputs(out, outs, E, hidden, n, out_dtype, accumulate, device, stream)
    if validate:
        kgw_validate_offsets(offsets, T, FP8_TOKEN_ALIGN, stream=stream)
    fn = getattr(load_library(), name)
    ws, ws_bytes = _workspace(E, hidden, n, T, True, device, stream, split_k)
    _used_on(stream, A, sfa, B, sfb, offsets, out, *(outs or ()))
    if native is None:
        st = fn(_ptr(A), _ptr(sfa), _ptr(B), _ptr(sfb), _ptr(offsets), E, hidden, n, T, _ptr(out), code,
                int(bool(accumulate)), _ptr(ws), ws_bytes, _stream_ptr(stream))
    else:
        st = fn(_ptr(A), _ptr(sfa), _ptr(B), _ptr(sfb), int(scale_format), int(bool(native)),
                (KGW_A_M_MAJOR if a_m_major else 0) | (KGW_B_K_MAJOR if b_k_major else 0) |
                (KGW_RAGGED if ragged_dims is not None else 0), _ptr(offsets), E,
                hidden, n, T, _ptr(out), _ptr(ptrs), code,
                int(bool(accumulate)), _ptr(ws), ws_bytes, _stream_ptr(stream))
    _check(st, name)
    return out if outs is None else outs


def kgw_wgrad_fp8_rows(A: torch.Tensor, sa: torch.Tensor, B: torch.Tensor, offsets: torch.Tensor, *,
                       sb: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, outs=None,
                       out_dtype: torch.dtype = torch.float32, accumulate: bool = False, validate: bool = False,
                       stream=None, split_k: bool = True):
    """Weight gradients from 8-bit token rows, scaled along the rows as the forward products take them:
    e4m3 A (T, hidden) with UE8M0 sa (ceil(hidden/128), T), and B (T, n) bf16, or e4m3 with sb
    (ceil(n/128), T).  Counts are multiples of 128; exact products, fp32 sums; outputs as for kgw_wgrad_bf16_ex."""
    fp8_types = (torch.uint8, torch.float8_e4m3fn)
    if A.dtype not in fp8_types or B.dtype not in (fp8_types if sb is not None else (torch.bfloat16,)):
        raise ValueError("kgw_wgrad_fp8_rows takes e4m3fn (or raw uint8) A, and B bfloat16 without or e4m3fn with sb")
    if A.dim() != 2 or B.dim() != 2 or A.shape[0] != B.shape[0]:
        raise ValueError(f"A must be (T, hidden) and B (T, n), got {tuple(A.shape)} and {tuple(B.shape)}")
    T, hidden = A.shape
    n = B.shape[1]
    device = _on_gpu(A, "A")
    for s, cols, what in ((sa, hidden, "sa"), (sb, n, "sb")):
        if s is None and what == "sb":
            continue
        shape = (-(-cols // FP8_TOKEN_ALIGN), T)
        if s is None or s.dtype != torch.uint8 or tuple(s.shape) != shape or not s.is_contiguous() or s.device != device:
            raise ValueError(f"{what} must be a contiguous uint8 {shape} tensor on the operands' device")
    if not (A.is_contiguous() and B.is_contiguous()) or B.device != device:
        raise ValueError("A and B must be contiguous, on the same device")
    _check_offsets(offsets, device)
    E = offsets.numel()
    out, outs, ptrs, code = _outputs(out, outs, E, hidden, n, out_dtype, accumulate, device, stream)
    if validate:
        kgw_validate_offsets(offsets, T, FP8_TOKEN_ALIGN, stream=stream)
    lib = load_library()
    ws_bytes = lib.kgw_wgrad_fp8_rows_workspace_bytes(E, hidden, n, T) if split_k else 0
    ws = _empty(ws_bytes, torch.uint8, device, stream) if ws_bytes else None
    if stream is not None:
        _used_on(stream, A, sa, B, sb, offsets, out, *(outs or ()))
    st = lib.kgw_wgrad_fp8_rows(_ptr(A), _ptr(sa), _ptr(B), _ptr(sb), _ptr(offsets), E, hidden, n, T, _ptr(out), _ptr(ptrs),
                                code, int(bool(accumulate)), _ptr(ws), ws_bytes, _launch_stream(stream, device))
    _check(st, "kgw_wgrad_fp8_rows")
    return out if outs is None else outs


def kgw_quantize_fp8(x: torch.Tensor, token_axis: int, stream=None,
                     scale_format: int = KGW_SCALES_U8) -> Tuple[torch.Tensor, torch.Tensor]:
    """bf16 x (rows, cols) -> (e4m3fn bytes as uint8 (rows, cols), UE8M0 scales in `scale_format`).

    token_axis 1: tokens along the columns (A (hidden, tokens)), scales with mn = rows;
    token_axis 0: tokens along the rows (B (tokens, n)), scales with mn = cols.  See
    scale_shape for the scale tensor of each format.
    """
    if x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_contiguous():
        raise ValueError("kgw_quantize_fp8 takes a contiguous 2-D bfloat16 tensor")
    if token_axis not in (0, 1):
        raise ValueError("token_axis must be 0 or 1")
    rows, cols = x.shape
    tokens, other = (cols, rows) if token_axis else (rows, cols)
    if tokens % FP8_TOKEN_ALIGN != 0:
        raise ValueError(f"the token length ({tokens}) must be a multiple of {FP8_TOKEN_ALIGN}")
    shape, sdtype = scale_shape(tokens, other, scale_format)
    q = _empty((rows, cols), torch.uint8, x.device, stream)
    s = _empty(shape, sdtype, x.device, stream)
    _used_on(stream, x)
    st = load_library().kgw_quantize_fp8(_ptr(x), rows, cols, int(token_axis), int(scale_format), _ptr(q), _ptr(s),
                                         _stream_ptr(stream))
    _check(st, "kgw_quantize_fp8")
    return q, s


def kgw_quantize_fp4(x: torch.Tensor, token_axis: int, stream=None,
                     scale_format: int = KGW_SCALES_PACKED_32) -> Tuple[torch.Tensor, torch.Tensor]:
    """bf16 x (rows, cols) -> (packed e2m1 bytes, UE8M0 scales per 32 tokens), the operands of
    kgw_wgrad_fp4.

    token_axis 1: tokens along the columns (A (hidden, tokens)): codes (rows, cols/2), scales
    with mn = rows; token_axis 0: tokens along the rows (B (tokens, n)): codes (cols, rows/2)
    (token-contiguous), scales with mn = cols.  scale_format KGW_SCALES_PACKED_32 (int32
    (tokens/128, mn), what kgw_wgrad_fp4 takes) or KGW_SCALES_U8 (uint8 (tokens/32, mn)).
    """
    if x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_contiguous():
        raise ValueError("kgw_quantize_fp4 takes a contiguous 2-D bfloat16 tensor")
    if token_axis not in (0, 1):
        raise ValueError("token_axis must be 0 or 1")
    if scale_format not in (KGW_SCALES_U8, KGW_SCALES_PACKED_32):
        raise ValueError("FP4 scales are KGW_SCALES_U8 or KGW_SCALES_PACKED_32")
    rows, cols = x.shape
    tokens, other = (cols, rows) if token_axis else (rows, cols)
    if tokens % 128 != 0:
        raise ValueError(f"the token length ({tokens}) must be a multiple of 128")
    if scale_format == KGW_SCALES_U8:
        shape, sdtype = (tokens // 32, other), torch.uint8
    else:
        shape, sdtype = scale_shape(tokens, other, scale_format)
    q = _empty((other, tokens // 2), torch.uint8, x.device, stream)
    s = _empty(shape, sdtype, x.device, stream)
    _used_on(stream, x)
    st = load_library().kgw_quantize_fp4(_ptr(x), rows, cols, int(token_axis), int(scale_format), _ptr(q), _ptr(s),
                                         _stream_ptr(stream))
    _check(st, "kgw_quantize_fp4")
    return q, s


def kgw_mgrouped_bf16(A: torch.Tensor, W: torch.Tensor, *, offsets: Optional[torch.Tensor] = None,
                      m_indices: Optional[torch.Tensor] = None, layout: str = "nt",
                      out: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                      accumulate: bool = False, stream=None) -> torch.Tensor:
    """m-grouped product: out[r] = A[r] @ W[g(r)]^T ("nt", W (E, N, K), the forward) or
    A[r] @ W[g(r)] ("nn", W (E, K, N), dgrad); groups from `offsets` (inclusive cumulative
    rows) or per-row `m_indices`; rows of no group are left untouched."""
    if A.dtype != torch.bfloat16 or W.dtype != torch.bfloat16:
        raise ValueError("kgw_mgrouped_bf16 takes bfloat16 A and W")
    if A.dim() != 2 or W.dim() != 3 or not A.is_contiguous() or not W.is_contiguous():
        raise ValueError("A must be a contiguous (M, K) and W a contiguous (E, ., .) tensor")
    if layout not in ("nt", "nn"):
        raise ValueError("layout is 'nt' (forward) or 'nn' (dgrad)")
    M, K = A.shape
    E = W.shape[0]
    N = W.shape[1] if layout == "nt" else W.shape[2]
    if (W.shape[2] if layout == "nt" else W.shape[1]) != K:
        raise ValueError(f"W {tuple(W.shape)} does not match A's K = {K} for layout {layout}")
    device = A.device
    if W.device != device:
        raise ValueError("A and W must be on the same device")
    if (offsets is None) == (m_indices is None):
        raise ValueError("pass exactly one of offsets and m_indices")
    idx = offsets if offsets is not None else m_indices
    if idx.dtype != torch.int32 or idx.dim() != 1 or not idx.is_contiguous() or idx.device != device:
        raise ValueError("offsets / m_indices must be a contiguous 1-D int32 tensor on the operands' device")
    if offsets is not None and offsets.numel() != E:
        raise ValueError(f"offsets must have one entry per group ({E})")
    if m_indices is not None and m_indices.numel() != M:
        raise ValueError(f"m_indices must have one entry per row ({M})")
    if out is not None:
        out_dtype = out.dtype
    code = _out_code(out_dtype)
    if out is None:
        if accumulate:
            raise ValueError("accumulate=True needs an initialised `out`")
        out = _empty((M, N), out_dtype, device, stream)
    elif tuple(out.shape) != (M, N) or not out.is_contiguous() or out.device != device:
        raise ValueError(f"out must be a contiguous {(M, N)} tensor on the operands' device")
    _used_on(stream, A, W, idx, out)
    st = load_library().kgw_mgrouped_bf16(_ptr(A), _ptr(W), KGW_LAYOUT_NT if layout == "nt" else KGW_LAYOUT_NN,
                                          _ptr(offsets), _ptr(m_indices), E, M, K, N, _ptr(out), code,
                                          int(bool(accumulate)), _stream_ptr(stream))
    _check(st, "kgw_mgrouped_bf16")
    return out


def kgw_mgrouped_fp8(A: torch.Tensor, sa: torch.Tensor, W: torch.Tensor, sw: torch.Tensor, *,
                     offsets: Optional[torch.Tensor] = None, m_indices: Optional[torch.Tensor] = None,
                     layout: str = "nt", out: Optional[torch.Tensor] = None,
                     out_dtype: torch.dtype = torch.bfloat16, accumulate: bool = False, stream=None) -> torch.Tensor:
    """m-grouped product with fp8 operands: A is e4m3 (M, K) with UE8M0 sa (K/128, M); W is e4m3
    (E, N, K) for layout "nt" (forward, out[r] = a(r) @ w(g(r))^T) or (E, K, N) for "nn" (dgrad,
    out[r] = a(r) @ w(g(r))), with UE8M0 sw (E, K/128, N) either way, one scale per 1x128 block
    along K; groups from `offsets` or `m_indices` as for kgw_mgrouped_bf16; rows of no group
    are left untouched."""
    fp8_types = (torch.uint8, torch.float8_e4m3fn)
    if A.dtype not in fp8_types or W.dtype not in fp8_types:
        raise ValueError("kgw_mgrouped_fp8 takes e4m3fn (or raw uint8) A and W")
    if sa is None or sw is None or sa.dtype != torch.uint8 or sw.dtype != torch.uint8:
        raise ValueError("kgw_mgrouped_fp8 needs uint8 scale tensors sa and sw")
    if A.dim() != 2 or W.dim() != 3:
        raise ValueError("A must be (M, K) and W (E, N, K)")
    for t in (A, W, sa, sw):
        if not t.is_contiguous():
            raise ValueError("fp8 operands and scales must be contiguous")
    if layout not in ("nt", "nn"):
        raise ValueError("layout is 'nt' (forward) or 'nn' (dgrad)")
    M, K = A.shape
    E = W.shape[0]
    N = W.shape[1] if layout == "nt" else W.shape[2]
    if (W.shape[2] if layout == "nt" else W.shape[1]) != K:
        raise ValueError(f"W {tuple(W.shape)} does not match A's K = {K} for layout {layout}")
    if K % FP8_TOKEN_ALIGN != 0:
        raise ValueError(f"K ({K}) must be a multiple of {FP8_TOKEN_ALIGN}")
    if tuple(sa.shape) != (K // FP8_TOKEN_ALIGN, M) or tuple(sw.shape) != (E, K // FP8_TOKEN_ALIGN, N):
        raise ValueError(f"scale shapes must be {(K // FP8_TOKEN_ALIGN, M)} and {(E, K // FP8_TOKEN_ALIGN, N)}")
    device = A.device
    if any(t.device != device for t in (W, sa, sw)):
        raise ValueError("operands and scales must be on the same device")
    if (offsets is None) == (m_indices is None):
        raise ValueError("pass exactly one of offsets and m_indices")
    idx = offsets if offsets is not None else m_indices
    if idx.dtype != torch.int32 or idx.dim() != 1 or not idx.is_contiguous() or idx.device != device:
        raise ValueError("offsets / m_indices must be a contiguous 1-D int32 tensor on the operands' device")
    if offsets is not None and offsets.numel() != E:
        raise ValueError(f"offsets must have one entry per group ({E})")
    if m_indices is not None and m_indices.numel() != M:
        raise ValueError(f"m_indices must have one entry per row ({M})")
    if out is not None:
        out_dtype = out.dtype
    code = _out_code(out_dtype)
    if out is None:
        if accumulate:
            raise ValueError("accumulate=True needs an initialised `out`")
        out = _empty((M, N), out_dtype, device, stream)
    elif tuple(out.shape) != (M, N) or not out.is_contiguous() or out.device != device:
        raise ValueError(f"out must be a contiguous {(M, N)} tensor on the operands' device")
    _used_on(stream, A, sa, W, sw, idx, out)
    st = load_library().kgw_mgrouped_fp8(_ptr(A), _ptr(sa), _ptr(W), _ptr(sw),
                                         KGW_LAYOUT_NT if layout == "nt" else KGW_LAYOUT_NN, _ptr(offsets),
                                         _ptr(m_indices), E, M, K, N, _ptr(out), code, int(bool(accumulate)),
                                         _stream_ptr(stream))
    _check(st, "kgw_mgrouped_fp8")
    return out


def kgw_workspace_bytes(num_experts: int, hidden: int, n: int, tokens_sum: int, fp8: bool = False) -> int:
    return int(load_library().kgw_workspace_bytes(num_experts, hidden, n, tokens_sum, int(bool(fp8))))


def kgw_validate_offsets_host(offsets, tokens_sum: int, alignment: int) -> Tuple[int, int]:
    """Check host offsets (sequence or CPU tensor); returns (status, first bad expert or -1)."""
    t = torch.as_tensor(offsets, dtype=torch.int32).contiguous()
    if t.device.type != "cpu":
        raise ValueError("kgw_validate_offsets_host takes host offsets")
    bad = ctypes.c_int32(-1)
    st = load_library().kgw_validate_offsets_host(t.data_ptr(), t.numel(), int(tokens_sum), int(alignment),
                                                  ctypes.byref(bad))
    return int(st), int(bad.value)


def kgw_validate_offsets(offsets: torch.Tensor, tokens_sum: int, alignment: int, stream=None) -> None:
    """Check device offsets (synchronising); raises ValueError naming the first bad expert."""
    bad = ctypes.c_int32(-1)
    st = load_library().kgw_validate_offsets(_ptr(offsets), offsets.numel(), int(tokens_sum), int(alignment),
                                             ctypes.byref(bad), _stream_ptr(stream))
    if st != KGW_SUCCESS:
        _check(st, f"kgw_validate_offsets (first bad expert {bad.value})")


def kgw_check_offsets(offsets: torch.Tensor, tokens_sum: int, alignment: int,
                      result: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Queue the offsets check on the device (no synchronisation): returns a one-element
    int32 device tensor that will hold the first bad expert, or -1 (`result` if given)."""
    if offsets.dtype != torch.int32 or offsets.dim() != 1 or not offsets.is_contiguous():
        raise ValueError("offsets must be a contiguous 1-D int32 tensor")
    if result is None:
        result = _empty(1, torch.int32, offsets.device, stream)
    elif result.dtype != torch.int32 or result.numel() < 1 or result.device != offsets.device:
        raise ValueError("result must be an int32 tensor on the offsets' device")
    _used_on(stream, offsets, result)
    st = load_library().kgw_check_offsets(_ptr(offsets), offsets.numel(), int(tokens_sum), int(alignment),
                                          _ptr(result), _stream_ptr(stream))
    _check(st, "kgw_check_offsets")
    return result


def kgw_mfma_ceiling(src: torch.Tensor, kind: int, iters: int = 20000, workgroups: int = 1024,
                     stream=None) -> Tuple[float, float]:
    """Time MFMA-only loops on the bytes of `src` (kind 0 bf16, 1 e4m3 as bf16, 2 e4m3 on the scaled
    fp8 MFMA, 3 e2m1 pairs on the scaled MFMA's FP4 mode): returns (TFLOP/s from HIP events around the launch, mean clock in GHz the loop ran
    at).  A measurement helper: it synchronises."""
    if not src.is_cuda or not src.is_contiguous():
        raise ValueError("src must be a contiguous device tensor")
    s = torch.cuda.current_stream(src.device) if stream is None else stream
    with torch.cuda.stream(s):
        cycles = torch.zeros(2 * workgroups, dtype=torch.int64, device=src.device)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record(s)
    st = load_library().kgw_mfma_ceiling(_ptr(src), src.numel() * src.element_size(), int(kind), int(iters),
                                         int(workgroups), _ptr(cycles), int(s.cuda_stream))
    end.record(s)
    _check(st, "kgw_mfma_ceiling")
    end.synchronize()
    ms = start.elapsed_time(end)
    c = cycles.view(-1, 2).double().cpu()
    ghz = float((c[:, 0] / c[:, 1]).mean()) * 0.1
    flop_per_mfma = 131072.0 if kind in (2, 3) else 32768.0
    flops = 16.0 * iters * workgroups * 4 * flop_per_mfma
    return flops / (ms * 1e-3) / 1e12, ghz


def kgw_device_info() -> dict:
    cus, g950, xcds = ctypes.c_int32(0), ctypes.c_int32(0), ctypes.c_int32(0)
    _check(load_library().kgw_device_info(ctypes.byref(cus), ctypes.byref(g950), ctypes.byref(xcds)),
           "kgw_device_info")
    return {"num_cus": cus.value, "is_gfx950": bool(g950.value), "num_xcds": xcds.value}


def wgrad(a: torch.Tensor, b: torch.Tensor, offsets: torch.Tensor, *, sfa: Optional[torch.Tensor] = None,
          sfb: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
          out_dtype: Optional[torch.dtype] = None, accumulate: bool = False, check: bool = True) -> torch.Tensor:
    """Dispatch on operand dtype like the cuDNN wrapper: bf16 operands take no scales
    (any scale is a ValueError, section "BF16 contract"); fp8 operands need both.

    check=True (the default, like the cuDNN page's wrapper, which rejects malformed or
    unaligned offsets: section "Scheduling, cache, and errors") validates the offsets first,
    which costs one synchronising copy of them to the host; check=False skips it and the
    kernels clamp malformed ranges instead (see kgw_check_offsets for an asynchronous flag)."""
    if a.dtype == torch.bfloat16 and b.dtype == torch.bfloat16:
        if sfa is not None or sfb is not None:
            raise ValueError("bf16 operands take no scale tensors")
        return kgw_wgrad_bf16(a, b, offsets, out, out_dtype=out_dtype or torch.float32, accumulate=accumulate,
                              validate=check)
    if a.dtype in (torch.float8_e4m3fn, torch.uint8) and b.dtype in (torch.float8_e4m3fn, torch.uint8):
        return kgw_wgrad_fp8(a, sfa, b, sfb, offsets, out, out_dtype=out_dtype or torch.bfloat16,
                             accumulate=accumulate, validate=check)
    raise ValueError(f"unsupported operand dtypes {a.dtype}, {b.dtype}")


# ----------------------------------------------------------------------------
# tokens sorted by expert and back
# ----------------------------------------------------------------------------
_MOE_MAX_EXPERTS = 2048     # of one kgw_moe_sort


def _int32(value: int, what: str) -> int:
    """The C calls' 32-bit arguments: a number that does not fit would be cut to another one."""
    if not -2 ** 31 <= int(value) < 2 ** 31:
        raise ValueError(f"{what} must fit 32 bits, got {value}")
    return int(value)


def kgw_moe_rows(tokens: int, topk: int, num_experts: int, alignment: int = FP8_TOKEN_ALIGN) -> int:
    """Rows that always hold `tokens` tokens of `topk` experts each, every expert's rows padded
    to a multiple of `alignment`."""
    rows = load_library().kgw_moe_rows(int(tokens), _int32(topk, "topk"), _int32(num_experts, "num_experts"),
                                       _int32(alignment, "alignment"))
    if rows < 0:
        raise ValueError(f"no row count for tokens={tokens}, topk={topk}, num_experts={num_experts}, "
                         f"alignment={alignment}")
    return rows


def _on_gpu(t: torch.Tensor, what: str) -> torch.device:
    """The tensor's device: the current GPU, whose memory the kernels address."""
    device = t.device
    if not t.is_cuda:
        raise ValueError(f"{what} must be a GPU tensor, got one on {device}")
    if device.index != torch._C._cuda_getDevice():
        raise ValueError(f"{what} is on {device}, the current device is cuda:{torch.cuda.current_device()}")
    return device


def _launch_stream(stream, device: torch.device) -> int:
    """The stream's handle; without making a Stream object of the current one (3 us of a 12 us call)."""
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None else int(stream.cuda_stream)


def _rows_2d(t: torch.Tensor, what: str) -> int:
    """Row stride of a 2-D tensor with contiguous rows."""
    if t.dim() != 2:
        raise ValueError(f"{what} must be 2-D, got shape {tuple(t.shape)}")
    rows, cols = t.shape
    ld, step = t.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{what} needs contiguous rows (stride 1 along the last axis)")
    if rows <= 1:
        return cols
    if ld < cols:
        raise ValueError(f"{what} has overlapping rows")
    return ld


def _routing(t: torch.Tensor, what: str, dim: int, device):
    if t.dtype != torch.int32 or t.dim() != dim or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dim}-D int32 tensor")
    if t.device != device:
        raise ValueError(f"{what} must live on the rows' device")


def _weights(t: torch.Tensor, row_of: torch.Tensor, what: str = "weights"):
    if t.dtype != torch.float32 or t.shape != row_of.shape or not t.is_contiguous() or t.device != row_of.device:
        raise ValueError(f"{what} must be a contiguous float32 tensor of row_of's shape, on its device")


def _result(out: Optional[torch.Tensor], shape, dtype, device, what: str, stream) -> torch.Tensor:
    if out is None:
        return _empty(shape, dtype, device, stream)
    if out.shape != shape or out.dtype != dtype or out.device != device or not out.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {tuple(shape)} {dtype} tensor on {device}")
    return out


def kgw_moe_sort(ids: torch.Tensor, num_experts: int, *, alignment: int = FP8_TOKEN_ALIGN,
                 rows: Optional[int] = None, stream=None):
    """Sort the assignments ids (tokens, topk), int32 or int64, by expert.

    Returns int32 tensors (counts, offsets, row_of, src_of): counts (num_experts,) and offsets
    (num_experts,) as kgw_wgrad_* and kgw_mgrouped_* take them (every count rounded up to
    `alignment`), row_of (tokens, topk) and src_of (rows,).  An id outside [0, num_experts)
    gets row -1.  `rows` (default: kgw_moe_rows, which always suffices) bounds the sorted rows; the
    assignments past it get row -1.

    The four are views of one buffer: clone() a small one to keep it without the others, and
    write to none in place while autograd holds another.
    """
    if ids.dtype not in (torch.int32, torch.int64) or ids.dim() != 2 or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous 2-D int32 or int64 tensor")
    tokens, topk = ids.shape
    E = int(num_experts)
    if not 1 <= E <= _MOE_MAX_EXPERTS or topk < 1 or not 1 <= alignment < 2 ** 31 or not (rows is None or 0 <= rows < 2 ** 31):
        raise ValueError(f"need 1 .. {_MOE_MAX_EXPERTS} experts, one expert per token, an alignment of 1 or more and "
                         "0 .. 2^31 - 1 rows")
    rows = kgw_moe_rows(tokens, topk, E, alignment) if rows is None else int(rows)
    device = _on_gpu(ids, "ids")
    lib = load_library()
    need = lib.kgw_moe_sort_workspace_bytes(tokens, topk, E)
    # one allocation for all results and the workspace: five would take a third of a short call's time
    n = tokens * topk
    size = rows + n + 2 * E + need // 4
    results = torch.empty(size, dtype=torch.int32, device=device) if stream is None else _empty(size, torch.int32, device, stream)
    src_of, row_of, counts, offsets, _ = results.split((rows, n, E, E, need // 4))
    if stream is not None:
        _used_on(stream, ids)
    at = results.data_ptr()
    counts_at = at + 4 * (rows + n)
    st = lib.kgw_moe_sort(ids.data_ptr(), ids.element_size(), tokens, topk, E, int(alignment), rows, counts_at,
                          counts_at + 4 * E, at + 4 * rows, at, counts_at + 8 * E if need else None, need,
                          _launch_stream(stream, device))
    _check(st, "kgw_moe_sort")
    return counts, offsets, row_of.view(tokens, topk), src_of


def kgw_moe_permute(x: torch.Tensor, row_of: torch.Tensor, src_of: torch.Tensor,
                    out: Optional[torch.Tensor] = None, *, stream=None) -> torch.Tensor:
    """x (tokens, hidden) -> out (rows, hidden): out[row_of[t][j]] = x[t], every other row zero.

    fp32, bf16 or fp16; x may have any row stride that keeps its rows apart.  Gradient: kgw_moe_unpermute without weights.
    """
    code = _out_code(x.dtype)
    ld = _rows_2d(x, "x")
    device = _on_gpu(x, "x")
    _routing(row_of, "row_of", 2, device)
    _routing(src_of, "src_of", 1, device)
    tokens, hidden = x.shape
    if row_of.shape[0] != tokens:
        raise ValueError(f"row_of has {row_of.shape[0]} tokens, x has {tokens}")
    rows = src_of.shape[0]
    out = _result(out, (rows, hidden), x.dtype, device, "out", stream)
    if stream is not None:
        _used_on(stream, x, row_of, src_of, out)
    st = load_library().kgw_moe_permute(x.data_ptr(), ld, code, row_of.data_ptr(), src_of.data_ptr(), tokens,
                                        row_of.shape[1], rows, hidden, out.data_ptr(), _launch_stream(stream, device))
    _check(st, "kgw_moe_permute")
    return out


def kgw_moe_unpermute(y: torch.Tensor, row_of: torch.Tensor, weights: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None, *, stream=None) -> torch.Tensor:
    """y (rows, hidden) -> out (tokens, hidden): out[t] = sum_j weights[t][j] * y[row_of[t][j]].

    weights float32 (tokens, topk), None for all ones (the gradient of kgw_moe_permute).  Summed in
    fp32, rounded once to y's type; an assignment without a row adds nothing.
    """
    code = _out_code(y.dtype)
    ld = _rows_2d(y, "y")
    device = _on_gpu(y, "y")
    _routing(row_of, "row_of", 2, device)
    if weights is not None:
        _weights(weights, row_of)
    rows, hidden = y.shape
    tokens, topk = row_of.shape
    out = _result(out, (tokens, hidden), y.dtype, device, "out", stream)
    if stream is not None:
        _used_on(stream, y, row_of, weights, out)
    st = load_library().kgw_moe_unpermute(y.data_ptr(), ld, code, row_of.data_ptr(), _ptr(weights), tokens, topk,
                                          rows, hidden, out.data_ptr(), _launch_stream(stream, device))
    _check(st, "kgw_moe_unpermute")
    return out


def kgw_moe_unpermute_grad(dout: torch.Tensor, y: torch.Tensor, row_of: torch.Tensor, src_of: torch.Tensor,
                           weights: torch.Tensor, dy: Optional[torch.Tensor] = None,
                           dweights: Optional[torch.Tensor] = None, *, stream=None):
    """Gradients of kgw_moe_unpermute(y, row_of, weights) for dout (tokens, hidden): (dy, dweights).

    dy (rows, hidden) in y's type, zero in every row without a source; dweights float32
    (tokens, topk), zero for an assignment without a row.  (Without weights dy is
    kgw_moe_permute(dout, row_of, src_of).)
    """
    code = _out_code(y.dtype)
    ld_y, ld_d = _rows_2d(y, "y"), _rows_2d(dout, "dout")
    device = _on_gpu(y, "y")
    _routing(row_of, "row_of", 2, device)
    _routing(src_of, "src_of", 1, device)
    _weights(weights, row_of)
    rows, hidden = y.shape
    tokens, topk = row_of.shape
    if dout.dtype != y.dtype or dout.device != device or tuple(dout.shape) != (tokens, hidden):
        raise ValueError(f"dout must be a {(tokens, hidden)} {y.dtype} tensor on {device}")
    if src_of.shape[0] != rows:
        raise ValueError(f"src_of has {src_of.shape[0]} rows, y has {rows}")
    dy = _result(dy, (rows, hidden), y.dtype, device, "dy", stream)
    dweights = _result(dweights, (tokens, topk), torch.float32, device, "dweights", stream)
    if stream is not None:
        _used_on(stream, dout, y, row_of, src_of, weights, dy, dweights)
    st = load_library().kgw_moe_unpermute_grad(dout.data_ptr(), ld_d, y.data_ptr(), ld_y, code, row_of.data_ptr(),
                                               src_of.data_ptr(), weights.data_ptr(), tokens, topk, rows, hidden,
                                               dy.data_ptr(), dweights.data_ptr(), _launch_stream(stream, device))
    _check(st, "kgw_moe_unpermute_grad")
    return dy, dweights


# ----------------------------------------------------------------------------
# the router
# ----------------------------------------------------------------------------
_ROUTE_MAX_TOPK = 64
_SCORES = {"softmax": KGW_SCORE_SOFTMAX, "sigmoid": KGW_SCORE_SIGMOID}


def _route_args(scores: torch.Tensor, topk: int, mask, score: str):
    """Checks what the router and its gradient share: (device, type code, row stride, score code, tokens, experts)."""
    code = _out_code(scores.dtype)
    ld = _rows_2d(scores, "scores")
    device = _on_gpu(scores, "scores")
    tokens, E = scores.shape
    if not 1 <= E <= _MOE_MAX_EXPERTS or not 1 <= topk <= min(E, _ROUTE_MAX_TOPK):
        raise ValueError(f"need 1 .. {_MOE_MAX_EXPERTS} experts and 1 .. min(experts, {_ROUTE_MAX_TOPK}) a token, got {E}, {topk}")
    if mask is not None and (mask.dtype not in (torch.bool, torch.uint8) or mask.shape != (tokens,) or
                             mask.device != device or not mask.is_contiguous()):
        raise ValueError(f"mask must be a contiguous bool ({tokens},) tensor on {device}")
    score_code = _SCORES.get(score)
    if score_code is None:
        raise ValueError(f"score is 'softmax' or 'sigmoid', got {score!r}")
    return device, code, ld, score_code, tokens, E


def _route_ids(ids: torch.Tensor, tokens: int, device):
    if ids.dtype not in (torch.int32, torch.int64) or ids.dim() != 2 or ids.shape[0] != tokens or \
            not ids.is_contiguous() or ids.device != device:
        raise ValueError(f"ids must be a contiguous int32 or int64 ({tokens}, topk) tensor on {device}")


def _floats(t: torch.Tensor, shape, device, what: str):
    if t.dtype != torch.float32 or t.shape != shape or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{what} must be a contiguous float32 {shape} tensor on {device}")


def kgw_moe_route(scores: torch.Tensor, topk: int, *, ids: Optional[torch.Tensor] = None,
                  mask: Optional[torch.Tensor] = None, score: str = "softmax", renormalize: bool = True,
                  scale: float = 1.0, stream=None):
    """Route tokens by their scores (tokens, experts), fp32, bf16 or fp16 with any row stride.

    Returns (ids, weights, counts, loss, slope): int32 ids (tokens, topk) of the largest scores (ties to the lowest
    index), what kgw_moe_sort takes; float32 weights (tokens, topk), what kgw_moe_unpermute takes; int32 counts
    (experts,); the balance loss, a float32 scalar that is 1 where all experts are used alike; and slope (experts,), its
    derivative by every token's shares, for kgw_moe_route_grad.

    Shares are softmax(scores), or sigmoids divided by their sum; weights are the chosen shares (score="sigmoid": the
    sigmoids), divided by their sum if `renormalize`, times `scale`.  A score of -inf is an expert that its token may not
    take, a False in `mask` (tokens,) a token that takes none: id -1, weight 0, no part in the loss.  `ids`
    (int32 or int64, (tokens, topk)) are experts chosen elsewhere.

    Every result has memory of its own.
    """
    topk = int(topk)
    device, code, ld, score_code, tokens, E = _route_args(scores, topk, mask, score)
    if ids is not None:
        _route_ids(ids, tokens, device)
        if ids.shape[1] != topk:
            raise ValueError(f"ids has {ids.shape[1]} experts a token, topk is {topk}")
    lib = load_library()
    need = lib.kgw_moe_route_workspace_bytes(tokens, E, ids is not None)
    workspace = _empty(need, torch.uint8, device, stream) if need else None
    if stream is None:
        results = _route_results(tokens, topk, E, device)
    else:
        _used_on(stream, scores, mask, ids)
        caller = torch.cuda.current_stream(device)
        with torch.cuda.stream(stream):                    # (as _empty)
            results = _route_results(tokens, topk, E, device)
        _used_on(caller, *results)
    chosen, weights, counts, loss, slope = results
    st = lib.kgw_moe_route(scores.data_ptr(), ld, code, _ptr(mask), _ptr(ids), 0 if ids is None else ids.element_size(),
                           tokens, E, topk, score_code, int(bool(renormalize)), scale, chosen.data_ptr(), weights.data_ptr(),
                           counts.data_ptr(), loss.data_ptr(), slope.data_ptr(), _ptr(workspace), need,
                           _launch_stream(stream, device))
    _check(st, "kgw_moe_route")
    return results


def _route_results(tokens: int, topk: int, E: int, device):
    """ids, weights, counts, loss and slope, each in memory of its own: a caller keeps some of them for long, and changes some
    in place that autograd knows.  (Views of one buffer save 0.6 us of a call's 12.5, 2 us of 17 where it has a workspace too,
    and allow neither: whoever keeps one keeps all.)"""
    real, whole = torch.float32, torch.int32
    new = torch.empty_strided                              # (with its strides given an allocation takes 1.3 us, without 1.6)
    return (new((tokens, topk), (topk, 1), dtype=whole, device=device), new((tokens, topk), (topk, 1), dtype=real, device=device),
            new((E,), (1,), dtype=whole, device=device), new((), (), dtype=real, device=device),
            new((E,), (1,), dtype=real, device=device))


def kgw_moe_route_grad(scores: torch.Tensor, ids: torch.Tensor, dweights: Optional[torch.Tensor], *,
                       dloss: Optional[torch.Tensor] = None, slope: Optional[torch.Tensor] = None,
                       mask: Optional[torch.Tensor] = None, score: str = "softmax", renormalize: bool = True,
                       scale: float = 1.0, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of sum(dweights * weights) + dloss * loss of kgw_moe_route by its scores, (tokens, experts) in their type.

    dweights float32 (tokens, topk) or None; dloss a float32 tensor of one value, with the slope that kgw_moe_route
    gave (or one made of counts summed over ranks: experts * counts / (topk * tokens^2)); both or neither.
    mask, score, renormalize and scale as given to kgw_moe_route.  Masked tokens and scores of -inf get zeros, also where
    dloss or a weight's gradient is not finite.
    """
    if ids.dim() != 2:
        raise ValueError(f"ids must be (tokens, topk), got {tuple(ids.shape)}")
    topk = ids.shape[1]
    device, code, ld, score_code, tokens, E = _route_args(scores, topk, mask, score)
    _route_ids(ids, tokens, device)
    if (dloss is None) != (slope is None):
        raise ValueError("pass dloss and slope, or neither")
    if dweights is not None:
        _floats(dweights, (tokens, topk), device, "dweights")
    if dloss is not None:
        _floats(slope, (E,), device, "slope")
        if dloss.dtype != torch.float32 or dloss.numel() != 1 or dloss.device != device:
            raise ValueError(f"dloss must be a float32 tensor of one value on {device}")
    out = _result(out, (tokens, E), scores.dtype, device, "out", stream)
    if stream is not None:
        _used_on(stream, scores, ids, dweights, dloss, slope, mask, out)
    st = load_library().kgw_moe_route_grad(scores.data_ptr(), ld, code, _ptr(mask), ids.data_ptr(), ids.element_size(),
                                           _ptr(dweights), _ptr(dloss), _ptr(slope), tokens, E, topk, score_code,
                                           int(bool(renormalize)), scale, out.data_ptr(), _launch_stream(stream, device))
    _check(st, "kgw_moe_route_grad")
    return out


# ----------------------------------------------------------------------------
# the activation and its 8-bit checkpoint
# ----------------------------------------------------------------------------
_ACTS = {"swiglu": KGW_ACT_SWIGLU, "relu2": KGW_ACT_RELU2}


def _act_args(act: str, offsets: Optional[torch.Tensor], device):
    if act not in _ACTS:
        raise ValueError(f"act is 'swiglu' or 'relu2', got {act!r}")
    if offsets is not None:
        _check_offsets(offsets, device)


def _act_rows(t: Optional[torch.Tensor], rows: int, cols: int, halves: int, fp8: bool, dtype, device, what: str, stream):
    """A result of the activation and its scales: rows of `dtype`, or e4m3 bytes."""
    dtype = torch.uint8 if fp8 else dtype
    blocks = halves * -(-(cols // halves) // FP8_TOKEN_ALIGN) if fp8 else 0
    if stream is None and t is None:                       # (with its strides given an allocation takes 1.3 us, without 1.6)
        t = torch.empty_strided((rows, cols), (cols or 1, 1), dtype=dtype, device=device)
        return t, torch.empty_strided((blocks, rows), (rows or 1, 1), dtype=torch.uint8, device=device) if fp8 else None
    t = _result(t, (rows, cols), dtype, device, what, stream)
    return t, _empty((blocks, rows), torch.uint8, device, stream) if fp8 else None


def kgw_moe_act_fp8(h: torch.Tensor, *, act: str = "swiglu", offsets: Optional[torch.Tensor] = None, fp8: bool = False,
                    save: bool = True, out: Optional[torch.Tensor] = None, stream=None):
    """The activation between the expert products, keeping its input in 8 bits: (y, y_scales, saved, saved_scales).

    act "swiglu": h (rows, 2 inner) = [g | u], y = silu(g) * u; "relu2": h (rows, inner), y = relu(h)^2.  h is fp32, bf16 or
    fp16 with any row stride, inner a multiple of 8.  y (rows, inner) has h's type and y_scales is None; with `fp8`
    it is e4m3 bytes (uint8) with UE8M0 y_scales (ceil(inner/128), rows), the A of kgw_mgrouped_fp8 and kgw_wgrad_fp8_rows.
    saved and saved_scales are h in that form (swiglu: the blocks of g, then those of u), for kgw_moe_act_fp8_grad;
    None with save=False.  With `offsets` the rows from the last one on are neither read nor written.
    """
    code = _out_code(h.dtype)
    ld = _rows_2d(h, "h")
    device = _on_gpu(h, "h")
    _act_args(act, offsets, device)
    halves = 2 if act == "swiglu" else 1
    rows, wide = h.shape
    if wide % (8 * halves):
        raise ValueError(f"h must have {'twice ' if halves == 2 else ''}a multiple of 8 columns, got {wide}")
    inner = wide // halves
    y, y_scales = _act_rows(out, rows, inner, 1, fp8, h.dtype, device, "out", stream)
    saved, saved_scales = _act_rows(None, rows, wide, halves, True, None, device, "saved", stream) if save else (None, None)
    if stream is not None:
        _used_on(stream, h, offsets, y)
    st = load_library().kgw_moe_act_fp8(h.data_ptr(), ld, code, _ACTS[act], _ptr(offsets),
                                        0 if offsets is None else offsets.numel(), rows, inner, y.data_ptr(),
                                        _ptr(y_scales), _ptr(saved), _ptr(saved_scales), _launch_stream(stream, device))
    _check(st, "kgw_moe_act_fp8")
    return y, y_scales, saved, saved_scales


def kgw_moe_act_fp8_grad(dy: torch.Tensor, saved: torch.Tensor, saved_scales: torch.Tensor, *, act: str = "swiglu",
                         offsets: Optional[torch.Tensor] = None, fp8: bool = False, again: bool = False,
                         again_fp8: Optional[bool] = None, dh: Optional[torch.Tensor] = None,
                         y: Optional[torch.Tensor] = None, stream=None):
    """Gradient of kgw_moe_act_fp8 at the h it kept: (dh, dh_scales, y, y_scales).

    dy (rows, inner) is fp32, bf16 or fp16 with any row stride.  dh has dy's type and h's shape; with `fp8` it is in
    8 bits, scales laid out as saved_scales.  `again` also gives y = act(h) of the kept h (else None), in 8
    bits if `again_fp8` (default: as `fp8`).
    """
    code = _out_code(dy.dtype)
    ld = _rows_2d(dy, "dy")
    device = _on_gpu(dy, "dy")
    _act_args(act, offsets, device)
    halves = 2 if act == "swiglu" else 1
    rows, inner = dy.shape
    if inner % 8:
        raise ValueError(f"dy must have a multiple of 8 columns, got {inner}")
    blocks = halves * -(-inner // FP8_TOKEN_ALIGN)
    for t, shape, what in ((saved, (rows, halves * inner), "saved"), (saved_scales, (blocks, rows), "saved_scales")):
        if t.dtype not in (torch.uint8, torch.float8_e4m3fn) or tuple(t.shape) != shape or not t.is_contiguous() or \
                t.device != device:
            raise ValueError(f"{what} must be a contiguous uint8 {shape} tensor on {device}")
    if y is not None and not again:
        raise ValueError("y is written with again=True only")
    again_fp8 = fp8 if again_fp8 is None else again_fp8
    dh, dh_scales = _act_rows(dh, rows, halves * inner, halves, fp8, dy.dtype, device, "dh", stream)
    y, y_scales = _act_rows(y, rows, inner, 1, again_fp8, dy.dtype, device, "y", stream) if again else (None, None)
    if stream is not None:
        _used_on(stream, dy, saved, saved_scales, offsets, dh, y)
    st = load_library().kgw_moe_act_fp8_grad(dy.data_ptr(), ld, code, _ACTS[act], saved.data_ptr(), saved_scales.data_ptr(),
                                             _ptr(offsets), 0 if offsets is None else offsets.numel(), rows, inner,
                                             dh.data_ptr(), _ptr(dh_scales), _ptr(y), _ptr(y_scales),
                                             _launch_stream(stream, device))
    _check(st, "kgw_moe_act_fp8_grad")
    return dh, dh_scales, y, y_scales


# ----------------------------------------------------------------------------
# weight gradients made orthogonal
# ----------------------------------------------------------------------------
# a, b, c of X <- a X + (b A + c A A) X: steep at zero, so five steps bring singular values
# from 0.01 of the norm on into [0.7, 1.2].  Published with the Muon optimiser (K. Jordan et al., 2024).
NEWTON_SCHULZ_COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def kgw_newton_schulz(G: torch.Tensor, *, steps: int = 5, coefficients=NEWTON_SCHULZ_COEFFICIENTS, eps: float = 1e-7,
                      out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                      precise: bool = False, workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Orthogonalise G (m, n) or a batch (batch, m, n) by `steps` Newton-Schulz steps:
    X = G / (|G|_F + eps), then X <- a X + (b A + c A A) X with A = X X^T.

    G is fp32, bf16 or fp16 with contiguous rows (any row and batch stride), as kgw_wgrad_* writes
    it.  `coefficients` is one (a, b, c) or one per step.  The result has `out_dtype` (default: G's).
    fp32 and fp16 results, and those of short sides up to 128, take three fp16 products and keep fp32's precision.  Other bf16 results
    take one and are 1.7e-3 to 2.5e-3 off (of the norm, their own rounding's 1.66e-3 included), unless `precise`, which
    costs 1.3 to 2.4 times as much and leaves that rounding alone.  `workspace`: a uint8 tensor of
    kgw_newton_schulz_workspace_bytes bytes to reuse; allocated here when None.
    """
    code = _out_code(G.dtype)
    if G.dim() not in (2, 3):
        raise ValueError(f"G must be (m, n) or (batch, m, n), got {tuple(G.shape)}")
    batch = 1 if G.dim() == 2 else _int32(G.shape[0], "the batch")
    m, n = G.shape[-2:]
    if n > 1 and G.stride(-1) != 1:
        raise ValueError("G needs contiguous rows (stride 1 along the last axis)")
    ld = G.stride(-2) if m > 1 else n
    if ld < n:
        raise ValueError("G has overlapping rows")
    stride = G.stride(0) if G.dim() == 3 else 0
    steps = int(steps)
    if steps < 1 or steps > 64:
        raise ValueError("steps must be 1 .. 64")
    values = list(coefficients)
    if len(values) == 3 and not hasattr(values[0], "__len__"):
        values = values * steps
    elif len(values) == steps and all(len(v) == 3 for v in values):
        values = [float(x) for v in values for x in v]
    else:
        raise ValueError("coefficients must be (a, b, c), or one such triple per step")
    device = _on_gpu(G, "G")
    dtype = out.dtype if out is not None else (G.dtype if out_dtype is None else out_dtype)
    out_code = _out_code(dtype) | (KGW_NEWTON_PRECISE if precise else 0)
    out = _result(out, G.shape, dtype, device, "out", stream)
    lib = load_library()
    need = lib.kgw_newton_schulz_workspace_bytes(batch, m, n, out_code)
    if workspace is None:
        workspace = _empty(need, torch.uint8, device, stream)
    elif workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.device != device:
        raise ValueError("workspace must be a contiguous uint8 tensor on G's device")
    if stream is not None:
        _used_on(stream, G, out, workspace)
    st = lib.kgw_newton_schulz(G.data_ptr(), ld, stride, code, batch, m, n, steps,
                               (ctypes.c_float * (3 * steps))(*values), eps, out.data_ptr(), out_code,
                               workspace.data_ptr(), workspace.numel(), _launch_stream(stream, device))
    _check(st, "kgw_newton_schulz")
    return out
