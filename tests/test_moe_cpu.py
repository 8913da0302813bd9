"""Token sort, permute and unpermute: what the C-ABI and the binding refuse, with no GPU touched."""
import pytest
import torch

import grouped_gemm_expert_offsets_amd as kgw

INVALID, MISALIGNED, OFFSETS, UNSUPPORTED = (kgw.KGW_ERROR_INVALID_VALUE, kgw.KGW_ERROR_MISALIGNED,
                                             kgw.KGW_ERROR_BAD_OFFSETS, kgw.KGW_ERROR_UNSUPPORTED)
P = 0x10000  # 16-byte aligned non-null address; never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    return kgw.load_library()


def test_rows_bound():
    # one assignment wastes at most align - 1 rows of its expert
    assert kgw.kgw_moe_rows(0, 2, 4, 128) == 0
    assert kgw.kgw_moe_rows(1, 1, 1, 128) == 128
    assert kgw.kgw_moe_rows(1, 2, 8, 128) == 256
    assert kgw.kgw_moe_rows(64, 8, 256, 128) == (512 + 256 * 127) // 128 * 128
    assert kgw.kgw_moe_rows(10, 3, 7, 1) == 30
    # the bound holds for the worst split: every expert one past a multiple
    assert kgw.kgw_moe_rows(129 * 4, 1, 4, 128) >= 4 * 256
    for bad in [(-1, 1, 1, 1), (1, 0, 1, 1), (1, 1, 0, 1), (1, 1, 1, 0), (2 ** 31, 1, 1, 1), (2 ** 30, 2, 1, 1)]:
        with pytest.raises(ValueError):
            kgw.kgw_moe_rows(*bad)


def test_sort_workspace(lib):
    assert lib.kgw_moe_sort_workspace_bytes(64, 8, 256) == 0                     # one workgroup, one launch
    assert lib.kgw_moe_sort_workspace_bytes(32768, 8, 32) == 128 * 32 * 4
    assert lib.kgw_moe_sort_workspace_bytes(10 ** 7, 8, 32) == 128 * 32 * 4      # never more workgroups
    assert lib.kgw_moe_sort_workspace_bytes(-1, 8, 32) == 0
    sizes = [lib.kgw_moe_sort_workspace_bytes(t, 2, 7) for t in range(0, 200000, 331)]
    assert sizes == sorted(sizes)                                                # enough for fewer tokens too


def sort(lib, ids=P, id_bytes=8, tokens=64, k=8, E=16, align=128, rows=4096, counts=P, offsets=P, row_of=P, src_of=P,
         ws=None, ws_bytes=0):
    return lib.kgw_moe_sort(ids, id_bytes, tokens, k, E, align, rows, counts, offsets, row_of, src_of, ws, ws_bytes,
                            None)


def test_sort_arguments(lib):
    assert sort(lib, id_bytes=2) == INVALID
    assert sort(lib, tokens=-1) == INVALID
    assert sort(lib, k=0) == INVALID
    assert sort(lib, E=0) == INVALID
    assert sort(lib, align=0) == INVALID
    for name in ("ids", "counts", "offsets", "row_of", "src_of"):
        assert sort(lib, **{name: None}) == INVALID, name
    assert sort(lib, E=2049) == UNSUPPORTED
    assert sort(lib, tokens=2 ** 28, k=8) == UNSUPPORTED
    assert sort(lib, align=2 ** 30) == UNSUPPORTED
    assert sort(lib, rows=2 ** 31, align=1) == UNSUPPORTED
    assert sort(lib, rows=100) == OFFSETS
    assert sort(lib, ids=P + 4) == MISALIGNED
    assert sort(lib, ids=P + 2, id_bytes=4) == MISALIGNED
    assert sort(lib, row_of=P + 1) == MISALIGNED
    assert sort(lib, tokens=32768, rows=2 ** 19) == INVALID                      # needs its workspace
    assert sort(lib, tokens=32768, rows=2 ** 19, ws=P, ws_bytes=8) == INVALID


def permute(lib, x=P, ld=16, dt=1, row_of=P, src_of=P, tokens=4, k=2, rows=256, hidden=16, out=P):
    return lib.kgw_moe_permute(x, ld, dt, row_of, src_of, tokens, k, rows, hidden, out, None)


def unpermute(lib, y=P, ld=16, dt=1, row_of=P, w=P, tokens=4, k=2, rows=256, hidden=16, out=P):
    return lib.kgw_moe_unpermute(y, ld, dt, row_of, w, tokens, k, rows, hidden, out, None)


def grad(lib, dout=P, ldd=16, y=P, ldy=16, dt=1, row_of=P, src_of=P, w=P, tokens=4, k=2, rows=256, hidden=16, dy=P, dw=P):
    return lib.kgw_moe_unpermute_grad(dout, ldd, y, ldy, dt, row_of, src_of, w, tokens, k, rows, hidden, dy, dw, None)


@pytest.mark.parametrize("call", [permute, unpermute, grad])
def test_row_arguments(lib, call):
    assert call(lib, dt=3) == INVALID
    assert call(lib, tokens=-1) == INVALID
    assert call(lib, k=0) == INVALID
    assert call(lib, rows=-1) == INVALID
    assert call(lib, hidden=-1) == INVALID
    assert call(lib, row_of=None) == INVALID
    assert call(lib, row_of=P + 2) == MISALIGNED
    assert call(lib, tokens=2 ** 30, k=2) == UNSUPPORTED
    assert call(lib, rows=2 ** 31) == UNSUPPORTED
    assert call(lib, hidden=2 ** 28) == UNSUPPORTED
    assert call(lib, tokens=2 ** 24 + 1, k=1) == UNSUPPORTED


def test_pointer_arguments(lib):
    assert permute(lib, x=None) == INVALID and permute(lib, out=None) == INVALID and permute(lib, src_of=None) == INVALID
    assert permute(lib, ld=15) == INVALID and permute(lib, x=P + 1) == MISALIGNED
    assert permute(lib, dt=0, x=P + 2) == MISALIGNED
    assert unpermute(lib, y=None) == INVALID and unpermute(lib, out=None) == INVALID and unpermute(lib, ld=15) == INVALID
    assert unpermute(lib, w=P + 2) == MISALIGNED and unpermute(lib, out=P + 1) == MISALIGNED
    for name in ("dout", "y", "src_of", "w", "dy", "dw"):
        assert grad(lib, **{name: None}) == INVALID, name
    assert grad(lib, ldd=15) == INVALID and grad(lib, ldy=15) == INVALID
    assert grad(lib, dw=P + 2) == MISALIGNED and grad(lib, dy=P + 1) == MISALIGNED


def test_nothing_to_do_needs_no_device(lib):
    assert permute(lib, rows=0, x=None, row_of=None, src_of=None, out=None) == kgw.KGW_SUCCESS
    assert permute(lib, hidden=0) == kgw.KGW_SUCCESS
    assert unpermute(lib, tokens=0, y=None, row_of=None, out=None) == kgw.KGW_SUCCESS
    assert grad(lib, tokens=0, rows=0, dout=None, y=None, dy=None, dw=None, w=None, row_of=None) == kgw.KGW_SUCCESS


def test_binding_refuses_cpu_tensors():
    ids = torch.zeros((4, 2), dtype=torch.int64)
    x = torch.zeros((4, 16))
    row_of, src_of, w = torch.zeros((4, 2), dtype=torch.int32), torch.zeros(128, dtype=torch.int32), torch.zeros((4, 2))
    for call in (lambda: kgw.kgw_moe_sort(ids, 3), lambda: kgw.kgw_moe_permute(x, row_of, src_of),
                 lambda: kgw.kgw_moe_unpermute(x, row_of, w),
                 lambda: kgw.kgw_moe_unpermute_grad(x, x, row_of, src_of, w)):
        with pytest.raises(ValueError):
            call()


def test_launches_that_do_not_fit_are_refused(lib):
    # a launch holds fewer than 2^24 workgroups of four waves; empty rows take a wave for two of them
    assert grad(lib, tokens=2 ** 23, k=1, rows=2 ** 26 - 1) == UNSUPPORTED
    assert grad(lib, tokens=2 ** 23, k=1, rows=2 ** 26 - 7) == UNSUPPORTED
    assert permute(lib, tokens=2 ** 23, k=1, rows=2 ** 27 - 2 ** 24) == UNSUPPORTED
    assert permute(lib, tokens=2 ** 23, k=1, rows=256, hidden=8192, ld=8192) == UNSUPPORTED       # 8 waves a token
    assert unpermute(lib, tokens=2 ** 23, k=1, rows=2 ** 30, hidden=8192, ld=8192) == UNSUPPORTED
    assert grad(lib, tokens=2 ** 62, k=4) == UNSUPPORTED                         # tokens * topk passes 64 bits


@pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers are not real")
def test_launches_that_just_fit_reach_the_device(lib):
    device = kgw.KGW_ERROR_DEVICE
    assert grad(lib, tokens=2 ** 23, k=1, rows=2 ** 26 - 8) == device
    assert permute(lib, tokens=2 ** 23, k=1, rows=2 ** 27 - 2 ** 24 - 8) == device
    assert permute(lib, tokens=2 ** 23 - 1, k=1, rows=8, hidden=8192, ld=8192) == device
    assert unpermute(lib, tokens=2 ** 23, k=1, rows=2 ** 30) == device


@pytest.mark.parametrize("kw", [dict(num_experts=2 ** 30), dict(num_experts=2 ** 32 + 4), dict(num_experts=2049),
                                dict(alignment=2 ** 32 + 128), dict(alignment=2 ** 32 + 128, rows=256), dict(rows=2 ** 31),
                                dict(rows=-128), dict(num_experts=0, rows=128)])
def test_binding_refuses_before_it_allocates(monkeypatch, kw):
    # numbers that do not fit the C call's arguments are not cut to ones that do
    monkeypatch.setattr(kgw, "_on_gpu", lambda t, what: t.device)
    monkeypatch.setattr(kgw, "_empty", lambda *a: pytest.fail("memory was asked for"))
    with pytest.raises(ValueError):
        kgw.kgw_moe_sort(torch.zeros((4, 2), dtype=torch.int32), **{"num_experts": 4, **kw})


def test_rows_arguments_are_not_cut():
    for bad in [(4, 2, 2 ** 32 + 4, 128), (4, 2, 4, 2 ** 32 + 128), (4, 2 ** 32 + 2, 4, 128)]:
        with pytest.raises(ValueError):
            kgw.kgw_moe_rows(*bad)
