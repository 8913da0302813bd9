"""kgw_newton_schulz: what the C-ABI and the binding refuse, and its workspace sizes, with no GPU touched."""
import ctypes

import pytest
import torch

import grouped_gemm_expert_offsets_amd as kgw

INVALID, MISALIGNED, UNSUPPORTED = kgw.KGW_ERROR_INVALID_VALUE, kgw.KGW_ERROR_MISALIGNED, kgw.KGW_ERROR_UNSUPPORTED
P = 0x10000  # aligned non-null address; never dereferenced on these paths
CO = (ctypes.c_float * 15)(*([3.4445, -4.7750, 2.0315] * 5))


@pytest.fixture(scope="module")
def lib():
    return kgw.load_library()


def call(lib, G=P, ld=64, stride=2048, dt=0, batch=2, m=32, n=64, steps=5, co=CO, eps=1e-7, out=P, odt=0, ws=P,
         ws_bytes=1 << 40):
    return lib.kgw_newton_schulz(G, ld, stride, dt, batch, m, n, steps, co, eps, out, odt, ws, ws_bytes, None)


def test_arguments(lib):
    assert call(lib, dt=3) == INVALID and call(lib, odt=-1) == INVALID
    assert call(lib, steps=0) == INVALID and call(lib, steps=65) == UNSUPPORTED
    assert call(lib, co=None) == INVALID
    assert call(lib, eps=-1.0) == INVALID and call(lib, eps=float("nan")) == INVALID
    assert call(lib, batch=-1) == INVALID and call(lib, m=-1) == INVALID and call(lib, n=-1) == INVALID
    assert call(lib, batch=65536) == UNSUPPORTED and call(lib, m=2 ** 20 + 1) == UNSUPPORTED
    assert call(lib, batch=1000, m=2 ** 17, n=2 ** 17, ld=2 ** 17) == UNSUPPORTED
    assert call(lib, G=None) == INVALID and call(lib, out=None) == INVALID and call(lib, ws=None) == INVALID
    assert call(lib, ld=63) == INVALID and call(lib, stride=-1) == INVALID
    assert call(lib, G=P + 2) == MISALIGNED and call(lib, dt=1, G=P + 1) == MISALIGNED
    assert call(lib, out=P + 2) == MISALIGNED and call(lib, ws=P + 128) == MISALIGNED
    assert call(lib, ws_bytes=100) == INVALID and call(lib, m=200, n=300, ld=300, ws_bytes=100000) == INVALID
    for empty in (dict(batch=0), dict(m=0), dict(n=0)):
        assert call(lib, G=None, out=None, ws=None, **empty) == kgw.KGW_SUCCESS


def test_workspace(lib):
    size = lib.kgw_newton_schulz_workspace_bytes
    assert size(0, 4, 4, 0) == 0 and size(1, 0, 4, 0) == 0 and size(-1, 4, 4, 0) == 0 and size(1, 4, 4, 9) == 0
    # the same for a matrix and its transpose; more for results that keep three products
    assert size(3, 200, 300, 0) == size(3, 300, 200, 0) > size(3, 200, 300, 1) > 0
    # short sides of at most 128 always keep three products
    assert size(3, 100, 300, 0) == size(3, 300, 100, 1) > 0
    assert size(8, 4096, 2048, 1) >= 8 * (2 * 4 * 4096 * 2048 + 2 * 2 * 2048 * 2048)


def test_binding_refuses_without_a_gpu():
    with pytest.raises(ValueError):
        kgw.kgw_newton_schulz(torch.zeros((4, 8)))
    with pytest.raises(ValueError):
        kgw.kgw_newton_schulz(torch.zeros((4, 8), dtype=torch.float64))
    with pytest.raises(ValueError):
        kgw.kgw_newton_schulz(torch.zeros((4, 8)), coefficients=(1.0,))


def test_binding_does_not_cut_the_batch(monkeypatch):
    monkeypatch.setattr(kgw, "_on_gpu", lambda t, what: t.device)
    monkeypatch.setattr(kgw, "_empty", lambda *a: pytest.fail("memory was asked for"))
    with pytest.raises(ValueError):
        kgw.kgw_newton_schulz(torch.zeros((1, 1, 1)).expand(2 ** 32 + 1, 1, 1))


def test_precise_results(lib):
    size, precise = lib.kgw_newton_schulz_workspace_bytes, kgw.KGW_NEWTON_PRECISE
    assert size(3, 200, 300, kgw.KGW_OUT_BF16 | precise) == size(3, 200, 300, kgw.KGW_OUT_FP32)
    assert size(3, 200, 300, kgw.KGW_OUT_FP32 | precise) == size(3, 200, 300, kgw.KGW_OUT_FP32)
    assert size(3, 200, 300, 3 | precise) == 0 and size(3, 200, 300, 1 | 0x200) == 0
    assert call(lib, odt=3 | precise) == INVALID and call(lib, odt=1 | 0x200) == INVALID
    assert call(lib, odt=precise, out=P + 2) == MISALIGNED
    assert call(lib, odt=1 | precise, ws_bytes=100) == INVALID
