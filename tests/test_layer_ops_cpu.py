"""The router, the activation and the weight gradient from 8-bit rows: what the C-ABI and the binding refuse, with no GPU
touched."""
import pytest
import torch

import grouped_gemm_expert_offsets_amd as kgw

OK, INVALID, MISALIGNED, OFFSETS, UNSUPPORTED = (kgw.KGW_SUCCESS, kgw.KGW_ERROR_INVALID_VALUE, kgw.KGW_ERROR_MISALIGNED,
                                                 kgw.KGW_ERROR_BAD_OFFSETS, kgw.KGW_ERROR_UNSUPPORTED)
P = 0x10000  # 16-byte aligned non-null address; never dereferenced on these paths
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers are not real")


@pytest.fixture(scope="module")
def lib():
    return kgw.load_library()


def route(lib, scores=P, ld=16, dt=0, mask=None, given=None, id_bytes=0, tokens=4, E=16, k=2, score=0, renorm=1, scale=1.0,
          ids=P, weights=P, counts=P, loss=P, slope=P, ws=None, ws_bytes=0):
    return lib.kgw_moe_route(scores, ld, dt, mask, given, id_bytes, tokens, E, k, score, renorm, scale, ids, weights, counts,
                             loss, slope, ws, ws_bytes, None)


def route_grad(lib, scores=P, ld=16, dt=0, mask=None, ids=P, id_bytes=4, dw=P, dloss=P, slope=P, tokens=4, E=16, k=2, score=0,
               renorm=1, scale=1.0, out=P):
    return lib.kgw_moe_route_grad(scores, ld, dt, mask, ids, id_bytes, dw, dloss, slope, tokens, E, k, score, renorm, scale,
                                  out, None)


@pytest.mark.parametrize("call", [route, route_grad])
def test_router_arguments(lib, call):
    for kw in (dict(dt=3), dict(dt=-1), dict(score=2), dict(renorm=2), dict(tokens=-1), dict(E=0), dict(k=0), dict(k=17), dict(ld=15),
               dict(scores=None), dict(ids=None)):
        assert call(lib, **kw) == INVALID, kw
    for kw in (dict(E=2049, ld=4096), dict(E=100, k=65, ld=100), dict(tokens=2 ** 23 + 1)):
        assert call(lib, **kw) == UNSUPPORTED, kw
    assert call(lib, scores=P + 2) == MISALIGNED and call(lib, dt=1, scores=P + 1) == MISALIGNED
    assert call(lib, ids=P + 2) == MISALIGNED


def test_router_pointers(lib):
    for name in ("weights", "counts", "loss", "slope"):
        assert route(lib, **{name: None}) == INVALID, name
        assert route(lib, **{name: P + 2}) == MISALIGNED, name
    assert route(lib, given=P, id_bytes=2) == INVALID and route(lib, given=P + 4, id_bytes=8) == MISALIGNED
    need = lib.kgw_moe_route_workspace_bytes(4096, 16, 0)
    assert need > 0
    assert route(lib, tokens=4096) == INVALID and route(lib, tokens=4096, ws=P, ws_bytes=need - 1) == INVALID
    assert route(lib, tokens=4096, ws=P + 4, ws_bytes=need) == MISALIGNED
    assert route_grad(lib, out=None) == INVALID and route_grad(lib, out=P + 1) == MISALIGNED
    assert route_grad(lib, dloss=None) == INVALID and route_grad(lib, slope=None) == INVALID
    assert route_grad(lib, id_bytes=3) == INVALID and route_grad(lib, id_bytes=8, ids=P + 4) == MISALIGNED
    for name in ("dw", "dloss", "slope"):
        assert route_grad(lib, **{name: P + 1}) == MISALIGNED, name
    assert route_grad(lib, tokens=0, scores=None, ids=None, out=None) == OK


def test_router_workspace(lib):
    f = lib.kgw_moe_route_workspace_bytes
    assert f(64, 256, 0) == 0 and f(0, 8, 0) == f(0, 8, 1) == 0        # one workgroup, one launch
    assert f(-1, 8, 0) == 0 and f(8, 0, 0) == 0 and f(8, 2049, 1) == 0 and f(2 ** 23 + 1, 8, 0) == 0
    assert f(2 ** 23, 256, 0) == f(10 ** 6, 256, 0) > 0               # never more workgroups


@no_gpu
def test_router_reaches_the_device(lib):
    device = kgw.KGW_ERROR_DEVICE
    need = lib.kgw_moe_route_workspace_bytes(2 ** 23, 2048, 0)
    assert route(lib) == device and route(lib, tokens=2 ** 23, E=2048, ld=2048, k=64, ws=P, ws_bytes=need) == device
    assert route(lib, tokens=0, scores=None, ids=None, weights=None) == device
    assert route_grad(lib) == device and route_grad(lib, dw=None, dloss=None, slope=None) == device
    assert route_grad(lib, tokens=2 ** 23, E=2048, ld=2048, k=64) == device


def act(lib, h=P, ld=256, dt=1, kind=0, off=None, E=0, rows=4, inner=128, y=P, ys=None, saved=P, ss=P):
    return lib.kgw_moe_act_fp8(h, ld, dt, kind, off, E, rows, inner, y, ys, saved, ss, None)


def act_grad(lib, dy=P, ld=128, dt=1, kind=0, saved=P, ss=P, off=None, E=0, rows=4, inner=128, dh=P, ds=None, y=None, ys=None):
    return lib.kgw_moe_act_fp8_grad(dy, ld, dt, kind, saved, ss, off, E, rows, inner, dh, ds, y, ys, None)


@pytest.mark.parametrize("call", [act, act_grad])
def test_activation_arguments(lib, call):
    for kw in (dict(dt=3), dict(kind=2), dict(kind=-1), dict(rows=-1), dict(inner=-8), dict(off=P, E=0), dict(saved=None), dict(ss=None),
               dict(ld=127)):
        assert call(lib, **kw) == INVALID, kw
    assert call(lib, rows=2 ** 31) == UNSUPPORTED and call(lib, inner=2 ** 28, ld=2 ** 29) == UNSUPPORTED
    assert call(lib, rows=2 ** 31 - 1, inner=4096, ld=8192) == UNSUPPORTED       # more workgroups than a launch holds
    assert call(lib, inner=132, ld=300) == MISALIGNED and call(lib, off=P + 2, E=1) == MISALIGNED
    assert call(lib, saved=P + 4) == MISALIGNED
    assert call(lib, rows=0) == OK and call(lib, inner=0) == OK


def test_activation_pointers(lib):
    assert act(lib, ld=255) == INVALID and act(lib, h=None) == INVALID and act(lib, y=None) == INVALID
    assert act(lib, h=P + 1) == MISALIGNED and act(lib, y=P + 1) == MISALIGNED and act(lib, y=P + 2, ys=P) == MISALIGNED
    assert act_grad(lib, dy=None) == INVALID and act_grad(lib, dh=None) == INVALID and act_grad(lib, ys=P) == INVALID
    assert act_grad(lib, dh=P + 1) == MISALIGNED and act_grad(lib, dh=P + 2, ds=P) == MISALIGNED
    assert act_grad(lib, y=P + 1) == MISALIGNED and act_grad(lib, y=P + 2, ys=P) == MISALIGNED


@no_gpu
def test_activation_reaches_the_device(lib):
    device = kgw.KGW_ERROR_DEVICE
    assert act(lib) == device and act(lib, saved=None, ss=None) == device and act(lib, ys=P + 1, ss=P + 3) == device
    assert act(lib, kind=1, ld=128) == device and act_grad(lib) == device and act_grad(lib, y=P, ys=P + 1, ds=P + 1) == device


def wgrad(lib, A=P, sa=P, B=P, sb=None, off=P, E=2, hidden=128, n=64, T=256, out=P, ptrs=None, dt=0, acc=0, ws=None, nb=0):
    return lib.kgw_wgrad_fp8_rows(A, sa, B, sb, off, E, hidden, n, T, out, ptrs, dt, acc, ws, nb, None)


def test_weight_gradient_arguments(lib):
    for kw in (dict(A=None), dict(sa=None), dict(B=None), dict(off=None), dict(out=None), dict(ptrs=P), dict(E=0), dict(hidden=-1),
               dict(n=-1), dict(T=-1), dict(dt=3), dict(acc=2)):
        assert wgrad(lib, **kw) == INVALID, kw
    for kw in (dict(A=P + 8), dict(B=P + 8), dict(out=P + 8), dict(sa=P + 2), dict(sb=P + 1), dict(off=P + 2), dict(hidden=124),
               dict(n=60), dict(n=68, sb=P), dict(out=None, ptrs=P + 4)):
        assert wgrad(lib, **kw) == MISALIGNED, kw
    assert wgrad(lib, T=200) == OFFSETS
    for kw in (dict(E=65537), dict(hidden=2 ** 25), dict(n=2 ** 28), dict(T=2 ** 31)):
        assert wgrad(lib, **kw) == UNSUPPORTED, kw
    assert wgrad(lib, hidden=0) == OK and wgrad(lib, n=0) == OK and wgrad(lib, T=0, acc=1) == OK


@no_gpu
def test_weight_gradient_reaches_the_device(lib):
    device = kgw.KGW_ERROR_DEVICE
    assert wgrad(lib) == device and wgrad(lib, sb=P) == device and wgrad(lib, n=72, hidden=24, sb=P) == device and wgrad(lib, n=72, T=128) == device
    assert wgrad(lib, T=0, A=None, sa=None, B=None) == device            # zeros to write


def test_binding_refuses_cpu_tensors():
    s, ids = torch.zeros((4, 8)), torch.zeros((4, 2), dtype=torch.int32)
    h, q = torch.zeros((4, 256)), torch.zeros((4, 256), dtype=torch.uint8)
    for call in (lambda: kgw.kgw_moe_route(s, 2), lambda: kgw.kgw_moe_route_grad(s, ids, torch.zeros((4, 2))),
                 lambda: kgw.kgw_moe_act_fp8(h), lambda: kgw.kgw_moe_act_fp8_grad(h[:, :128].contiguous(), q, q),
                 lambda: kgw.kgw_wgrad_fp8_rows(torch.zeros((128, 8), dtype=torch.uint8), torch.zeros((1, 128), dtype=torch.uint8),
                                                torch.zeros((128, 8), dtype=torch.bfloat16), ids.flatten()[:1])):
        with pytest.raises(ValueError):
            call()


BAD = {"experts past the limit": lambda s, i: kgw.kgw_moe_route(torch.zeros((2, 2049)), 2), "topk of zero": lambda s, i: kgw.kgw_moe_route(s, 0),
       "topk past the experts": lambda s, i: kgw.kgw_moe_route(s, 9), "topk past 32 bits": lambda s, i: kgw.kgw_moe_route(s, 2 ** 32 + 2),
       "a score name": lambda s, i: kgw.kgw_moe_route(s, 2, score="other"), "ids of another width": lambda s, i: kgw.kgw_moe_route(s, 3, ids=i),
       "a float mask": lambda s, i: kgw.kgw_moe_route(s, 2, mask=torch.ones(4)), "dloss alone": lambda s, i: kgw.kgw_moe_route_grad(s, i, None, dloss=s[0, :1]),
       "an act name": lambda s, i: kgw.kgw_moe_act_fp8(s, act="other"), "an inner size": lambda s, i: kgw.kgw_moe_act_fp8(torch.zeros((2, 24))),
       "no offsets": lambda s, i: kgw.kgw_moe_act_fp8(torch.zeros((2, 32)), offsets=torch.zeros(0, dtype=torch.int32)),
       "a checkpoint of another size": lambda s, i: kgw.kgw_moe_act_fp8_grad(s, torch.zeros((4, 8), dtype=torch.uint8), torch.zeros((2, 4), dtype=torch.uint8))}


@pytest.mark.parametrize("name", BAD)
def test_binding_refuses_before_it_allocates(monkeypatch, name):
    monkeypatch.setattr(kgw, "_on_gpu", lambda t, what: t.device)
    monkeypatch.setattr(kgw, "_empty", lambda *a: pytest.fail("memory was asked for"))
    with pytest.raises(ValueError):
        BAD[name](torch.zeros((4, 8)), torch.zeros((4, 2), dtype=torch.int32))
