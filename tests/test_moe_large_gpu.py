"""Rows whose buffer passes 512 MiB, which are read past the caches' retention: unpermute, weighted and not, and its
gradient, with odd row lengths and contents that vary along the row.

Against 64 bits, in parts; tolerances as in test_moe_gpu.py.
"""
import pytest
import torch

import grouped_gemm_expert_offsets_amd as kgw

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs an MI355X")]

DEV = "cuda"
U32 = 2.0 ** -24
CASES = [(140001, 2, 5, 1001, torch.bfloat16), (90001, 3, 7, 1030, torch.float16), (70001, 4, 6, 501, torch.float32),
         (9001, 8, 16, 4096, torch.bfloat16)]


def half_step(dtype):
    f = torch.finfo(dtype)
    return f.eps / 2, f.tiny * f.eps / 2


def routed(tokens, k, E, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    ids = torch.rand((tokens, E + 1), generator=g, device=DEV).topk(k, dim=1).indices       # id E: another rank's
    _, _, row_of, src_of = kgw.kgw_moe_sort(ids, E, alignment=256)
    return g, row_of, src_of


@pytest.mark.parametrize("tokens,k,E,hidden,dtype", CASES)
def test_unpermute_and_its_gradient(tokens, k, E, hidden, dtype):
    g, row_of, src_of = routed(tokens, k, E, hidden)
    rows = src_of.numel()
    assert rows * hidden * dtype.itemsize > 2 ** 29
    y = torch.randn((rows, hidden), generator=g, device=DEV).to(dtype)
    y[src_of < 0] = float("nan")
    w = torch.softmax(torch.randn((tokens, k), generator=g, device=DEV), 1)
    dout = torch.randn((tokens, hidden), generator=g, device=DEV).to(dtype)
    weighted, plain = kgw.kgw_moe_unpermute(y, row_of, w), kgw.kgw_moe_unpermute(y, row_of)
    dy = torch.full((rows, hidden), float("nan"), dtype=dtype, device=DEV)
    dw = torch.full((tokens, k), float("nan"), device=DEV)
    kgw.kgw_moe_unpermute_grad(dout, y, row_of, src_of, w, dy, dw)
    assert not dy[src_of < 0].any()
    rel, tiny = half_step(dtype)
    for t in range(0, tokens, 8192):
        r = row_of[t:t + 8192].long()
        here = (r >= 0)[..., None]
        terms = torch.where(here, y[r.clamp(min=0)].double(), 0.0)
        wd, d = w[t:t + 8192].double()[..., None], dout[t:t + 8192].double()[:, None]
        for got, scaled in ((weighted, wd * terms), (plain, terms)):
            want, size = scaled.sum(1), scaled.abs().sum(1)
            err = (got[t:t + 8192].double() - want).abs()
            assert bool((err <= rel * want.abs() + (1 + rel) * (k + 2) * U32 * size + tiny).all()), t
        want, size = (d * terms).sum(2), (d * terms).abs().sum(2)
        assert bool(((dw[t:t + 8192].double() - want).abs() <= (hidden / 256 + 24) * U32 * size).all()), t
        want = wd * d
        err = (dy[r.clamp(min=0)].double() - want).abs()
        assert bool(torch.where(here, err <= (rel + 1.01 * U32) * want.abs() + tiny, True).all()), t
