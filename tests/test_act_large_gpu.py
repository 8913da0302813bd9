"""The activation and its gradient where results go past the caches' retention, and 8-bit results with offsets.

Rows repeat every PERIOD, so each result is bit for bit that of the first PERIOD rows alone (which test_act_gpu.py holds to
64 bits): the same arithmetic, in a call too small for any result to go past the caches.
"""
import pytest
import torch

import grouped_gemm_expert_offsets_amd as kgw
from test_act_gpu import DTYPES, HALVES, values

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs an MI355X")]

DEV = "cuda"
PERIOD = 251
PAST = 1 << 28                                              # bytes of a result that go past the caches
INNER = [4096, 768, 128, 904]                               # four blocks of 128 a workgroup, two, one; no multiple of 128


def repeated(x, rows):
    return x.repeat(-(-rows // PERIOD), 1)[:rows]


def same_rows(got, want, rows):
    """got (rows, ...) against want (PERIOD, ...), all rows, a part at a time."""
    whole = rows // PERIOD * PERIOD
    assert bool((got[:whole].view(-1, *want.shape) == want).all()) and torch.equal(got[whole:], want[:rows - whole])


def same_scales(got, want, rows):
    same_rows(got.t().contiguous(), want.t().contiguous(), rows)


def run(h, dy, act, fp8, again):
    y, ys, saved, ss = kgw.kgw_moe_act_fp8(h, act=act, fp8=fp8)
    dh, dhs, y2, y2s = kgw.kgw_moe_act_fp8_grad(dy, saved, ss, act=act, fp8=fp8, again=again)
    return [t for t in (y, saved, dh, y2) if t is not None], [t for t in (ys, ss, dhs, y2s) if t is not None]


def check(rows, inner, act, dtype, fp8, again):
    h, dy = values(PERIOD, HALVES[act] * inner, dtype, inner), values(PERIOD, inner, dtype, inner + 1)
    want, want_scales = run(h, dy, act, fp8, again)
    got, got_scales = run(repeated(h, rows), repeated(dy, rows), act, fp8, again)
    for g, w in zip(got, want):
        same_rows(g, w, rows)
    for g, w in zip(got_scales, want_scales):
        same_scales(g, w, rows)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ["swiglu", "relu2"])
@pytest.mark.parametrize("inner", INNER)
def test_every_result_past_the_caches(inner, act, dtype, fp8):
    row = inner * (1 if fp8 else dtype.itemsize)
    rows = PAST // row + 38                                 # the last workgroup's rows are few
    assert rows * row >= PAST
    check(rows, inner, act, dtype, fp8, True)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("inner", INNER)
def test_only_the_gradient_past_the_caches(inner, dtype, fp8):
    row = inner * (1 if fp8 else dtype.itemsize)
    rows = PAST // (2 * row) + 1
    assert rows * row < PAST <= 2 * rows * row
    for again in (False, True):
        check(rows, inner, "swiglu", dtype, fp8, again)


@pytest.mark.parametrize("inner,dtype", [(2048, torch.bfloat16), (1024, torch.float32)])
def test_as_many_bytes_as_go_past(inner, dtype):
    """The bound itself, and a row less."""
    rows = PAST // (inner * dtype.itemsize)
    for n in (rows, rows - 1):
        check(n, inner, "swiglu", dtype, False, True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ["swiglu", "relu2"])
@pytest.mark.parametrize("rows,last,inner", [(200, 1, 136), (200, 64, 512), (200, 130, 768), (200, 200, 136), (5000, 3333, 136), (70, 69, 4096)])
def test_eight_bit_results_up_to_the_last_offset(rows, last, inner, act, dtype):
    h, dy = values(rows, HALVES[act] * inner, dtype, 1, 3, 1), values(rows, inner, dtype, 2, 5, 1)
    want, want_scales = run(h, dy, act, True, True)
    h[last:], dy[last:] = float("nan"), float("nan")
    offsets = torch.tensor([0, min(last, 64), last], dtype=torch.int32, device=DEV)
    y, ys, saved, ss = kgw.kgw_moe_act_fp8(h, act=act, fp8=True, offsets=offsets)
    dh, dhs, y2, y2s = kgw.kgw_moe_act_fp8_grad(dy, saved, ss, act=act, fp8=True, again=True, offsets=offsets)
    assert all(torch.equal(g[:last], w[:last]) for g, w in zip((y, saved, dh, y2), want))
    assert all(torch.equal(g[:, :last], w[:, :last]) for g, w in zip((ys, ss, dhs, y2s), want_scales))
