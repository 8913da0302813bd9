"""The router, its balance loss and their gradient against plain 64-bit forms.

u = 2^-24 is fp32's half step.  With z the distance of a score to the largest of its row (sigmoid: its size), the share
exp2(fl(fl(x - top) log2 e)) is off by at most 3 z u from the argument's roundings and 2 u from the function: (3 z + 3) u of
itself; a sigmoid by (2 z + 6) u.  Sums of E shares add at most 45 u (32 additions on a lane, 6 across lanes, products
and a division), so weights are within (6 Z + 60) u of themselves, Z the largest z of the row.  The loss adds the tokens
of a lane, 16 waves, 64 + 32 partial sums of workgroups and their results: (6 Z + 400) u.  A gradient is within
(10 Z + 200) u of the sum of its terms' sizes, and half a step of its type.  Shares below 2^-126 may become zero.
"""
import numpy as np
import pytest
import torch

import grouped_gemm_expert_offsets_amd as kgw

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs an MI355X")]

DEV = "cuda"
U = 2.0 ** -24
LEAST = 2.0 ** -126
INF = float("inf")
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def half_step(dtype):
    f = torch.finfo(dtype)
    return (0.0, 0.0) if dtype == torch.float32 else (f.eps / 2, f.tiny * f.eps / 2)


def make_scores(tokens, experts, dtype, seed, pad=0, offset=0, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    wide = (spread * torch.randn(tokens * (experts + pad) + offset + 1, generator=g)).to(dtype).to(DEV)
    return wide[offset:offset + tokens * (experts + pad)].view(tokens, experts + pad)[:, :experts]


def reference(scores, k, mask=None, score="softmax", renormalize=True, scale=1.0, ids=None, dweights=None, dloss=None):
    """ids, weights, counts, loss, slope, gradient, and the sizes that the tolerances count, in 64 bits on the CPU."""
    x = scores.detach().double().cpu()
    T, E = x.shape
    if mask is not None:
        x = torch.where(mask.cpu()[:, None], x, torch.tensor(-INF, dtype=torch.float64))
    allowed = x > -INF
    if ids is None:
        top, ids = torch.sort(x, dim=1, descending=True, stable=True)
        ids = torch.where(top[:, :k] > -INF, ids[:, :k], -1)
    else:
        ids = ids.cpu().long()
        inside = (ids >= 0) & (ids < E)
        ids = torch.where(inside & allowed.gather(1, ids.clamp(0, E - 1)), ids, -1)
    here = ids >= 0
    x = torch.where(allowed, x, 0.0).requires_grad_()
    rows = allowed.any(1)
    if score == "softmax":
        u = torch.where(allowed, torch.exp(x - torch.where(allowed, x.detach(), -1e9).amax(1, keepdim=True).clamp(min=-1e8)), 0.0)
        p = u / torch.where(rows, u.sum(1), 1.0)[:, None]
        u = p
    else:
        u = torch.where(allowed, torch.sigmoid(x), 0.0)
        p = u / (u.sum(1, keepdim=True) + 1e-20)
    w = torch.where(here, u.gather(1, ids.clamp(min=0)), 0.0)
    if renormalize:
        total = w.sum(1, keepdim=True)
        w = w / (total + 1e-20 if score == "sigmoid" else torch.where(total > 0, total, 1.0))
    w = w * scale
    counts = torch.bincount(ids[here], minlength=E)
    n = int(rows.sum())
    slope = counts.double() * E / (k * n * n) if n else torch.zeros(E, dtype=torch.float64)
    loss = (p.sum(0) * slope).sum()
    grad = size = None
    if dweights is not None or dloss is not None:
        dw = torch.zeros_like(w) if dweights is None else torch.where(here, dweights.double().cpu(), 0.0)
        dl = 0.0 if dloss is None else float(dloss)
        ((w * dw).sum() + dl * loss).backward()
        grad = torch.where(allowed, x.grad, 0.0)
        with torch.no_grad():
            push = abs(dl) * slope[None]
            pushed = (p * push).sum(1, keepdim=True)
            q = w / scale
            part = torch.zeros_like(x).scatter_add_(1, ids.clamp(min=0), torch.where(
                here, q * (abs(scale) * dw.abs() + (abs(scale) * dw.abs() * q).sum(1, keepdim=True)), 0.0))
            spread = p * (q * dw.abs() * abs(scale)).sum(1, keepdim=True)
            size = p * (push + pushed) + part + spread
    z = torch.where(allowed, x.detach().abs() if score == "sigmoid" else
                    (x.detach() - torch.where(allowed, x.detach(), -1e9).amax(1, keepdim=True)).abs(), 0.0)
    Z = float(z.max()) if z.numel() else 0.0
    return dict(ids=ids, weights=w.detach(), counts=counts, loss=float(loss.detach()), slope=slope, grad=grad, size=size, Z=Z)


def check(scores, k, seed=0, **kw):
    ids_given = kw.pop("ids", None)
    g = torch.Generator().manual_seed(seed + 77)
    T, E = scores.shape
    dw = torch.randn((T, k), generator=g).to(DEV)
    dl = torch.tensor(0.3 * T, device=DEV)
    want = reference(scores, k, ids=ids_given, dweights=dw, dloss=dl, **kw)
    ids, weights, counts, loss, slope = kgw.kgw_moe_route(scores, k, ids=ids_given, **kw)
    assert ids.dtype == counts.dtype == torch.int32 and weights.dtype == slope.dtype == loss.dtype == torch.float32
    assert torch.equal(ids.cpu().long(), want["ids"])
    assert torch.equal(counts.cpu().long(), want["counts"])
    Z = want["Z"]
    w, ww = weights.cpu().double(), want["weights"]
    assert bool(((w - ww).abs() <= (6 * Z + 60) * U * ww.abs() + LEAST).all())
    assert abs(float(loss) - want["loss"]) <= (6 * Z + 400) * U * abs(want["loss"])
    assert bool(((slope.cpu().double() - want["slope"]).abs() <= 5 * U * want["slope"]).all())
    out = torch.full((T, E), float("nan"), dtype=scores.dtype, device=DEV)
    got = kgw.kgw_moe_route_grad(scores, ids, dw, dloss=dl, slope=slope, out=out, **kw)
    assert got is out
    rel, tiny = half_step(scores.dtype)
    tol = (1 + rel) * (10 * Z + 200) * U * want["size"] + rel * want["grad"].abs() + tiny + LEAST
    d = (got.cpu().double() - want["grad"]).abs()
    assert bool((d <= tol).all()), f"gradient off by {float((d / tol).max())} times the bound"
    return ids, weights, counts, loss, slope, got


SHAPES = [(1, 1, 1), (1, 4, 2), (3, 8, 8), (64, 256, 8), (65, 256, 8), (500, 31, 3), (257, 32, 4), (1000, 33, 6), (300, 61, 2),
          (129, 64, 7), (77, 100, 16), (2000, 128, 8), (4099, 255, 6), (70, 257, 8), (33, 512, 20), (40, 700, 64),
          (17, 1025, 5), (9, 2048, 9), (30, 64, 64)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,experts,k", SHAPES)
def test_shapes_and_types(tokens, experts, k, dtype):
    odd = tokens % 2
    check(make_scores(tokens, experts, dtype, tokens + experts, 3 * odd, odd), k, score="sigmoid" if tokens % 3 == 0 else "softmax",
          renormalize=tokens % 5 != 0, scale=2.5 if odd else 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("tokens,experts,k", [(200, 16, 4), (333, 200, 8), (50, 600, 3)])
def test_masks_and_forbidden_experts(tokens, experts, k, score, renormalize):
    g = torch.Generator().manual_seed(tokens)
    scores = make_scores(tokens, experts, torch.float32, 1, 5, 1)
    scores[(torch.rand((tokens, experts), generator=g) < 0.3).to(DEV)] = -INF
    scores[3] = -INF                                        # a token that may take none
    scores[4, k // 2:] = -INF                               # one that may take fewer than k
    mask = (torch.rand(tokens, generator=g) < 0.8).to(DEV)
    mask[3] = mask[4] = True
    mask[0] = False
    scores[~mask] = float("nan")                            # padding holds anything
    ids, weights, _, loss, _, grad = check(scores, k, mask=mask, score=score, renormalize=renormalize)
    assert (ids[3] == -1).all() and (weights[3] == 0).all() and (grad[3] == 0).all()
    assert (ids[~mask] == -1).all() and (weights[~mask] == 0).all() and (grad[~mask] == 0).all()
    assert torch.equal(grad[mask] == 0, (scores[mask] == -INF) | (grad[mask] == 0))
    assert not grad.isnan().any() and not loss.isnan()
    byte = kgw.kgw_moe_route(scores, k, mask=mask.to(torch.uint8), score=score, renormalize=renormalize)
    assert torch.equal(byte[0], ids) and torch.equal(byte[1], weights)


@pytest.mark.parametrize("tokens,experts,k", [(100, 40, 4), (40, 256, 8), (3000, 8, 2)])
def test_no_token_takes_part(tokens, experts, k):
    scores = torch.full((tokens, experts), -INF, device=DEV)
    for s, m in ((scores, None), (torch.full_like(scores, float("nan")), torch.zeros(tokens, dtype=torch.bool, device=DEV))):
        ids, weights, counts, loss, slope, grad = check(s, k, mask=m)
        assert (ids == -1).all() and not weights.any() and not counts.any() and float(loss) == 0 and not slope.any()
        assert not grad.any()


def test_no_tokens():
    ids, weights, counts, loss, slope = kgw.kgw_moe_route(torch.empty((0, 12), device=DEV), 3)
    assert ids.shape == weights.shape == (0, 3) and counts.tolist() == [0] * 12 and float(loss) == 0
    assert slope.tolist() == [0.0] * 12
    assert kgw.kgw_moe_route_grad(torch.empty((0, 12), device=DEV), ids, weights, dloss=loss, slope=slope).shape == (0, 12)


@pytest.mark.parametrize("experts", [5, 24, 48, 90, 250, 300, 900, 1500])
def test_ties_go_to_the_lowest_index(experts):
    g = torch.Generator().manual_seed(experts)
    scores = torch.randint(-2, 3, (70, experts), generator=g).float().to(DEV)
    scores[scores == 0] *= -1                               # -0 equals 0
    scores[:, ::3] = scores[:, ::3].abs()
    check(scores, 5)
    check(torch.zeros((9, experts), dtype=torch.bfloat16, device=DEV), 4)


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("tokens,experts,k", [(90, 20, 3), (70, 256, 8), (20, 700, 70)])
def test_given_ids(tokens, experts, k, dtype):
    k = min(k, 64)
    g = torch.Generator().manual_seed(tokens)
    scores = make_scores(tokens, experts, torch.float32, 2)
    scores[2, 5] = -INF
    mask = (torch.rand(tokens, generator=g) < 0.9).to(DEV)
    ids = torch.rand((tokens, experts), generator=g).topk(k, dim=1).indices
    ids[2, 0] = 5
    ids[2, 1:] = torch.arange(k - 1) + 6
    ids[4, 0], ids[5, 1] = -7, experts
    ids = ids.to(dtype).to(DEV)
    for score in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            check(scores, k, ids=ids, mask=mask, score=score, renormalize=renormalize)


def test_the_same_expert_twice():
    scores = make_scores(6, 10, torch.float32, 3)
    ids = torch.tensor([[1, 1], [2, 3], [4, 4], [9, 9], [0, 1], [5, 5]], device=DEV)
    dw = torch.randn((6, 2), generator=torch.Generator().manual_seed(1)).to(DEV)
    for renormalize in (True, False):
        want = reference(scores, 2, ids=ids, renormalize=renormalize, dweights=dw)
        got = kgw.kgw_moe_route_grad(scores, ids, dw, renormalize=renormalize).cpu().double()
        assert bool(((got - want["grad"]).abs() <= (10 * want["Z"] + 200) * U * want["size"]).all())


def test_the_gradients_parts_alone():
    scores = make_scores(50, 24, torch.float32, 5)
    ids, _, _, _, slope = kgw.kgw_moe_route(scores, 3)
    dw, dl = torch.randn((50, 3), device=DEV), torch.tensor([2.0], device=DEV)
    both = kgw.kgw_moe_route_grad(scores, ids, dw, dloss=dl, slope=slope)
    a = kgw.kgw_moe_route_grad(scores, ids, dw)
    b = kgw.kgw_moe_route_grad(scores, ids, None, dloss=dl, slope=slope)
    assert a.abs().sum() > 0 and b.abs().sum() > 0
    assert float((a + b - both).abs().max()) <= 64 * U * float(dw.abs().max() + 1)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_gradient_against_differences(score, renormalize):
    """(f(x + h s) - f(x - h s)) / 2h for f = sum dw w + dloss loss, the counts held: f comes from fp32 weights, each within
    (6 Z + 60) u, so the quotient is within sum |dw w| 2 (6 Z + 60) u / 2h + O(h^2) with third derivatives of at most 6 sum |dw w|."""
    T, E, k = 40, 12, 3
    scores = make_scores(T, E, torch.float32, 8, spread=0.7)
    ids, _, _, _, slope = kgw.kgw_moe_route(scores, k, score=score, renormalize=renormalize)
    g = torch.Generator().manual_seed(2)
    dw, s = torch.randn((T, k), generator=g).to(DEV), torch.randn((T, E), generator=g).sign().to(DEV)
    dl = torch.tensor(3.0, device=DEV)

    def f(x):
        _, w, _, _, _ = kgw.kgw_moe_route(x, k, ids=ids, score=score, renormalize=renormalize)
        u = torch.softmax(x.double(), 1) if score == "softmax" else torch.sigmoid(x.double())
        return float((w.double() * dw).sum() + 3.0 * (u / u.sum(1, keepdim=True) * slope.double()).sum())

    h = 2.0 ** -6
    got = float((kgw.kgw_moe_route_grad(scores, ids, dw, dloss=dl, slope=slope, score=score, renormalize=renormalize).double() * s).sum())
    w = kgw.kgw_moe_route(scores, k, ids=ids, score=score, renormalize=renormalize)[1]
    size = float((w * dw).abs().sum()) + 3.0
    Z = float(scores.abs().max() * 2)
    assert abs((f(scores + h * s) - f(scores - h * s)) / (2 * h) - got) <= size * ((6 * Z + 60) * U / h + 6 * h * h)


def test_nan_and_infinity():
    scores = make_scores(70, 16, torch.float32, 9)
    clean = kgw.kgw_moe_route(scores, 3)
    scores[5, 2] = float("nan")
    ids, weights, _, loss, _ = kgw.kgw_moe_route(scores, 3)
    assert loss.isnan() and 2 not in ids[5].tolist() and ids.min() >= 0 and ids.max() < 16
    other = torch.arange(70, device=DEV) != 5
    assert torch.equal(ids[other], clean[0][other]) and torch.equal(weights[other], clean[1][other])
    scores[5] = float("nan")
    ids, _, _, loss, _ = kgw.kgw_moe_route(scores, 3)
    assert loss.isnan() and (ids[5] == -1).all() and torch.equal(ids[other], clean[0][other])
    scores[5] = 3e38                                        # far apart and large, still finite
    scores[5, 1::2] = -3e38
    ids, weights, _, loss, _ = kgw.kgw_moe_route(scores, 3)
    assert ids[5].tolist() == [0, 2, 4] and torch.allclose(weights[5], torch.full((3,), 1 / 3, device=DEV), rtol=4 * U, atol=0)
    assert not loss.isnan()
    scores[5] = -200.0                                      # sigmoids that vanish in fp32: 1e-20 keeps the quotient
    _, weights, _, loss, _ = kgw.kgw_moe_route(scores, 3, score="sigmoid")
    assert not weights.isnan().any() and not loss.isnan()


def test_loss_of_even_and_one_sided_use():
    E, k = 8, 2
    scores = torch.zeros((64, E), device=DEV)
    for t in range(64):
        scores[t, t % E] = scores[t, (t + 1) % E] = 1.0
    _, _, counts, loss, _ = kgw.kgw_moe_route(scores, k)
    assert counts.tolist() == [16] * E and abs(float(loss) - 1.0) <= 400 * U
    scores[:] = -40.0
    scores[:, 3] = 40.0
    scores[:, 5] = 39.0
    loss = kgw.kgw_moe_route(scores, k)[3]
    assert abs(float(loss) - E / k) <= 1e-6 * E


@pytest.mark.parametrize("tokens", [60000, 150001])
def test_many_tokens(tokens):
    """More tokens than workgroups take in one round; and the same twice, bit for bit."""
    scores = make_scores(tokens, 64, torch.bfloat16, 4)
    a, b = check(scores, 2), check(scores, 2)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("tokens,experts,k", [(17000, 512, 8), (4301, 2048, 8), (17001, 200, 6), (4200, 900, 5)])
def test_many_tokens_of_wide_rows(tokens, experts, k):
    """The large workgroups of every row length."""
    check(make_scores(tokens, experts, torch.float32, 4), k)


def test_scores_past_four_gigabytes():
    # 2^19 rows 2112 apart: offsets pass 2^30 elements, 2^32 bytes
    tokens, experts = 1 << 19, 64
    wide = torch.empty((tokens, 2112), device=DEV)
    part = wide[:, :experts]
    part.copy_(torch.randn((tokens, experts), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV))
    assert wide.numel() * 4 > 2 ** 32
    got = kgw.kgw_moe_route(part, 4)
    want = kgw.kgw_moe_route(part.contiguous(), 4)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    dw = torch.ones((tokens, 4), device=DEV)
    a = kgw.kgw_moe_route_grad(part, got[0], dw, dloss=got[3], slope=got[4])
    b = kgw.kgw_moe_route_grad(part.contiguous(), got[0], dw, dloss=got[3], slope=got[4])
    assert torch.equal(a, b)
    last = check(part[-100:].contiguous(), 4)
    assert torch.equal(got[0][-100:], last[0]) and torch.equal(got[1][-100:], last[1])


def test_refusals():
    s = torch.zeros((4, 8), device=DEV)
    ids = torch.zeros((4, 2), dtype=torch.int32, device=DEV)
    dw = torch.zeros((4, 2), device=DEV)
    one = torch.zeros((), device=DEV)
    slope = torch.zeros(8, device=DEV)
    route, grad = kgw.kgw_moe_route, kgw.kgw_moe_route_grad
    bad = [lambda: route(s.double(), 2), lambda: route(s[0], 2), lambda: route(s.t(), 2), lambda: route(s.cpu(), 2),
           lambda: route(s, 0), lambda: route(s, 9), lambda: route(torch.zeros((2, 100), device=DEV), 65),
           lambda: route(torch.zeros((2, 2049), device=DEV), 2), lambda: route(s, 2, score="tanh"),
           lambda: route(s, 2, mask=torch.zeros(4, device=DEV)), lambda: route(s, 2, mask=torch.ones(5, dtype=torch.bool, device=DEV)),
           lambda: route(s, 2, mask=torch.ones(4, dtype=torch.bool)), lambda: route(s, 3, ids=ids), lambda: route(s, 2, ids=ids.float()),
           lambda: route(s, 2, ids=ids[:3]), lambda: route(s, 2, ids=ids.cpu()), lambda: route(s.as_strided((4, 8), (4, 1)), 2),
           lambda: grad(s, ids, dw, dloss=one), lambda: grad(s, ids, dw, slope=slope), lambda: grad(s, ids[0], dw),
           lambda: grad(s, ids, dw.double()), lambda: grad(s, ids, dw[:, :1]), lambda: grad(s, ids, dw, dloss=one, slope=slope[:7]),
           lambda: grad(s, ids, dw, dloss=slope, slope=slope), lambda: grad(s, ids, dw, out=torch.zeros((4, 7), device=DEV)),
           lambda: grad(s, ids, dw, out=torch.zeros((4, 8), device=DEV, dtype=torch.bfloat16)),
           lambda: grad(s, ids, dw, dloss=one.cpu(), slope=slope), lambda: grad(s, ids, dw, score="none")]
    for k, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {k} was accepted")
