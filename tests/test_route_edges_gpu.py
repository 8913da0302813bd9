"""The router where its numbers end: gradients of losses that are not finite, and given experts whose shares vanish beside
the largest.  Tolerances are those of test_route_gpu.py."""
import pytest
import torch

import grouped_gemm_expert_offsets_amd as kgw
from test_route_gpu import DTYPES, check, make_scores

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs an MI355X")]

DEV = "cuda"
INF, NAN = float("inf"), float("nan")
# one of every number of lanes, rows of fewer than four, chosen experts beyond a row's lanes
SHAPES = [(9, 3, 2), (40, 30, 7), (70, 61, 20), (33, 128, 4), (50, 250, 8), (21, 500, 24), (10, 900, 5), (7, 2048, 64)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("tokens,experts,k", SHAPES)
def test_gradient_is_zero_where_nothing_is_chosen(tokens, experts, k, renormalize, score):
    """A masked token and a score of -inf have the gradient zero whatever is not finite elsewhere: in the loss's gradient, in
    a chosen weight's, among the scores."""
    g = torch.Generator().manual_seed(experts)
    scores = make_scores(tokens, experts, torch.float32, 3)
    scores[(torch.rand((tokens, experts), generator=g) < 0.3).to(DEV)] = -INF
    scores[2] = -INF
    mask = (torch.rand(tokens, generator=g) < 0.7).to(DEV)
    mask[1:6] = torch.tensor([False, True, True, True, True], device=DEV)
    scores[1] = NAN                                         # padding holds anything
    kw = dict(mask=mask, score=score, renormalize=renormalize)
    ids, _, _, _, slope = kgw.kgw_moe_route(scores, k, **kw)
    dw = torch.randn((tokens, k), generator=g).to(DEV)
    none = ~mask[:, None] | (scores == -INF)
    clean = kgw.kgw_moe_route_grad(scores, ids, dw, dloss=torch.ones((), device=DEV), slope=slope, **kw)
    assert (clean[none] == 0).all() and clean.isfinite().all()
    for bad in (INF, -INF, NAN):
        got = kgw.kgw_moe_route_grad(scores, ids, dw, dloss=torch.tensor(bad, device=DEV), slope=slope, **kw)
        assert (got[none] == 0).all(), bad
        assert not got[mask & (ids[:, 0] >= 0)].isfinite().all()
        wrong = dw.clone()
        wrong[3, 0] = bad
        got = kgw.kgw_moe_route_grad(scores, ids, wrong, dloss=torch.ones((), device=DEV), slope=slope, **kw)
        others = torch.arange(tokens, device=DEV) != 3
        assert (got[none] == 0).all() and torch.equal(got[others], clean[others])
    scores[4, int((scores[4] > -INF).nonzero()[-1])] = NAN
    got = kgw.kgw_moe_route_grad(scores, ids, dw, dloss=torch.ones((), device=DEV), slope=slope, **kw)
    none = ~mask[:, None] | (scores == -INF)
    others = torch.arange(tokens, device=DEV) != 4
    assert (got[none] == 0).all() and torch.equal(got[others], clean[others])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("gap", [60.0, 100.0, 300.0])
@pytest.mark.parametrize("tokens,experts,k", SHAPES)
def test_given_experts_far_below_the_largest(tokens, experts, k, gap, dtype):
    """Experts chosen elsewhere need not hold the largest score.  Their shares vanish in fp32 beside it; made to sum to one they
    do not: weights and gradients are those of the chosen alone."""
    g = torch.Generator().manual_seed(experts + int(gap))
    scores = make_scores(tokens, experts, dtype, 6)
    ids = torch.rand((tokens, experts), generator=g).topk(k, dim=1).indices
    top = ids[:, :1].to(DEV)
    ids[::3, 0] = ids[::3, 1]                               # every third token's largest is not among its chosen
    scores.scatter_add_(1, top, torch.full((tokens, 1), gap, dtype=dtype, device=DEV))
    ids = ids.int().to(DEV)
    _, weights, *_ = check(scores, k, ids=ids)
    assert bool(((weights.sum(1) - 1).abs() <= 1e-5).all())


def test_given_experts_at_the_ends_of_the_range():
    scores = torch.full((3, 40), -3e38, device=DEV)
    scores[:, 7] = 3e38
    scores[1, 3] = scores[2, :] = -INF
    scores[2, 7] = 1.0
    ids = torch.tensor([[1, 2, 3, 4]] * 3, device=DEV)
    got, weights, _, loss, _ = kgw.kgw_moe_route(scores, 4, ids=ids)
    assert got.tolist() == [[1, 2, 3, 4], [1, 2, -1, 4], [-1] * 4]
    third = torch.tensor(1.0) / 3
    want = torch.stack((torch.full((4,), 0.25), torch.stack((third, third, torch.tensor(0.0), third)), torch.zeros(4)))
    assert torch.allclose(weights.cpu(), want, rtol=2.0 ** -22, atol=0) and not loss.isnan()
    dw = torch.tensor([[1.0, 2.0, 3.0, 4.0]] * 3, device=DEV)
    grad = kgw.kgw_moe_route_grad(scores, got, dw).cpu()
    # q (dw - sum q dw) of the chosen, q = 1/4 and 1/3
    assert torch.allclose(grad[0, 1:5], torch.tensor([-1.5, -0.5, 0.5, 1.5]) / 4, rtol=2.0 ** -20, atol=0)
    assert torch.allclose(grad[1, 1:5], torch.tensor([1 - 7 / 3, 2 - 7 / 3, 0, 4 - 7 / 3]) / 3, rtol=2.0 ** -18, atol=0)
    assert not grad[2].any() and not grad[:2, 5:].any()
