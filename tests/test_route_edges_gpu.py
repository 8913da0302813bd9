"""The router where its numbers end: gradients of losses that are not finite."""
import pytest
import torch

import grouped_gemm_expert_offsets_amd as kgw
from test_route_gpu import make_scores

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
