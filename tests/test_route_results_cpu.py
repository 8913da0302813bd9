"""The router's results are the caller's: each in memory of its own, to be kept, changed in place and saved for a backward
pass apart from the others (no GPU; the library is a stand-in)."""
import pytest
import torch

import grouped_gemm_expert_offsets_amd as kgw
from test_streams_cpu import Library, watch  # noqa: F401  (a fixture)

TOKENS, E, K = 6, 16, 2


@pytest.fixture
def on_cpu(monkeypatch):
    monkeypatch.setattr(kgw, "_on_gpu", lambda t, what: t.device)
    monkeypatch.setattr(kgw, "load_library", lambda: Library())
    monkeypatch.setattr(kgw, "_launch_stream", lambda stream, device: 0)


def check_own(results):
    ids, weights, counts, loss, slope = results
    shapes = [((TOKENS, K), torch.int32), ((TOKENS, K), torch.float32), ((E,), torch.int32), ((), torch.float32), ((E,), torch.float32)]
    assert [(tuple(t.shape), t.dtype) for t in results] == shapes and all(t.is_contiguous() for t in results)
    assert len({t.untyped_storage().data_ptr() for t in results}) == 5
    # nothing of the launch's scratch, nor of another result
    assert all(t.untyped_storage().nbytes() == t.numel() * t.element_size() for t in results)
    assert not any(t._is_view() for t in results)
    before = [t._version for t in results]
    loss.zero_()
    assert [t._version - v for t, v in zip(results, before)] == [0, 0, 0, 1, 0]


@pytest.mark.parametrize("given", [False, True])
def test_own_memory(on_cpu, given):
    ids = torch.zeros((TOKENS, K), dtype=torch.int32) if given else None
    check_own(kgw.kgw_moe_route(torch.zeros(TOKENS, E), K, ids=ids))


def test_own_memory_from_the_launch_stream(watch, monkeypatch):  # noqa: F811
    """With `stream=` every result is made while the launch stream is the current one, and kept for the caller's."""
    launch, made, recorded = watch
    real, current = torch.empty_strided, lambda: torch.cuda.current_stream().name
    results = []

    def strided(*args, **kw):
        t = real(*args, **kw)
        results.append((current(), t))
        return t

    monkeypatch.setattr(torch, "empty_strided", strided)
    got = kgw.kgw_moe_route(torch.zeros(TOKENS, E), K, stream=launch)
    check_own(got)
    made = made + results
    assert {id(t) for t in got} <= {id(t) for _, t in made} and {name for name, _ in made} == {"launch"}
    for _, t in made:
        assert "caller" in recorded[t.untyped_storage().data_ptr()]


class Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, scores):
        ids, weights, counts, loss, slope = kgw.kgw_moe_route(scores, K)
        ctx.save_for_backward(scores, ids, slope)
        ctx.mark_non_differentiable(ids, counts)
        return ids, weights.fill_(0.5), counts, loss.fill_(1.0)

    @staticmethod
    def backward(ctx, dids, dweights, dcounts, dloss):
        scores, ids, slope = ctx.saved_tensors
        return torch.full_like(scores, float(dweights.sum() + dloss))


@pytest.mark.parametrize("change", ["weights", "loss", "counts"])
def test_changed_in_place_under_autograd(on_cpu, change):
    scores = torch.zeros((TOKENS, E), requires_grad=True)
    ids, weights, counts, loss = Route.apply(scores)
    if change == "weights":
        weights *= 3.0
    elif change == "loss":
        loss *= 0.25
    else:
        counts.zero_()                                      # (summed over ranks, say)
    (weights.sum() + loss).backward()
    assert (scores.grad == (3 if change == "weights" else 1) * TOKENS * K + (0.25 if change == "loss" else 1.0)).all()
