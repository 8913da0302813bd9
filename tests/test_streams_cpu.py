"""Which stream a call with `stream=` takes its memory from, without a GPU: the library is a stand-in and
the streams are only watched.

The kernels write results and workspaces on the launch stream, so that stream's pool has to hand
them out: a block of the caller's stream may still be in use by work queued there.
"""
import contextlib

import pytest
import torch

import grouped_gemm_expert_offsets_amd as kgw


class Stream:
    def __init__(self, name, handle):
        self.name, self.cuda_stream = name, handle


class Library:
    """Takes every call and wants a workspace for every size."""

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return lambda *a: 512
        if name == "kgw_moe_rows":
            return lambda tokens, topk, experts, align: 4 * align
        return lambda *a: kgw.KGW_SUCCESS


@pytest.fixture
def watch(monkeypatch):
    """(launch stream, [(current stream, shape) of every allocation], {tensor: streams it was recorded on})."""
    caller, launch = Stream("caller", 1), Stream("launch", 2)
    current, made, recorded = [caller], [], {}

    @contextlib.contextmanager
    def entered(s):
        current.append(s)
        yield
        current.pop()

    real = torch.empty

    def empty(*shape, dtype=None, device=None):
        t = real(*shape, dtype=dtype)
        made.append((current[-1].name, t))
        return t

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", entered)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[-1])
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, s: recorded.setdefault(t.untyped_storage().data_ptr(), set()).add(s.name))
    monkeypatch.setattr(kgw, "_on_gpu", lambda t, what: t.device)
    monkeypatch.setattr(kgw, "load_library", lambda: Library())
    return launch, made, recorded


def index(*shape):
    return torch.zeros(shape, dtype=torch.int32)


LAYER_CALLS = {
    "sort": (lambda s, t: kgw.kgw_moe_sort(t["ids"], 4, stream=s), ("ids",), 1),
    "permute": (lambda s, t: kgw.kgw_moe_permute(t["x"], t["row_of"], t["src_of"], stream=s), ("x", "row_of", "src_of"), 1),
    "unpermute": (lambda s, t: kgw.kgw_moe_unpermute(t["y"], t["row_of"], t["w"], stream=s), ("y", "row_of", "w"), 1),
    "unpermute_grad": (lambda s, t: kgw.kgw_moe_unpermute_grad(t["x"], t["y"], t["row_of"], t["src_of"], t["w"], stream=s),
                       ("x", "y", "row_of", "src_of", "w"), 2),
    "newton_schulz": (lambda s, t: kgw.kgw_newton_schulz(t["y"], stream=s), ("y",), 2),
}


def tensors():
    return dict(ids=index(6, 2), row_of=index(6, 2), src_of=index(128), x=torch.zeros(6, 16), y=torch.zeros(128, 16),
                w=torch.zeros(6, 2))


@pytest.mark.parametrize("name", LAYER_CALLS)
def test_memory_comes_from_the_launch_stream(watch, name):
    launch, made, recorded = watch
    call, used, count = LAYER_CALLS[name]
    inputs = tensors()
    call(launch, inputs)
    assert [who for who, _ in made] == ["launch"] * count
    for _, t in made:                                     # the caller's stream uses what comes back
        assert "caller" in recorded[t.untyped_storage().data_ptr()]
    for k in used:                                        # and may let go of what it gave
        assert "launch" in recorded[inputs[k].untyped_storage().data_ptr()], k


@pytest.mark.parametrize("name", LAYER_CALLS)
def test_without_a_stream_nothing_changes_hands(watch, monkeypatch, name):
    launch, made, recorded = watch
    monkeypatch.setattr(kgw, "_launch_stream", lambda stream, device: 0)
    call, _, count = LAYER_CALLS[name]
    call(None, tensors())
    assert [who for who, _ in made] == ["caller"] * count and not recorded
