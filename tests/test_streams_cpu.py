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


def operands():
    offsets = torch.tensor([256, 512], dtype=torch.int32)
    bytes_ = lambda *shape: torch.zeros(shape, dtype=torch.uint8)  # noqa: E731
    return dict(a=torch.zeros((32, 512), dtype=torch.bfloat16), b=torch.zeros((512, 64), dtype=torch.bfloat16),
                a8=bytes_(32, 512), b8=bytes_(512, 64), sa=bytes_(4, 32), sb=bytes_(4, 64), offsets=offsets,
                a4=bytes_(32, 256), b4=bytes_(64, 256), sa4=index(4, 32), sb4=index(4, 64),
                rows=torch.zeros((256, 64), dtype=torch.bfloat16), w=torch.zeros((2, 64, 64), dtype=torch.bfloat16),
                rows8=bytes_(256, 128), w8=bytes_(2, 64, 128), srows=bytes_(1, 256), sw=bytes_(2, 1, 64),
                out=torch.zeros((2, 32, 64)), one=torch.zeros((32, 64)))


# call, the caller's tensors it reads or writes, allocations
PRODUCT_CALLS = {
    "wgrad_bf16": (lambda s, t: kgw.kgw_wgrad_bf16(t["a"], t["b"], t["offsets"], stream=s), ("a", "b", "offsets"), 2),
    "wgrad_bf16_noalloc": (lambda s, t: kgw.kgw_wgrad_bf16_noalloc(t["a"], t["b"], t["offsets"], t["out"], stream=s),
                           ("a", "b", "offsets", "out"), 0),
    "wgrad_bf16_ex": (lambda s, t: kgw.kgw_wgrad_bf16_ex(t["a"], t["b"], t["offsets"], stream=s), ("a", "b", "offsets"), 2),
    "wgrad_bf16_ex outs": (lambda s, t: kgw.kgw_wgrad_bf16_ex(t["a"], t["b"], t["offsets"], outs=[t["one"], None], stream=s),
                           ("a", "b", "offsets", "one"), 1),
    "wgrad_fp8": (lambda s, t: kgw.kgw_wgrad_fp8(t["a8"], t["sa"], t["b8"], t["sb"], t["offsets"], stream=s),
                  ("a8", "sa", "b8", "sb", "offsets"), 2),
    "wgrad_fp8_native": (lambda s, t: kgw.kgw_wgrad_fp8_native(t["a8"], t["sa"], t["b8"], t["sb"], t["offsets"], stream=s),
                         ("a8", "sa", "b8", "sb", "offsets"), 2),
    "wgrad_fp8_ex": (lambda s, t: kgw.kgw_wgrad_fp8_ex(t["a8"], t["sa"], t["b8"], t["sb"], t["offsets"], out=t["out"],
                                                       stream=s), ("a8", "sa", "b8", "sb", "offsets", "out"), 1),
    "wgrad_fp4": (lambda s, t: kgw.kgw_wgrad_fp4(t["a4"], t["sa4"], t["b4"], t["sb4"], t["offsets"], stream=s),
                  ("a4", "sa4", "b4", "sb4", "offsets"), 2),
    "quantize_fp8": (lambda s, t: kgw.kgw_quantize_fp8(t["a"], 1, stream=s), ("a",), 2),
    "quantize_fp4": (lambda s, t: kgw.kgw_quantize_fp4(t["a"], 1, stream=s), ("a",), 2),
    "mgrouped_bf16": (lambda s, t: kgw.kgw_mgrouped_bf16(t["rows"], t["w"], offsets=t["offsets"], stream=s),
                      ("rows", "w", "offsets"), 1),
    "mgrouped_fp8": (lambda s, t: kgw.kgw_mgrouped_fp8(t["rows8"], t["srows"], t["w8"], t["sw"], offsets=t["offsets"],
                                                       stream=s), ("rows8", "srows", "w8", "sw", "offsets"), 1),
    "check_offsets": (lambda s, t: kgw.kgw_check_offsets(t["offsets"], 512, 256, stream=s), ("offsets",), 1),
}


@pytest.mark.parametrize("name", PRODUCT_CALLS)
def test_products_take_memory_from_the_launch_stream(watch, name):
    launch, made, recorded = watch
    call, used, count = PRODUCT_CALLS[name]
    inputs = operands()
    call(launch, inputs)
    assert [who for who, _ in made] == ["launch"] * count
    for _, t in made:
        assert "caller" in recorded[t.untyped_storage().data_ptr()]
    for k in used:
        assert "launch" in recorded[inputs[k].untyped_storage().data_ptr()], k


@pytest.mark.parametrize("name", LAYER_CALLS)
def test_without_a_stream_nothing_changes_hands(watch, monkeypatch, name):
    launch, made, recorded = watch
    monkeypatch.setattr(kgw, "_launch_stream", lambda stream, device: 0)
    call, _, count = LAYER_CALLS[name]
    call(None, tensors())
    assert [who for who, _ in made] == ["caller"] * count and not recorded
