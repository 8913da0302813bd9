"""The router, the 8-bit activation and the weight gradients from 8-bit rows in a run together, as the example's training step
has them: gradients against torch's autograd of the same layer in 64 bits, one captured graph replayed on new
tokens, calls with `stream=`, and two graphs whose workspaces are their own.

Tolerance of the gradients: e4m3 rounds by at most 2^-4 of a value, 2^-4 / sqrt(3) = 3.6e-2 in the mean square, bf16 by 2^-8.
A weight gradient is a product of two chains; the forward one (x, w1, h, act, w2) has at most 4 e4m3 roundings of which
each enters a product whose other terms are independent, the backward one (dy, dact, dh) is bf16 but reads h once more in
e4m3.  With 6 roundings in all the error is within 6 * 3.6e-2 = 0.22 of the norm.
"""
import importlib.util
import os

import pytest
import torch

import grouped_gemm_expert_offsets_amd as kgw

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs an MI355X")]

DEV = "cuda"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
_spec = importlib.util.spec_from_file_location("moe_fp8_layer_step", os.path.join(ROOT, "examples", "moe_fp8_layer_step.py"))
example = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(example)


@pytest.mark.parametrize("masked", [False, True])
def test_gradients(masked):
    tokens, experts, hidden, inner, topk = 200, 4, 128, 128, 2
    layer = example.GatedMoeLayer(experts, hidden, inner, topk, DEV, 3)
    g = torch.Generator(device=DEV).manual_seed(4)
    x = torch.randn((tokens, hidden), generator=g, device=DEV).bfloat16()
    dout = torch.randn((tokens, hidden), generator=g, device=DEV).bfloat16()
    mask = torch.rand(tokens, generator=g, device=DEV) < 0.8 if masked else None
    dloss = torch.tensor(50.0, device=DEV)
    out, loss, saved = layer.forward(x, mask)
    got = layer.backward(dout, dloss, saved)
    ids = saved[3].cpu().long()
    here = (ids >= 0) if mask is None else mask.cpu()[:, None].expand(-1, topk)
    assert torch.equal(ids >= 0, here)
    ids = ids.clamp(min=0)

    xd = x.double().cpu().requires_grad_()
    w1 = layer.w1.bfloat16().double().cpu().requires_grad_()
    w2 = layer.w2.bfloat16().double().cpu().requires_grad_()
    router = layer.router.double().cpu().requires_grad_()
    scores = xd @ router
    p = torch.softmax(scores.gather(1, ids), dim=1) * here
    want_out = torch.zeros((tokens, hidden), dtype=torch.float64)
    for j in range(topk):
        h = torch.bmm(w1[ids[:, j]], xd[:, :, None])[:, :, 0]
        act = torch.nn.functional.silu(h[:, :inner]) * h[:, inner:]
        want_out = want_out + p[:, j, None] * torch.bmm(w2[ids[:, j]], act[:, :, None])[:, :, 0]
    part = here.any(1)
    counts = torch.bincount(ids[here], minlength=experts).double()
    shares = torch.softmax(scores, dim=1)[part].sum(0)
    want_loss = (shares * counts).sum() * experts / (topk * int(part.sum()) ** 2)
    ((want_out * dout.double().cpu()).sum() + 50.0 * want_loss).backward()
    rel = lambda a, b: float((a.double().cpu() - b).norm() / b.norm())  # noqa: E731
    assert abs(float(loss) - float(want_loss.detach())) <= 1e-5 * float(want_loss.detach())
    assert rel(out, want_out.detach()) <= 0.22
    for a, b in zip(got, (w1.grad, w2.grad, router.grad, xd.grad)):
        assert rel(a, b) <= 0.22


def test_example_runs():
    losses = example.train(steps=3)
    assert len(losses) == 3 and all(torch.isfinite(torch.tensor(v)).all() for v in losses)


TOKENS, E, K, HIDDEN, INNER = 300, 8, 2, 256, 128


def inputs(seed):
    g = torch.Generator().manual_seed(seed)
    new = lambda *s: torch.randn(s, generator=g).to(DEV)  # noqa: E731
    return (new(TOKENS, E), (torch.rand(TOKENS, generator=g) < 0.9).to(DEV), new(TOKENS, HIDDEN).bfloat16(),
            (new(E, HIDDEN, 2 * INNER) * HIDDEN ** -0.5).bfloat16(), new(TOKENS, 2 * INNER).bfloat16())


def step(scores, mask, x, w, dh_tokens, stream=None):
    """Every new operator once, each on the results of the one before; nothing is looked at on the host."""
    s = stream
    ids, weights, counts, loss, slope = kgw.kgw_moe_route(scores, K, mask=mask, stream=s)
    _, offsets, row_of, src_of = kgw.kgw_moe_sort(ids, E, stream=s)
    rows = kgw.kgw_moe_permute(x, row_of, src_of, stream=s)
    q, qs = kgw.kgw_quantize_fp8(rows, 1, stream=s)
    h = kgw.kgw_moe_permute(dh_tokens, row_of, src_of, stream=s)
    kgw.kgw_mgrouped_bf16(rows, w, offsets=offsets, layout="nn", out=h, stream=s)
    y, ys, kept, ks = kgw.kgw_moe_act_fp8(h, fp8=True, stream=s)
    dy = kgw.kgw_moe_permute(x, row_of, src_of, stream=s)[:, :INNER]
    dh, dhs, y2, y2s = kgw.kgw_moe_act_fp8_grad(dy, kept, ks, fp8=True, again=True, stream=s)
    dw1 = kgw.kgw_wgrad_fp8_rows(q, qs, dh, offsets, sb=dhs, stream=s)
    dw2 = kgw.kgw_wgrad_fp8_rows(y2, y2s, rows, offsets, stream=s)
    dscores = kgw.kgw_moe_route_grad(scores, ids, weights, dloss=loss, slope=slope, mask=mask, stream=s)
    return ids, weights, counts, loss, slope, y, ys, kept, ks, dh, dhs, y2, y2s, dw1, dw2, dscores


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_graph_replays():
    held = inputs(1)
    want = step(*held)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*held)
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):                                      # two graphs, each with workspaces of its own
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = step(*held)
        graphs.append((graph, outs))
    for r in range(4):
        for t, new in zip(held, inputs(10 + r)):
            t.copy_(new)
        want = step(*held)
        torch.cuda.synchronize()
        for _, outs in graphs:
            for t in outs:
                t.fill_(77)
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert all(same(outs, want) for _, outs in graphs), r


def test_results_on_a_given_stream():
    want = step(*inputs(2))
    s = torch.cuda.Stream()
    for _ in range(3):
        given = inputs(2)                                   # written on the caller's stream ...
        s.wait_stream(torch.cuda.current_stream())
        got = step(*given, stream=s)
        del given                                           # ... let go of before the call's work is done ...
        again = inputs(2)                                   # ... and its memory written anew
        torch.cuda.current_stream().wait_stream(s)
        assert same(got, want)
        del again


def test_two_calls_at_once():
    """The same operators on two streams, each call with memory of its own."""
    one, two = inputs(3), inputs(4)
    want = step(*one), step(*two)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        with torch.cuda.stream(a):
            x = step(*one)
        with torch.cuda.stream(b):
            y = step(*two)
        got.append((x, y))
    torch.cuda.synchronize()
    assert all(same(x, want[0]) and same(y, want[1]) for x, y in got)
