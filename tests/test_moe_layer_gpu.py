"""The example's training step: its gradients against torch's autograd of the same layer in 64 bits on
the CPU, and its loss, which has to fall.

Every tensor between two operators is rounded to bf16 (half a step: 2^-8 of the value, 2^-8 / sqrt(3) in the mean
square).  A weight gradient is a product of two such chains of at most 6 roundings each, so its error
against the unrounded gradient is within 12 * 2^-8 / sqrt(3) = 2.7e-2 of its norm; dx passes through 8.
"""
import importlib.util
import os

import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs an MI355X")]

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
_spec = importlib.util.spec_from_file_location("moe_layer_step", os.path.join(ROOT, "examples", "moe_layer_step.py"))
example = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(example)


def test_gradients():
    tokens, experts, hidden, inner, topk = 200, 4, 128, 64, 2
    layer = example.MoeLayer(experts, hidden, inner, topk, "cuda", 3)
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((tokens, hidden), generator=g, device="cuda").bfloat16()
    dout = torch.randn((tokens, hidden), generator=g, device="cuda").bfloat16()
    out, saved = layer.forward(x)
    got = layer.backward(dout, saved)
    ids = saved[1].cpu()

    xd = x.double().cpu().requires_grad_()
    w1 = layer.w1.bfloat16().double().cpu().requires_grad_()
    w2 = layer.w2.bfloat16().double().cpu().requires_grad_()
    router = layer.router.double().cpu().requires_grad_()
    p = torch.softmax((xd.detach() @ router).gather(1, ids), dim=1)   # the router's scores pass no gradient to x here
    want_out = torch.zeros((tokens, hidden), dtype=torch.float64)
    for j in range(topk):
        h = torch.relu(torch.bmm(xd[:, None], w1[ids[:, j]]))
        want_out = want_out + p[:, j, None] * torch.bmm(h * h, w2[ids[:, j]])[:, 0]
    (want_out * dout.double().cpu()).sum().backward()
    unit = 2.0 ** -8 / 3 ** 0.5
    rel = lambda a, b: float((a.double().cpu() - b).norm() / b.norm())  # noqa: E731
    assert rel(out, want_out.detach()) <= 6 * unit
    for a, b, roundings in zip(got, (w1.grad, w2.grad, router.grad, xd.grad), (12, 12, 12, 8)):
        assert rel(a, b) <= roundings * unit


def test_loss_falls():
    losses = example.train(steps=8)
    assert losses[-1] < 0.7 * losses[0] and all(b < a for a, b in zip(losses, losses[1:]))
