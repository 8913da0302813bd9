"""One training step of a gated mixture-of-experts layer that keeps its activations in 8 bits.

    python examples/moe_fp8_layer_step.py [--steps N]

Router scores become experts, weights and a balance loss (kgw_moe_route).  Tokens are sorted and brought into expert order
(kgw_moe_sort, kgw_moe_permute) and quantised once (kgw_quantize_fp8): the first product reads them (kgw_mgrouped_fp8)
and the backward pass keeps nothing else of them.  The gated activation keeps its input in 8 bits and hands its result to
the second product in 8 bits (kgw_moe_act_fp8); results come back weighted (kgw_moe_unpermute).

Backward: kgw_moe_unpermute_grad, the data gradient of the second product (kgw_mgrouped_bf16, bf16 weights), the
activation's gradient from the kept values, with its result once more for the weight gradient (kgw_moe_act_fp8_grad),
weight gradients from the 8-bit rows (kgw_wgrad_fp8_rows), the data gradient of the first product, kgw_moe_unpermute,
and the router's gradient with that of the balance loss (kgw_moe_route_grad).

For a row of hidden size H and inner size I the step keeps H + 3 I bytes (and a scale for every 128 of them) where bf16
copies of x, h and act would be 2 H + 6 I.  The layer learns to reproduce a fixed random layer of the same shape.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import grouped_gemm_expert_offsets_amd as kgw  # noqa: E402

ALIGN = kgw.FP8_TOKEN_ALIGN       # rows of one expert: whole blocks of the grouped products
BALANCE = 0.01                    # weight of the balance loss


def quantise_weights(w):
    """w (E, n, k) bf16 -> e4m3 codes (E, n, k) and scales (E, k / 128, n), blocks along k."""
    E, n, k = w.shape
    codes, scales = kgw.kgw_quantize_fp8(w.reshape(E * n, k), 1)
    return codes.view(E, n, k), scales.view(k // 128, E, n).transpose(0, 1).contiguous()


class GatedMoeLayer:
    """y = sum over the topk experts e of p_e * (silu(x G_e) * (x U_e)) D_e, weights stored as the forward products take them:
    w1 (E, 2 inner, hidden) = [G; U] transposed, w2 (E, hidden, inner) = D transposed."""

    def __init__(self, experts, hidden, inner, topk, device, seed):
        g = torch.Generator(device=device).manual_seed(seed)
        self.topk = topk
        self.router = torch.randn((hidden, experts), generator=g, device=device) * hidden ** -0.5
        self.w1 = torch.randn((experts, 2 * inner, hidden), generator=g, device=device) * hidden ** -0.5
        self.w2 = torch.randn((experts, hidden, inner), generator=g, device=device) * inner ** -0.5

    def forward(self, x, mask=None):
        """Output, balance loss and what the backward pass needs; mask (tokens,): False for padding."""
        scores = x.float() @ self.router
        E = self.router.shape[1]
        ids, weights, _, loss, slope = kgw.kgw_moe_route(scores, self.topk, mask=mask)
        _, offsets, row_of, src_of = kgw.kgw_moe_sort(ids, E, alignment=ALIGN)
        rows8, rows_scales = kgw.kgw_quantize_fp8(kgw.kgw_moe_permute(x, row_of, src_of), 1)
        w1, w2 = self.w1.bfloat16(), self.w2.bfloat16()
        # rows past the last offset belong to no expert: nothing below reads or writes them
        h = torch.empty((rows8.shape[0], w1.shape[1]), dtype=torch.bfloat16, device=x.device)
        kgw.kgw_mgrouped_fp8(rows8, rows_scales, *quantise_weights(w1), offsets=offsets, out=h)
        act8, act_scales, kept, kept_scales = kgw.kgw_moe_act_fp8(h, offsets=offsets, fp8=True)
        y = torch.empty((rows8.shape[0], x.shape[1]), dtype=torch.bfloat16, device=x.device)
        kgw.kgw_mgrouped_fp8(act8, act_scales, *quantise_weights(w2), offsets=offsets, out=y)
        out = kgw.kgw_moe_unpermute(y, row_of, weights)
        return out, loss, (x, scores, mask, ids, weights, slope, offsets, row_of, src_of, rows8, rows_scales, kept,
                           kept_scales, y, w1, w2)

    def backward(self, dout, dloss, saved):
        """Gradients of w1, w2, the router and x for dout (tokens, hidden) bf16 and dloss, a float32 tensor of one value."""
        x, scores, mask, ids, weights, slope, offsets, row_of, src_of, rows8, rows_scales, kept, kept_scales, y, w1, w2 = saved
        dy, dweights = kgw.kgw_moe_unpermute_grad(dout, y, row_of, src_of, weights)
        dact = torch.empty((dy.shape[0], w2.shape[2]), dtype=torch.bfloat16, device=x.device)
        kgw.kgw_mgrouped_bf16(dy, w2, offsets=offsets, layout="nn", out=dact)
        dh, _, act8, act_scales = kgw.kgw_moe_act_fp8_grad(dact, kept, kept_scales, offsets=offsets, again=True, again_fp8=True)
        # (E, inner, hidden) and (E, hidden, 2 inner): the transposes of the stored weights
        dw2 = kgw.kgw_wgrad_fp8_rows(act8, act_scales, dy, offsets)
        dw1 = kgw.kgw_wgrad_fp8_rows(rows8, rows_scales, dh, offsets)
        drows = torch.empty_like(dy)
        kgw.kgw_mgrouped_bf16(dh, w1, offsets=offsets, layout="nn", out=drows)
        dscores = kgw.kgw_moe_route_grad(scores, ids, dweights, dloss=dloss, slope=slope, mask=mask)
        dx = kgw.kgw_moe_unpermute(drows, row_of).float() + dscores @ self.router.t()
        return dw1.transpose(1, 2), dw2.transpose(1, 2), x.float().t() @ dscores, dx

    def update(self, dw1, dw2, drouter, lr):
        for w, dw in ((self.w1, dw1), (self.w2, dw2)):
            step = kgw.kgw_newton_schulz(dw.transpose(1, 2), out_dtype=torch.bfloat16).transpose(1, 2)
            w.sub_(lr * max(1.0, w.shape[1] / w.shape[2]) ** 0.5 * step)
        self.router.sub_(lr * drouter)


def train(steps=10, tokens=1536, experts=8, hidden=512, inner=256, topk=2, lr=0.02, device="cuda", seed=0):
    """The losses and balance losses of `steps` steps."""
    teacher = GatedMoeLayer(experts, hidden, inner, topk, device, seed + 1)
    layer = GatedMoeLayer(experts, hidden, inner, topk, device, seed + 2)
    layer.router.copy_(teacher.router)
    g = torch.Generator(device=device).manual_seed(seed)
    x = torch.randn((tokens, hidden), generator=g, device=device).bfloat16()
    target = teacher.forward(x)[0].float()
    scale = 1024.0                                        # keeps bf16 gradients away from zero
    losses = []
    for _ in range(steps):
        out, balance, saved = layer.forward(x)
        diff = out.float() - target
        losses.append((float(diff.square().mean()), float(balance)))
        dout = (2.0 / diff.numel() * diff * scale).bfloat16()
        dw1, dw2, drouter, _ = layer.backward(dout, torch.full((), BALANCE * scale, device=device), saved)
        layer.update(dw1, dw2, drouter / scale, lr)
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=10)
    for k, (loss, balance) in enumerate(train(ap.parse_args().steps)):
        print(f"step {k:3d}  loss {loss:.5f}  balance {balance:.4f}")
