"""One training step of a mixture-of-experts layer through the package's own operators.

    python examples/moe_layer_step.py [--steps N]

Tokens are routed (kgw_moe_sort), brought into expert order (kgw_moe_permute), run through the
experts' two products (kgw_mgrouped_bf16), and brought back weighted (kgw_moe_unpermute).  Backward
takes the same way: kgw_moe_unpermute_grad, the products' data gradients (kgw_mgrouped_bf16, nn), their
weight gradients (kgw_wgrad_bf16_ex on the token rows as they lie) and kgw_moe_unpermute for the
tokens' gradient.  The weight gradients, orthogonalised by kgw_newton_schulz, move the weights; router
scores take a plain gradient step.  The activation and the softmax over the chosen experts are torch's.

The layer learns to reproduce a fixed random layer of the same shape, so the loss falls.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import grouped_gemm_expert_offsets_amd as kgw  # noqa: E402

ALIGN = kgw.BF16_TOKEN_ALIGN      # rows of one expert: whole weight-gradient steps


class MoeLayer:
    """y = sum over the topk experts e of p_e * relu(x W1_e) ** 2 W2_e."""

    def __init__(self, experts, hidden, inner, topk, device, seed):
        g = torch.Generator(device=device).manual_seed(seed)
        self.topk = topk
        self.router = torch.randn((hidden, experts), generator=g, device=device) * hidden ** -0.5
        self.w1 = torch.randn((experts, hidden, inner), generator=g, device=device) * hidden ** -0.5
        self.w2 = torch.randn((experts, inner, hidden), generator=g, device=device) * inner ** -0.5

    def forward(self, x):
        """Output and what the backward pass needs."""
        scores = x.float() @ self.router
        top, ids = scores.topk(self.topk, dim=1)
        p = torch.softmax(top, dim=1)
        counts, offsets, row_of, src_of = kgw.kgw_moe_sort(ids, self.router.shape[1], alignment=ALIGN)
        rows = kgw.kgw_moe_permute(x, row_of, src_of)
        w1, w2 = self.w1.bfloat16(), self.w2.bfloat16()
        # rows past the last offset belong to no expert: the products neither read nor write them, and nothing has to
        # be read back to the host
        h = torch.empty((rows.shape[0], w1.shape[2]), dtype=torch.bfloat16, device=x.device)
        kgw.kgw_mgrouped_bf16(rows, w1, offsets=offsets, layout="nn", out=h)
        act = torch.relu(h).square()
        y = torch.empty_like(rows)
        kgw.kgw_mgrouped_bf16(act, w2, offsets=offsets, layout="nn", out=y)
        out = kgw.kgw_moe_unpermute(y, row_of, p)
        return out, (x, ids, p, offsets, row_of, src_of, rows, h, act, y, w1, w2)

    def backward(self, dout, saved):
        """Gradients of the weights, the router and x for dout (tokens, hidden) bf16."""
        x, ids, p, offsets, row_of, src_of, rows, h, act, y, w1, w2 = saved
        dy, dp = kgw.kgw_moe_unpermute_grad(dout, y, row_of, src_of, p)
        dact = torch.empty_like(act)
        kgw.kgw_mgrouped_bf16(dy, w2, offsets=offsets, layout="nt", out=dact)
        dw2 = kgw.kgw_wgrad_bf16_ex(act, dy, offsets, a_major="m")
        dh = (2 * dact.float() * torch.relu(h).float()).bfloat16()
        drows = torch.empty_like(rows)
        kgw.kgw_mgrouped_bf16(dh, w1, offsets=offsets, layout="nt", out=drows)
        dw1 = kgw.kgw_wgrad_bf16_ex(rows, dh, offsets, a_major="m")
        dx = kgw.kgw_moe_unpermute(drows, row_of)
        dtop = p * (dp - (p * dp).sum(1, keepdim=True))
        dscores = torch.zeros((x.shape[0], self.router.shape[1]), device=x.device).scatter_(1, ids, dtop)
        return dw1, dw2, x.float().t() @ dscores, dx

    def update(self, dw1, dw2, drouter, lr):
        for w, dw in ((self.w1, dw1), (self.w2, dw2)):
            # one orthogonal step per expert, of the same size for every shape; an expert without tokens stays
            w.sub_(lr * max(1.0, w.shape[1] / w.shape[2]) ** 0.5 * kgw.kgw_newton_schulz(dw, out_dtype=torch.bfloat16))
        self.router.sub_(lr * drouter)


def train(steps=10, tokens=1536, experts=8, hidden=512, inner=256, topk=2, lr=0.02, device="cuda", seed=0):
    """The losses of `steps` steps."""
    teacher = MoeLayer(experts, hidden, inner, topk, device, seed + 1)
    layer = MoeLayer(experts, hidden, inner, topk, device, seed + 2)
    layer.router.copy_(teacher.router)
    g = torch.Generator(device=device).manual_seed(seed)
    x = torch.randn((tokens, hidden), generator=g, device=device).bfloat16()
    target = teacher.forward(x)[0].float()
    losses = []
    for _ in range(steps):
        out, saved = layer.forward(x)
        diff = out.float() - target
        losses.append(float(diff.square().mean()))
        dout = (2.0 / diff.numel() * diff * 1024.0).bfloat16()      # 1024: keeps bf16 gradients away from zero
        dw1, dw2, drouter, _ = layer.backward(dout, saved)
        layer.update(dw1, dw2, drouter / 1024.0, lr)
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=10)
    for k, loss in enumerate(train(ap.parse_args().steps)):
        print(f"step {k:3d}  loss {loss:.5f}")
