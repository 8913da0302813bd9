"""Weight gradients whose offsets end before tokens_sum, as the token sort makes them in a buffer of fixed size: the rows
behind the last offset belong to no expert.  They hold NaN here, and the results are bit for bit those of the same
tokens with one more expert, which owns the rows behind (one pass: every output element is summed by itself).

With the sort's offsets as they are, a whole layer step is queued without a look at them on the host, so it
can be captured in a graph.
"""
import pytest
import torch

import grouped_gemm_expert_offsets_amd as kgw
import workloads

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs an MI355X")]

DEV = "cuda"
CASES = [([256, 0, 512, 768], 264, 400), ([2048] * 3 + [1024], 320, 384), ([0, 0, 256], 256, 256), ([1024] * 40 + [4096], 256, 512)]


def same(got, want):
    assert torch.equal(got, want) and not got.isnan().any()


def tails(t, axis, tokens, per=1):
    """A copy whose entries of the tokens from `tokens` on are NaN (e4m3: 0x7F, scales: 0xFF)."""
    t = t.clone()
    part = t.narrow(axis, tokens // per, t.shape[axis] - tokens // per)
    part.fill_(float("nan") if t.is_floating_point() else 0x7F if per == 1 else 0xFF)
    return t


@pytest.mark.parametrize("counts,hidden,n", CASES)
def test_bf16(counts, hidden, n):
    wl = workloads.make_operands(counts, hidden, n, "bf16", torch.float32, False, seed=1, device=DEV)
    used = sum(counts[:-1])
    short = wl.offsets[:-1].contiguous()
    want = kgw.kgw_wgrad_bf16(wl.A, wl.B, wl.offsets, split_k=False)[:-1]
    A, B = tails(wl.A, 1, used), tails(wl.B, 0, used)
    same(kgw.kgw_wgrad_bf16(A, B, short, split_k=False), want)
    split = kgw.kgw_wgrad_bf16(A, B, short)
    assert float((split - want).norm()) <= 1e-5 * float(want.norm())
    for a, b in (("m", "n"), ("k", "k"), ("m", "k")):
        got = kgw.kgw_wgrad_bf16_ex(A.t().contiguous() if a == "m" else A, B.t().contiguous() if b == "k" else B, short,
                                    a_major=a, b_major=b, split_k=False)
        full = kgw.kgw_wgrad_bf16_ex(wl.A.t().contiguous() if a == "m" else wl.A, wl.B.t().contiguous() if b == "k" else wl.B,
                                     wl.offsets, a_major=a, b_major=b, split_k=False)
        same(got, full[:-1])
    blocks = lambda t, axis: torch.cat([p.reshape(-1) for p in t.split(counts, axis)])  # noqa: E731
    ra, rb = blocks(wl.A, 1), blocks(wl.B.t().contiguous(), 1)
    full = kgw.kgw_wgrad_bf16_ex(ra, rb, wl.offsets, b_major="k", ragged=True, hidden=hidden, n=n, split_k=False)
    ra[used * hidden:] = float("nan")
    rb[used * n:] = float("nan")
    same(kgw.kgw_wgrad_bf16_ex(ra, rb, short, b_major="k", ragged=True, hidden=hidden, n=n, split_k=False), full[:-1])
    start = torch.randn_like(want)
    out = start.clone()
    kgw.kgw_wgrad_bf16(A, B, short, out, accumulate=True, split_k=False)
    assert not out.isnan().any()
    empty = [e for e, c in enumerate(counts[:-1]) if c == 0]
    assert torch.equal(out[empty], start[empty])


@pytest.mark.parametrize("counts,hidden,n", CASES)
def test_fp8(counts, hidden, n):
    wl = workloads.make_operands(counts, hidden, n, "fp8", torch.float32, False, seed=2, device=DEV)
    used = sum(counts[:-1])
    short = wl.offsets[:-1].contiguous()
    A, B = tails(wl.A.view(torch.uint8), 1, used), tails(wl.B.view(torch.uint8), 0, used)
    sfa, sfb = tails(wl.sfa, 0, used, 128), tails(wl.sfb, 0, used, 128)
    for call in (kgw.kgw_wgrad_fp8, kgw.kgw_wgrad_fp8_native):
        want = call(wl.A, wl.sfa, wl.B, wl.sfb, wl.offsets, out_dtype=torch.float32, split_k=False)[:-1]
        same(call(A, sfa, B, sfb, short, out_dtype=torch.float32, split_k=False), want)
    if hidden % 16 == 0:
        for a, b in (("m", "n"), ("k", "k"), ("m", "k")):
            turned = lambda x, y: (x.t().contiguous() if a == "m" else x, y.t().contiguous() if b == "k" else y)  # noqa: E731
            (fa, fb), (ta, tb) = turned(wl.A, wl.B), turned(A, B)
            kw = dict(a_major=a, b_major=b, out_dtype=torch.float32, split_k=False)
            same(kgw.kgw_wgrad_fp8_ex(ta, sfa, tb, sfb, short, **kw), kgw.kgw_wgrad_fp8_ex(fa, wl.sfa, fb, wl.sfb, wl.offsets, **kw)[:-1])


@pytest.mark.parametrize("counts,hidden,n", CASES)
def test_fp4(counts, hidden, n):
    wl = workloads.make_fp4_operands(counts, hidden, n, seed=3)
    A, B, offsets = (wl[k].to(DEV) for k in ("A", "B", "offsets"))
    sfa, sfb = (workloads.pack_scale_words(wl[k]).to(DEV) for k in ("sfa", "sfb"))
    used = sum(counts[:-1])
    short = offsets[:-1].contiguous()
    want = kgw.kgw_wgrad_fp4(A, sfa, B, sfb, offsets, out_dtype=torch.float32, split_k=False)[:-1]
    sfa, sfb = sfa.clone(), sfb.clone()
    sfa[used // 128:] = -1                                             # scale bytes of NaN
    sfb[used // 128:] = -1
    same(kgw.kgw_wgrad_fp4(A, sfa, B, sfb, short, out_dtype=torch.float32, split_k=False), want)


def test_a_layer_step_in_a_graph():
    tokens, k, E, hidden, inner = 700, 2, 6, 256, 128
    g = torch.Generator().manual_seed(5)
    new = lambda *shape: torch.randn(shape, generator=g).bfloat16().to(DEV)  # noqa: E731
    x, dout, w1, w2 = new(tokens, hidden), new(tokens, hidden), new(E, hidden, inner), new(E, inner, hidden)
    p = torch.softmax(torch.randn((tokens, k), generator=g), 1).to(DEV)
    choose = lambda: torch.rand((tokens, E), generator=g).topk(k, dim=1).indices.to(DEV)  # noqa: E731
    ids = choose()

    def step():
        _, offsets, row_of, src_of = kgw.kgw_moe_sort(ids, E, alignment=256)
        rows = kgw.kgw_moe_permute(x, row_of, src_of)
        h = torch.full((rows.shape[0], inner), float("nan"), dtype=rows.dtype, device=DEV)    # rows of no expert stay so
        kgw.kgw_mgrouped_bf16(rows, w1, offsets=offsets, layout="nn", out=h)
        y = torch.full_like(rows, float("nan"))
        kgw.kgw_mgrouped_bf16(h, w2, offsets=offsets, layout="nn", out=y)
        out = kgw.kgw_moe_unpermute(y, row_of, p)
        dy, dp = kgw.kgw_moe_unpermute_grad(dout, y, row_of, src_of, p)
        dh = torch.full_like(h, float("nan"))
        kgw.kgw_mgrouped_bf16(dy, w2, offsets=offsets, layout="nt", out=dh)
        dw2 = kgw.kgw_wgrad_bf16_ex(h, dy, offsets, a_major="m")
        dw1 = kgw.kgw_wgrad_bf16_ex(rows, dh, offsets, a_major="m")
        drows = torch.full_like(rows, float("nan"))
        kgw.kgw_mgrouped_bf16(dh, w1, offsets=offsets, layout="nt", out=drows)
        dx = kgw.kgw_moe_unpermute(drows, row_of)
        return out, dp, dw1, dw2, dx, kgw.kgw_newton_schulz(dw1)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for r in range(4):
        for t in held:
            t.fill_(float("nan"))
        ids.copy_(choose())
        x.mul_(0.9)
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, want):
            same(a, b)
