"""kgw_newton_schulz on matrices whose short side is above 128: the kernels of tiled products.

fp32 and fp16 results are held against the iteration in 64 bits, with the tolerances of test_newton_gpu.py.  bf16
results keep two fp16 planes of the iterate and multiply the first one alone, which leaves about as much as the result's
own rounding; a bound counted from roundings is too wide to see an iterate that lost its second plane.
So their error is held against the error of that very scheme, its roundings repeated with sums in 64 bits.  The two are
not the same matrix: an fp32 sum that is off in its last bit turns some element's rounding to fp16, and after two or
three steps all roundings are others.  But both are sums of as many independent roundings, of which the norm
is near its mean (by 1 / sqrt(r) for r directions, 8% at most here), while operands of eight bits are 2.6 times as far
off or more, and an iterate without its second plane 1.6 times where singular values fall off along a power law
(normal matrices have few small ones and do not show it): a quarter more than the scheme's error is allowed.
"""
import pytest
import torch

import grouped_gemm_expert_offsets_amd as kgw

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs an MI355X")]

DEV = "cuda"
CO = kgw.NEWTON_SCHULZ_COEFFICIENTS
EPS = 1e-7
# 64-edged tiles, alone and sharing K, as they are and turned; 128-edged ones; 256-edged ones with strips
SHAPES = [(2, 150, 290), (2, 290, 150), (1, 200, 4100), (8, 500, 700), (24, 1021, 1019)]


def triples(co, steps):
    return [tuple(co)] * steps if not hasattr(co[0], "__len__") else [tuple(t) for t in co]


def iterate(G, co, step):
    X = G.double() / (torch.linalg.vector_norm(G.double(), dim=(1, 2), keepdim=True) + EPS)
    tall = X.shape[1] > X.shape[2]
    X = X.transpose(1, 2).contiguous() if tall else X
    for a, b, c in torch.tensor(co, dtype=torch.float32).double().tolist():
        X = step(X, a, b, c)
    return X.transpose(1, 2).contiguous() if tall else X


def exact_step(X, a, b, c):
    A = X @ X.transpose(1, 2).contiguous()
    return a * X + (b * A + c * (A @ A)) @ X


def reference(G, co):
    return iterate(G, co, exact_step)


def scheme(G, co, low=True, operand=torch.float16):
    """The two-plane iteration with its roundings, before the last one to bf16.  low, operand: as kernels would be that
    lost the second plane, or multiplied another type."""
    def plane(x, power, dtype=torch.float16):
        return (x * 2.0 ** power).to(dtype).double() * 2.0 ** -power

    def step(X, a, b, c):
        hi = plane(X, 13)
        X = hi + plane(X - hi, 13) if low else hi
        hi = plane(hi, 13, operand)
        A = plane(hi @ hi.transpose(1, 2).contiguous(), 10, operand)
        return a * X + plane(b * A + c * (A @ A), 7, operand) @ hi
    return iterate(G, co, step)


def distance(a, b):
    return float((a.double() - b).norm() / b.norm())


def check(got, G, co):
    want = reference(G, co)
    grown = 1.0
    for a, _, _ in co:
        grown *= abs(a)
    size = max(G.shape[1:])
    if got.dtype == torch.bfloat16:
        for g, near, w in zip(got, scheme(G, co).bfloat16(), want):
            tol = 1.25 * distance(near, w)
            assert distance(g, w) <= tol, (distance(g, w), tol)
        return
    for g, w in zip(got, want):
        total = torch.finfo(got.dtype).eps / 2 + 4 * len(co) * 2.0 ** -22 + 1.5 * grown * 2.0 ** -22 / float(w.norm())
        tol = total / 3 ** 0.5 + 3 * len(co) * size ** 0.5 * 2.0 ** -24
        assert distance(g, w) <= tol, (distance(g, w), tol)


def gradients(batch, m, n, dtype, seed, normal=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    if normal:
        return torch.randn((batch, m, n), generator=g, device=DEV).to(dtype)
    r = min(m, n)
    strength = 0.02 * torch.arange(1, r + 1, device=DEV, dtype=torch.float32) ** -0.75
    return torch.stack([(torch.randn((m, r), generator=g, device=DEV) * strength)
                        @ torch.randn((r, n), generator=g, device=DEV) for _ in range(batch)]).to(dtype)


@pytest.mark.parametrize("wrong", [dict(low=False), dict(operand=torch.bfloat16)])
@pytest.mark.parametrize("batch,m,n", SHAPES)
def test_the_oracle_sees_lost_planes_and_other_operands(batch, m, n, wrong):
    """What check() allows is less than what either mistake makes."""
    G = gradients(batch, m, n, torch.float32, 1)
    co = triples(CO, 5)
    with pytest.raises(AssertionError):
        check(scheme(G, co, **wrong).bfloat16(), G, co)
    check(scheme(G, co).bfloat16(), G, co)


@pytest.mark.parametrize("normal", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("batch,m,n", SHAPES + [(4, 256, 512), (3, 1777, 1000), (1, 1536, 2900), (8, 4219, 381), (5, 1149, 3451)])
def test_bf16_results(batch, m, n, dtype, normal):
    G = gradients(batch, m, n, dtype, m + n, normal)
    check(kgw.kgw_newton_schulz(G, out_dtype=torch.bfloat16), G, triples(CO, 5))


PER_STEP = [(4.0848, -6.8946, 2.9270), (3.9505, -6.3029, 2.6377), (3.7418, -5.5913, 2.3037)]


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("co,steps", [(CO, 1), (CO, 2), (CO, 3), (CO, 6), (PER_STEP, 3), ((1.5, -0.5, 0.0), 4)])
@pytest.mark.parametrize("batch,m,n", SHAPES)
def test_steps_and_coefficients(batch, m, n, co, steps, out):
    G = gradients(batch, m, n, torch.float32, 4)
    check(kgw.kgw_newton_schulz(G, steps=steps, coefficients=co, out_dtype=out), G, triples(co, steps))


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("batch,m,n", SHAPES)
def test_strides(batch, m, n, dtype, out):
    wide = gradients(batch, m + 7, n + 21, dtype, 6)
    view = wide[:, 3:3 + m, 5:5 + n]                                   # rows start at odd elements, matrices too
    whole = view.contiguous()
    got = kgw.kgw_newton_schulz(view, out_dtype=out)
    check(got, whole, triples(CO, 5))
    assert torch.equal(got, kgw.kgw_newton_schulz(whole, out_dtype=out))
    out_of = torch.full((got.numel() + 1,), float("nan"), dtype=out, device=DEV)[1:].view(got.shape)
    assert torch.equal(kgw.kgw_newton_schulz(view, out=out_of), got)   # a result that starts at an odd element
    same = wide[:1, 3:3 + m, 5:5 + n].expand(batch, -1, -1)            # batch stride 0
    assert torch.equal(kgw.kgw_newton_schulz(same, out_dtype=out)[batch - 1], got[0])
    assert torch.equal(kgw.kgw_newton_schulz(view[0], out_dtype=out), kgw.kgw_newton_schulz(whole[:1], out_dtype=out)[0])


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n", [(150, 290), (290, 150), (1021, 1019)])
def test_zero_and_special_matrices_stay_apart(m, n, out):
    batch = 24 if m > 1000 else 5
    G = gradients(batch, m, n, torch.float32, 7)
    G[1] = 0
    G[2, 3, 4] = float("nan")
    G[3, m - 1, n - 1] = float("inf")
    got = kgw.kgw_newton_schulz(G, out_dtype=out)
    assert not got[1].any()
    assert got[2].isnan().all() and got[3].isnan().all()
    keep = [k for k in range(batch) if k not in (1, 2, 3)]
    check(got[keep], G[keep], triples(CO, 5))


@pytest.mark.parametrize("batch,m,n", SHAPES + [(2, 100, 300)])
def test_precise_bf16_results_are_the_fp32_ones_rounded(batch, m, n):
    G = gradients(batch, m, n, torch.bfloat16, 8)
    want = kgw.kgw_newton_schulz(G, out_dtype=torch.float32)
    assert torch.equal(kgw.kgw_newton_schulz(G, precise=True), want.bfloat16())
    assert torch.equal(kgw.kgw_newton_schulz(G, precise=True, out_dtype=torch.float32), want)
