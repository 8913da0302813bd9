"""kgw_newton_schulz over the sizes of gradients, eps and coefficients, with errors relative to the result.

A matrix whose norm is far below eps has a small X_0 = G / (|G| + eps) that grows by |a| at every step; coefficients
may make an iterate, B = b A + c A A or the result as small or large as they like (a learning rate folded into the
last three, say).  Tolerances count, per matrix as |got - want|_F / |want|_F with a rounding to type t at most
h_t = finfo(t).eps / 2 of the value and h_t / sqrt(3) in the mean square:
  * the result's own rounding h_t;
  * four roundings of the products' operands a step, u = 2^-11 (fp16) for a bf16 result of short sides above 128,
    2^-22 (a half and its remainder) otherwise;
  * the kept iterate's 2^-22 of |X_0|, which later steps multiply by their |a| at most where singular values are
    small: 1.5 |a_1 .. a_n| 2^-22 |X_0| against |want|;
  * fp32 sums over at most c terms, 3 products a step: 3 steps sqrt(c) 2^-24.
"""
import math

import pytest
import torch

import grouped_gemm_expert_offsets_amd as kgw

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs an MI355X")]

DEV = "cuda"
CO = kgw.NEWTON_SCHULZ_COEFFICIENTS
# one workgroup a matrix, a launch a step, wide with 64-edged tiles as they are and turned, 128- and 256-edged ones
SHAPES = [(50, 80), (128, 100), (50, 900), (150, 290), (290, 150), (600, 1000)]


def triples(co, steps):
    return [co] * steps if not hasattr(co[0], "__len__") else list(co)


def reference(G, co, eps):
    """(batch, m, n) in 64 bits; coefficients as the library gets them, in fp32."""
    X = G.double()
    X = X / (torch.linalg.vector_norm(X, dim=(1, 2), keepdim=True) + eps)
    tall = X.shape[1] > X.shape[2]
    X = X.transpose(1, 2).contiguous() if tall else X
    for a, b, c in torch.tensor(co, dtype=torch.float32).double().tolist():
        A = X @ X.transpose(1, 2).contiguous()
        X = a * X + (b * A + c * (A @ A)) @ X
    return X.transpose(1, 2) if tall else X


def gradients(batch, m, n, seed):
    """Matrices of norm 1 in 64 bits, singular values along a power law."""
    g = torch.Generator().manual_seed(seed)
    r = min(m, n)
    strength = torch.arange(1, r + 1, dtype=torch.float64) ** -0.75
    G = torch.stack([(torch.randn((m, r), generator=g, dtype=torch.float64) * strength)
                     @ torch.randn((r, n), generator=g, dtype=torch.float64) for _ in range(batch)])
    return (G / torch.linalg.vector_norm(G, dim=(1, 2), keepdim=True)).to(DEV)


def check(G, co=CO, steps=5, eps=1e-7, out=torch.float32):
    co = triples(co, steps)
    eps = float(torch.tensor(eps, dtype=torch.float32))
    want = reference(G, co, eps)
    got = kgw.kgw_newton_schulz(G, steps=len(co), coefficients=co, eps=eps, out_dtype=out)
    grown = abs(math.prod(a for a, _, _ in co))
    for k, (g, w) in enumerate(zip(got.double(), want)):
        norm, first = float(w.norm()), float(G[k].double().norm())
        first = first / (first + eps)
        u = 2.0 ** -11 if out == torch.bfloat16 and min(w.shape) > 128 else 2.0 ** -22
        total = torch.finfo(out).eps / 2 + 4 * len(co) * u + 1.5 * grown * 2.0 ** -22 * first / norm
        tol = total / 3 ** 0.5 + 3 * len(co) * max(w.shape) ** 0.5 * 2.0 ** -24
        err = float((g - w).norm()) / norm
        assert err <= tol, (k, norm, err, tol)


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,n", SHAPES)
def test_norms_far_below_eps_each_in_one_batch(m, n, out):
    G = gradients(8, m, n, m + n)
    sizes = torch.tensor([1.0, 1e-6, 1e-8, 1e-10, 1e-13, 1e-16, 1e-24, 1e-33], device=DEV, dtype=torch.float64)
    check((G * sizes[:, None, None]).float(), out=out)


@pytest.mark.parametrize("eps", [1e-30, 1.0, 1e4])
def test_eps_of_any_size(eps):
    for m, n in ((50, 900), (150, 290)):
        G = gradients(3, m, n, 2)
        check((G * torch.tensor([1.0, 1e-4, 1e4], device=DEV, dtype=torch.float64)[:, None, None]).float(), eps=eps)


@pytest.mark.parametrize("size", [1e-37, 1e33, 3e38])
def test_norms_at_the_ends_of_fp32(size):
    for m, n in ((50, 80), (150, 290), (900, 1100)):
        G = gradients(2, m, n, 3)
        G = (G / G.abs().amax() * size).float()          # up to 1e41: the norm leaves fp32, no element does
        check(G, eps=0.0)


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("factor", [1e-20, 1e-8, 1e-4, 0.02, 1e3, 1e10])
@pytest.mark.parametrize("m,n", SHAPES)
def test_a_factor_folded_into_the_last_step(m, n, factor, out):
    check(gradients(2, m, n, 4).float(), co=[CO] * 4 + [tuple(factor * v for v in CO)], out=out)


@pytest.mark.parametrize("factor", [1e-8, 0.02])
@pytest.mark.parametrize("m,n", SHAPES)
def test_a_factor_folded_into_an_earlier_step(m, n, factor):
    check(gradients(2, m, n, 5).float(), co=[CO] * 2 + [tuple(factor * v for v in CO)] + [CO] * 2)


# steps that start steeply, cubic ones, linear ones, and one whose square term alone is large
OTHERS = [[(8.2872, -23.5959, 17.3004), (4.1071, -2.9478, 0.5448), (3.9487, -2.9089, 0.5518)], (1.5, -0.5, 0.0),
          (2.0, 0.0, 0.0), (0.5, 0.0, 2.0), (3.0, -30.0, 90.0)]


@pytest.mark.parametrize("co", OTHERS)
@pytest.mark.parametrize("m,n", SHAPES)
def test_other_coefficients(m, n, co):
    G = gradients(2, m, n, 6)
    check((G * torch.tensor([1.0, 1e-9], device=DEV, dtype=torch.float64)[:, None, None]).float(), co=co, steps=3)


@pytest.mark.parametrize("co,power", [((0.0, 1.0, 0.0), 3), ((0.0, 0.0, 1.0), 5)])
@pytest.mark.parametrize("m,n", SHAPES)
def test_powers_alone(m, n, co, power):
    """Singular values to the third or fifth power, far below what the norm says.  A relative error grows by the power
    at every step: power^2 times the roundings of one step, four of 2^-22 and three sums, in two."""
    G = gradients(2, m, n, 9).float()
    want = reference(G, [co] * 2, 0.0)
    got = kgw.kgw_newton_schulz(G, steps=2, coefficients=co, eps=0.0)
    tol = 2.0 ** -24 + power ** 2 * (4 * 2.0 ** -22 + 3 * max(m, n) ** 0.5 * 2.0 ** -24)
    for g, w in zip(got.double(), want):
        assert float((g - w).norm() / w.norm()) <= tol


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,n", [(50, 80), (50, 900), (150, 290)])
def test_zeros_stay_zeros_beside_others(m, n, out):
    G = gradients(3, m, n, 7).float()
    G[1] = 0
    G[2] *= 1e-12
    for eps in (1e-7, 1e-38):
        got = kgw.kgw_newton_schulz(G, eps=eps, out_dtype=out)
        assert not got[1].any() and not got.isnan().any()


def test_results_keep_a_matrix_and_its_batch_apart():
    """A matrix far below eps has the same result alone as beside one that is not."""
    for m, n in ((50, 80), (50, 900), (150, 290)):
        G = gradients(2, m, n, 8).float()
        G[1] *= 1e-12
        both = kgw.kgw_newton_schulz(G)
        assert torch.equal(both[0], kgw.kgw_newton_schulz(G[0])) and torch.equal(both[1], kgw.kgw_newton_schulz(G[1]))
