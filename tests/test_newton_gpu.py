"""kgw_newton_schulz against the iteration in 64 bits.

Errors are judged per matrix as |got - want|_F / |want|_F.  A rounding to type t is off by at most
half a step, h_t = finfo(t).eps / 2 of the value, and by h_t / sqrt(3) in the mean square.
  * the result's own rounding: h_t;
  * operands: each step rounds X, A (twice used) and B, 4 roundings of u, u = 2^-11 (fp16) for a
    bf16 result and 2^-22 (a half and its remainder) otherwise;
  * the kept iterate, 2^-22, whose error the linear term multiplies by |a| at every step where
    singular values are small: in all 1.5 |a|^steps 2^-22 of |X_0| = 1, against |want|_F;
  * fp32 sums over at most c terms, 3 products a step: 3 steps sqrt(c) 2^-24.
"""
import numpy as np
import pytest
import torch

import grouped_gemm_expert_offsets_amd as kgw

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs an MI355X")]

DEV = "cuda"
CO = kgw.NEWTON_SCHULZ_COEFFICIENTS


def reference(G, steps=5, co=CO, eps=1e-7):
    """(batch, m, n) in 64 bits."""
    per_step = [co] * steps if not hasattr(co[0], "__len__") else co
    X = G.detach().double()
    X = X / (torch.linalg.vector_norm(X, dim=(1, 2), keepdim=True) + eps)
    tall = X.shape[1] > X.shape[2]
    X = X.transpose(1, 2).contiguous() if tall else X
    for a, b, c in per_step:
        A = X @ X.transpose(1, 2).contiguous()
        X = a * X + (b * A + c * (A @ A)) @ X
    return X.transpose(1, 2) if tall else X


def tolerance(want, dtype, steps, a=CO[0]):
    norm = float(want.norm())
    u = 2.0 ** -11 if dtype == torch.bfloat16 else 2.0 ** -22
    c = max(want.shape)
    total = torch.finfo(dtype).eps / 2 + 4 * steps * u + 1.5 * abs(a) ** steps * 2.0 ** -22 / norm
    return total / 3 ** 0.5 + 3 * steps * c ** 0.5 * 2.0 ** -24


def check(got, want, steps=5, a=CO[0]):
    assert got.shape == want.shape
    for g, w in zip(got, want):
        if not w.any():
            assert not g.any()
            continue
        err = float((g.double() - w).norm() / w.norm())
        tol = tolerance(w, got.dtype, steps, a)
        assert err <= tol, (err, tol)


def gradients(batch, m, n, dtype, seed, scale=0.02):
    g = torch.Generator().manual_seed(seed)
    r = min(m, n)
    strength = scale * torch.arange(1, r + 1, dtype=torch.float32) ** -0.75
    G = torch.stack([(torch.randn((m, r), generator=g) * strength) @ torch.randn((r, n), generator=g)
                     for _ in range(batch)])
    return G.to(dtype).to(DEV)


SIZES = [(1, 1, 1), (1, 1, 300), (1, 129, 1), (2, 7, 5), (3, 64, 64), (2, 65, 63), (4, 128, 128), (4, 256, 512), (2, 200, 1100),
         (5, 1000, 333), (1, 513, 514), (3, 31, 4099)]
TYPES = [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.bfloat16), (torch.float16, torch.bfloat16),
         (torch.bfloat16, torch.float32), (torch.float32, torch.float32), (torch.float32, torch.float16)]


@pytest.mark.parametrize("batch,m,n", SIZES)
@pytest.mark.parametrize("dtype,out", TYPES)
def test_against_the_iteration(batch, m, n, dtype, out):
    G = gradients(batch, m, n, dtype, m + n)
    got = kgw.kgw_newton_schulz(G, out_dtype=out)
    assert got.dtype == out
    check(got, reference(G))


# One batch for every way a size is taken: 64-edged tiles alone and several workgroups a tile, 128-edged ones
# likewise, 256-edged ones with the last round whole or in quarters and with strips on one side, the other, both
# or none; short sides with one workgroup a matrix, a launch a step, and several chunks a workgroup.
WAYS = [(4, 256, 512), (1, 200, 7000), (1, 4096, 512), (64, 300, 500), (3, 1777, 1000), (1, 1536, 2900), (10, 381, 3323),
        (8, 4219, 381), (10, 3451, 509), (10, 509, 2555), (5, 1149, 3451), (24, 1021, 1019), (24, 1147, 1149), (12, 1531, 1405),
        (3, 20, 30), (70, 400, 60), (130, 40, 300), (40, 60, 2100), (20, 3500, 120), (4, 128, 128), (1, 1700, 1690),
        (1, 1690, 1700)]


@pytest.mark.parametrize("batch,m,n", WAYS)
@pytest.mark.parametrize("dtype,out", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32)])
def test_every_way_a_size_is_taken(batch, m, n, dtype, out):
    G = gradients(batch, m, n, dtype, m + n)
    check(kgw.kgw_newton_schulz(G, out_dtype=out), reference(G))


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_singular_values_come_out_near_one(out):
    G = gradients(1, 96, 160, torch.float32, 3)
    s = torch.linalg.svdvals(kgw.kgw_newton_schulz(G, out_dtype=out)[0].double())
    assert float(s.max()) < 1.25 and float(s[:48].min()) > 0.65


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_steps_and_coefficients(out):
    G = gradients(2, 90, 130, torch.float32, 4)
    check(kgw.kgw_newton_schulz(G, steps=1, out_dtype=out), reference(G, 1), 1)
    check(kgw.kgw_newton_schulz(G, steps=8, out_dtype=out), reference(G, 8), 8)
    co = [(4.0848, -6.8946, 2.9270), (3.9505, -6.3029, 2.6377), (3.7418, -5.5913, 2.3037)]
    check(kgw.kgw_newton_schulz(G, steps=3, coefficients=co, out_dtype=out), reference(G, 3, co), 3, 4.1)
    cubic = (1.5, -0.5, 0.0)
    check(kgw.kgw_newton_schulz(G, steps=4, coefficients=cubic, out_dtype=out), reference(G, 4, cubic), 4, 1.5)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n", [(100, 260), (260, 100), (128, 128)])
def test_transposes_give_transposes(m, n, out):
    G = gradients(2, m, n, torch.float32, 5)
    if m == n:                      # a square matrix is not transposed inside: same value, other rounding
        check(kgw.kgw_newton_schulz(G.transpose(1, 2).contiguous(), out_dtype=out), reference(G).transpose(1, 2))
        return
    a = kgw.kgw_newton_schulz(G, out_dtype=out)
    b = kgw.kgw_newton_schulz(G.transpose(1, 2).contiguous(), out_dtype=out)
    assert torch.equal(a, b.transpose(1, 2))


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_strides(out):
    wide = gradients(3, 70, 200, torch.bfloat16, 6)
    view = wide[:, 3:66, 5:150]
    check(kgw.kgw_newton_schulz(view, out_dtype=out), reference(view))
    two = wide[1, :, :77]
    assert torch.equal(kgw.kgw_newton_schulz(two, out_dtype=out), kgw.kgw_newton_schulz(two[None].contiguous(),
                                                                                        out_dtype=out)[0])
    same = wide[:1].expand(4, -1, -1)                                  # batch stride 0
    assert torch.equal(kgw.kgw_newton_schulz(same, out_dtype=out)[3], kgw.kgw_newton_schulz(wide[0], out_dtype=out))


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_zero_and_special_matrices_stay_apart(out):
    G = gradients(5, 60, 100, torch.float32, 7)
    G[1] = 0
    G[2, 3, 4] = float("nan")
    G[3, 59, 99] = float("inf")
    got = kgw.kgw_newton_schulz(G, out_dtype=out)
    assert not got[1].any()
    assert got[2].isnan().all() and got[3].isnan().all()
    check(got[[0, 4]], reference(G[[0, 4]]))


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-12, 1e12, 1e30])
def test_scales_whose_squares_leave_fp32(scale):
    for m, n in ((50, 80), (50, 900), (150, 170)):
        G = gradients(2, m, n, torch.float32, 8, scale)
        check(kgw.kgw_newton_schulz(G, eps=0.0), reference(G, eps=0.0))
    if scale == 1e-30:              # eps takes over: X stays small, the steps multiply it by a^5
        check(kgw.kgw_newton_schulz(G * 1e20), reference(G * 1e20))


def test_repeats_are_equal_and_workspace_is_reused():
    lib = kgw.load_library()
    G = gradients(3, 150, 290, torch.float32, 9)
    ws = torch.full((lib.kgw_newton_schulz_workspace_bytes(3, 150, 290, kgw.KGW_OUT_FP32),), 0xFF, dtype=torch.uint8,
                    device=DEV)     # NaN patterns everywhere
    first = kgw.kgw_newton_schulz(G, workspace=ws)
    out = torch.full_like(G, float("nan"))
    assert kgw.kgw_newton_schulz(G, workspace=ws, out=out) is out
    assert torch.equal(first, out)
    assert torch.equal(first, kgw.kgw_newton_schulz(G))
    with pytest.raises(ValueError):
        kgw.kgw_newton_schulz(G, workspace=ws[:-256])


@pytest.mark.parametrize("shape,out", [((2, 100, 300), torch.bfloat16), ((4, 256, 512), torch.float32),
                                       ((64, 300, 500), torch.bfloat16)])
def test_on_another_stream_and_in_a_graph(shape, out):
    G = gradients(*shape, torch.float32, 10)
    want = kgw.kgw_newton_schulz(G, out_dtype=out)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = kgw.kgw_newton_schulz(G, out_dtype=out)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = kgw.kgw_newton_schulz(G, out_dtype=out)
    for r in range(4):
        held.fill_(float("nan"))
        G.mul_(0.7).add_(1e-3)
        want = kgw.kgw_newton_schulz(G, out_dtype=out)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, want), r


def test_empty_sizes():
    for shape in [(0, 4, 4), (2, 0, 5), (2, 5, 0)]:
        assert kgw.kgw_newton_schulz(torch.empty(shape, device=DEV)).shape == shape


def test_a_wgrad_result_goes_in_as_it_is():
    import workloads
    wl = workloads.make_workload("tiny", seed=1, device=DEV)
    dw = kgw.kgw_wgrad_bf16(wl.A, wl.B, wl.offsets, out_dtype=torch.float32)
    got = kgw.kgw_newton_schulz(dw)
    assert not got[1].any()                                            # the expert without tokens
    check(got, reference(dw))


def test_refusals():
    G = torch.zeros((2, 8, 16), device=DEV)
    bad = [dict(G=G.double()), dict(G=G[0, 0]), dict(G=G.transpose(1, 2)), dict(G=G.cpu()), dict(G=G, steps=0),
           dict(G=G, steps=65), dict(G=G, coefficients=(1.0, 2.0)), dict(G=G, steps=2, coefficients=[(1, 2, 3)]),
           dict(G=G, eps=-1.0), dict(G=G, eps=float("nan")), dict(G=G, out_dtype=torch.float64),
           dict(G=G, out=torch.zeros((2, 16, 8), device=DEV)), dict(G=G, out=G.cpu()),
           dict(G=G, workspace=torch.zeros(16, dtype=torch.uint8, device=DEV)),
           dict(G=G, workspace=torch.zeros(1 << 20, device=DEV))]
    for k, kw in enumerate(bad):
        with pytest.raises(ValueError):
            kgw.kgw_newton_schulz(**kw)
            pytest.fail(f"call {k} was accepted")
