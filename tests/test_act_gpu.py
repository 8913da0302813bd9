"""The activation with its 8-bit checkpoint against plain 64-bit forms.

u = 2^-24.  The kept values are rounded from the exact inputs, so codes and scales are compared bit for bit with the
definition.  A sigmoid s of g is off by r = ((1 - s)(2 |g| + 3) + 5) u of itself (the argument's two roundings pass
through s's derivative; the exponential, the sum and the reciprocal are within 5 u).  So, before the rounding to the
result's type (half a step of the value, or of the type's smallest step):
    swiglu  y = g s u:                     (r + 3 u) |y|
            du = dy g s:                   (r + 3 u) |du|
            dg = dy u (s + g s (1 - s)):   |dy u| [(r + 6 u)(s + |g| s (1 - s)) + |g| s (2 r s + 2 u)]
    relu2   y, dh: 2 u of themselves
A sigmoid below 2^-126 (g below -87.3) is zero: the reciprocal has no subnormal results.  It is off by less than 2^-126 then,
which the factors of s above multiply: |g u|, |dy g| and |dy u| (1 + |g|) times 2^-126 are allowed on top.
8-bit results: the scale is that of a largest magnitude within those bounds, the values half a step of e4m3 (2^-4 of the
value, or 2^-10 of the scale).
"""
import pytest
import torch

import grouped_gemm_expert_offsets_amd as kgw

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs an MI355X")]

DEV = "cuda"
U = 2.0 ** -24
LEAST = 2.0 ** -126
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
HALVES = {"swiglu": 2, "relu2": 1}


def values(rows, cols, dtype, seed, pad=0, offset=0, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    wide = (spread * torch.randn(rows * (cols + pad) + offset + 1, generator=g)).to(dtype).to(DEV)
    return wide[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]


def quantise(x):
    """The definition, on the CPU: fp64 rows -> codes (rows, cols) and scale bytes (blocks, rows)."""
    rows, cols = x.shape
    codes, scales = torch.empty((rows, cols), dtype=torch.uint8), torch.empty((-(-cols // 128), rows), dtype=torch.uint8)
    for b in range(scales.shape[0]):
        part = x[:, 128 * b:128 * (b + 1)]
        top = part.abs().amax(1)
        bad = ~torch.isfinite(part).all(1)
        m, e = torch.frexp(torch.where(bad, 1.0, top))
        byte = torch.where(top == 0, 127, (e - 9 + (m > 0.875).int() + 127).clamp(1, 254))
        q = (part * torch.exp2(127.0 - byte.double())[:, None]).float().to(torch.float8_e4m3fn).view(torch.uint8)
        codes[:, 128 * b:128 * (b + 1)] = torch.where(bad[:, None], torch.tensor(0x7F, dtype=torch.uint8), q)
        scales[b] = torch.where(bad, 255, byte).to(torch.uint8)
    return codes, scales


def dequantise(codes, scales):
    v = codes.cpu().view(torch.float8_e4m3fn).double()
    s = torch.exp2(scales.cpu().double() - 127)
    s[scales.cpu() == 255] = float("nan")
    return v * s.t().repeat_interleave(128, 1)[:, :v.shape[1]]


def by_halves(f, x, act, *more):
    """f of each half of gated rows, put together again."""
    if act == "relu2":
        return f(x, *more)
    i = x.shape[1] // 2
    return tuple(torch.cat(p, d) for p, d in zip(zip(f(x[:, :i]), f(x[:, i:])), (1, 0)))


def kept_values(saved, scales, act):
    if act == "relu2":
        return dequantise(saved, scales)
    i, b = saved.shape[1] // 2, scales.shape[0] // 2
    return torch.cat((dequantise(saved[:, :i].contiguous(), scales[:b]), dequantise(saved[:, i:].contiguous(), scales[b:])), 1)


def forward(h, act):
    """y and the bound on the fp32 value's error."""
    if act == "relu2":
        y = h.clamp(min=0) ** 2
        return y, 2 * U * y
    i = h.shape[1] // 2
    g, u = h[:, :i], h[:, i:]
    s = torch.sigmoid(g)
    r = (torch.sigmoid(-g) * (2 * g.abs() + 3) + 5) * U
    y = g * s * u
    return y, (r + 3 * U) * y.abs() + LEAST * (g * u).abs()


def backward(h, dy, act):
    if act == "relu2":
        d = 2 * h.clamp(min=0) * dy
        return d, 2 * U * d.abs()
    i = h.shape[1] // 2
    g, u = h[:, :i], h[:, i:]
    s, c = torch.sigmoid(g), torch.sigmoid(-g)
    r = (c * (2 * g.abs() + 3) + 5) * U
    dg, du = dy * u * s * (1 + g * c), dy * g * s
    tol = (dy * u).abs() * ((r + 6 * U) * (s + g.abs() * s * c) + g.abs() * s * (2 * r * s + 2 * U) + LEAST * (1 + g.abs()))
    return torch.cat((dg, du), 1), torch.cat((tol, (r + 3 * U) * du.abs() + LEAST * (dy * g).abs()), 1)


def check_rows(got, want, tol, dtype):
    f = torch.finfo(dtype)
    rel, tiny = (0.0, 0.0) if dtype == torch.float32 else (f.eps / 2, f.tiny * f.eps / 2)
    got = got.cpu().double()
    over = want.abs() > f.max * (1 - f.eps)                 # past the type's range: infinity, or its largest value
    off = (got - want).abs()
    bad = (off > (1 + rel) * tol + rel * want.abs() + tiny + LEAST) & ~over
    assert not bool(bad.any()), f"{int(bad.sum())} values off, first {bad.nonzero()[0].tolist()}"


def check_8bit(codes, scales, want, tol):
    """One half: 8-bit rows against the values that they are rounded from."""
    got = dequantise(codes, scales)
    for b in range(scales.shape[0]):
        part = slice(128 * b, 128 * (b + 1))
        top, slack = want[:, part].abs().amax(1), tol[:, part].amax(1) + LEAST
        byte = scales[b].cpu().double()
        scale = torch.exp2(byte - 127)
        assert bool((top - slack <= 448 * scale).all())
        assert bool(((top + slack > 224 * scale) | (byte == 1) | ((top <= slack) & (byte == 127))).all())
        w = want[:, part]
        assert bool(((got[:, part] - w).abs() <= 2.0 ** -4 * w.abs() + 2.0 ** -10 * scale[:, None] + 1.1 * tol[:, part] + LEAST).all())


SHAPES = [(1, 8), (1, 128), (3, 64), (5, 136), (63, 128), (64, 512), (65, 520), (130, 1408), (257, 712), (7, 4096), (1029, 256)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ["swiglu", "relu2"])
@pytest.mark.parametrize("rows,inner", SHAPES)
def test_forward_and_backward(rows, inner, act, dtype):
    odd = rows % 2
    h = values(rows, HALVES[act] * inner, dtype, rows + inner, 3 * odd, odd)
    dy = values(rows, inner, dtype, rows, 5 * odd, odd)
    out = torch.full((rows, inner), float("nan"), dtype=dtype, device=DEV)
    y, none, saved, scales = kgw.kgw_moe_act_fp8(h, act=act, out=out)
    assert y is out and none is None
    want_codes, want_scales = by_halves(quantise, h.double().cpu(), act)
    assert torch.equal(saved.cpu(), want_codes) and torch.equal(scales.cpu(), want_scales)
    check_rows(y, *forward(h.double().cpu(), act), dtype)
    kept = kept_values(saved, scales, act)
    dh, none, y2, none2 = kgw.kgw_moe_act_fp8_grad(dy, saved, scales, act=act, again=True)
    assert none is None and none2 is None
    check_rows(dh, *backward(kept, dy.double().cpu(), act), dtype)
    check_rows(y2, *forward(kept, act), dtype)
    # without a checkpoint, and without y again
    assert torch.equal(kgw.kgw_moe_act_fp8(h, act=act, save=False)[0], y)
    assert kgw.kgw_moe_act_fp8(h, act=act, save=False)[2:] == (None, None)
    alone = kgw.kgw_moe_act_fp8_grad(dy, saved, scales, act=act)
    assert torch.equal(alone[0], dh) and alone[1:] == (None, None, None)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ["swiglu", "relu2"])
@pytest.mark.parametrize("rows,inner", [(1, 8), (66, 136), (130, 512), (257, 712), (2049, 384)])
def test_eight_bit_results(rows, inner, act, dtype):
    halves = HALVES[act]
    h = values(rows, halves * inner, dtype, 3 * rows + inner, 1, 1)
    dy = values(rows, inner, dtype, rows + 1, 1, 1, spread=0.3)
    y, ys, saved, scales = kgw.kgw_moe_act_fp8(h, act=act, fp8=True)
    assert y.dtype == ys.dtype == torch.uint8 and ys.shape == (-(-inner // 128), rows)
    check_8bit(y, ys, *forward(h.double().cpu(), act))
    assert torch.equal(saved, kgw.kgw_moe_act_fp8(h, act=act)[2])
    kept = kept_values(saved, scales, act)
    dh, ds, y2, ys2 = kgw.kgw_moe_act_fp8_grad(dy, saved, scales, act=act, fp8=True, again=True)
    want, tol = backward(kept, dy.double().cpu(), act)
    b = ds.shape[0] // halves
    for k in range(halves):
        part = slice(k * inner, (k + 1) * inner)
        check_8bit(dh[:, part].contiguous(), ds[k * b:(k + 1) * b], want[:, part], tol[:, part])
    check_8bit(y2, ys2, *forward(kept, act))
    mixed = kgw.kgw_moe_act_fp8_grad(dy, saved, scales, act=act, fp8=False, again=True, again_fp8=True)
    assert mixed[0].dtype == dtype and torch.equal(mixed[2], y2) and torch.equal(mixed[3], ys2)


@pytest.mark.parametrize("rows,inner", [(65, 256), (128, 1408)])
def test_checkpoint_is_the_quantisers(rows, inner):
    h = values(rows, 2 * inner, torch.bfloat16, 9)
    q, s = kgw.kgw_quantize_fp8(h, 1)
    _, _, saved, scales = kgw.kgw_moe_act_fp8(h)
    assert torch.equal(saved, q) and torch.equal(scales, s)


def test_sizes_of_values():
    """Zeros, subnormals, values near the type's ends, large gates of both signs."""
    x = torch.tensor([0.0, -0.0, 1e-40, -1e-38, 1e-30, 3e38, -3e38, 1.0, -1.0, 88.0, -88.0, 104.0, -104.0, 1e4, -1e4, 448.0])
    h = torch.cat((x.repeat(8, 8), x.flip(0).roll(3).repeat(8, 8)), 1).to(DEV)
    h[1] *= 1e-3
    h[2] = 0
    h[3, :128] = 0
    dy = torch.full((8, 128), 0.5, device=DEV)
    y, _, saved, scales = kgw.kgw_moe_act_fp8(h)
    codes, want = by_halves(quantise, h.double().cpu(), "swiglu")
    assert torch.equal(saved.cpu(), codes) and torch.equal(scales.cpu(), want)
    hd = h.double().cpu()
    exact, tol = forward(hd, "swiglu")
    inside = exact.abs() < 3.4e38
    assert bool(((y.cpu().double() - exact).abs() <= tol + LEAST)[inside].all())
    dh = kgw.kgw_moe_act_fp8_grad(dy, saved, scales)[0].cpu().double()
    exact, tol = backward(kept_values(saved, scales, "swiglu"), dy.double().cpu(), "swiglu")
    inside = exact.abs() < 1e38
    assert bool(((dh - exact).abs() <= tol + LEAST)[inside].all()) and not dh.isnan().any()


def test_not_finite_stays_in_its_block():
    h = values(6, 512, torch.bfloat16, 2)
    clean = kgw.kgw_moe_act_fp8(h)
    h[1, 3], h[2, 130 + 256], h[4, 255] = float("nan"), float("inf"), -float("inf")
    y, _, saved, scales = kgw.kgw_moe_act_fp8(h)
    codes, want = by_halves(quantise, h.double().cpu(), "swiglu")
    assert torch.equal(saved.cpu(), codes) and torch.equal(scales.cpu(), want) and int((scales == 255).sum()) == 3
    changed = (y != clean[0]) | y.isnan()
    assert changed.nonzero().tolist() == [[1, 3], [2, 130], [4, 255]] and y[1, 3].isnan()
    dy = values(6, 256, torch.bfloat16, 3)
    dh = kgw.kgw_moe_act_fp8_grad(dy, saved, scales)[0]
    bad = dh.isnan().view(6, 2, 2, 128)
    want_bad = torch.zeros_like(bad)
    for r, halves, b in ((1, [0, 1], 0), (2, [0], 1), (4, [0, 1], 1)):      # du = dy g s has no u in it
        want_bad[r, halves, b] = True
    assert torch.equal(bad, want_bad)


@pytest.mark.parametrize("act", ["swiglu", "relu2"])
@pytest.mark.parametrize("rows,last", [(200, 0), (200, 1), (200, 64), (200, 130), (200, 200), (200, 500), (200, -3), (5000, 3333)])
def test_rows_past_the_last_offset_are_left_alone(rows, last, act):
    inner, halves = 136, HALVES[act]
    n = min(max(last, 0), rows)
    h = values(rows, halves * inner, torch.bfloat16, 1)
    dy = values(rows, inner, torch.bfloat16, 2)
    want = kgw.kgw_moe_act_fp8(h, act=act)
    want_grad = kgw.kgw_moe_act_fp8_grad(dy, want[2], want[3], act=act, again=True)
    h[n:], dy[n:] = float("nan"), float("nan")
    offsets = torch.tensor([0, min(n, 64), last], dtype=torch.int32, device=DEV)
    lib, code = kgw.load_library(), kgw.KGW_OUT_BF16
    fill = lambda *shape, t=torch.uint8: torch.full(shape, 77, dtype=t, device=DEV)  # noqa: E731
    blocks = -(-inner // 128)
    for fp8 in (False, True):
        y = fill(rows, inner) if fp8 else fill(rows, inner, t=torch.bfloat16)
        ys, saved, ss = fill(blocks, rows), fill(rows, halves * inner), fill(halves * blocks, rows)
        stream = torch.cuda.current_stream().cuda_stream
        p = lambda t: t.data_ptr()  # noqa: E731
        assert lib.kgw_moe_act_fp8(p(h), h.stride(0), code, kgw._ACTS[act], p(offsets), 3, rows, inner, p(y), p(ys) if fp8 else None,
                                   p(saved), p(ss), stream) == 0
        assert (y[n:] == 77).all() and (saved[n:] == 77).all() and (ss[:, n:] == 77).all() and (ys[:, n if fp8 else 0:] == 77).all()
        assert torch.equal(saved[:n], want[2][:n]) and torch.equal(ss[:, :n], want[3][:, :n])
        if not fp8:
            assert torch.equal(y[:n], want[0][:n])
        dh = fill(rows, halves * inner) if fp8 else fill(rows, halves * inner, t=torch.bfloat16)
        ds, y2 = fill(halves * blocks, rows), fill(rows, inner) if fp8 else fill(rows, inner, t=torch.bfloat16)
        assert lib.kgw_moe_act_fp8_grad(p(dy), dy.stride(0), code, kgw._ACTS[act], p(saved), p(ss), p(offsets), 3, rows, inner, p(dh),
                                        p(ds) if fp8 else None, p(y2), p(ys) if fp8 else None, stream) == 0
        assert (dh[n:] == 77).all() and (y2[n:] == 77).all() and (ds[:, n if fp8 else 0:] == 77).all() and (ys[:, n if fp8 else 0:] == 77).all()
        if not fp8:
            assert torch.equal(dh[:n], want_grad[0][:n]) and torch.equal(y2[:n], want_grad[2][:n])


def test_gradient_against_differences():
    """sum dy (act(h + d s) - act(h - d s)) / 2d at the kept h, against <dh, s>: act in 64 bits here, so the quotient is off by
    d^2 / 6 times third derivatives (below 2 |u| + 2 for every direction of signs), and dh by its own bound."""
    h = values(20, 256, torch.float32, 4, spread=1.0)
    dy = values(20, 128, torch.float32, 5)
    _, _, saved, scales = kgw.kgw_moe_act_fp8(h)
    kept, s = kept_values(saved, scales, "swiglu"), values(20, 256, torch.float32, 6).sign().double().cpu()
    d = 2.0 ** -10
    dyd = dy.double().cpu()
    want = float((dyd * (forward(kept + d * s, "swiglu")[0] - forward(kept - d * s, "swiglu")[0])).sum() / (2 * d))
    got = float((kgw.kgw_moe_act_fp8_grad(dy, saved, scales)[0].double().cpu() * s).sum())
    _, tol = backward(kept, dyd, "swiglu")
    assert abs(got - want) <= float(tol.sum()) + d * d * float((dyd.abs() * (2 * kept[:, 128:].abs() + 2)).sum())


def test_empty_sizes():
    for rows, inner in ((0, 64), (5, 0)):
        h = torch.empty((rows, 2 * inner), dtype=torch.bfloat16, device=DEV)
        y, _, saved, scales = kgw.kgw_moe_act_fp8(h)
        assert y.shape == (rows, inner) and saved.shape == (rows, 2 * inner)
        dh = kgw.kgw_moe_act_fp8_grad(torch.empty((rows, inner), dtype=torch.bfloat16, device=DEV), saved, scales)[0]
        assert dh.shape == (rows, 2 * inner)


def test_rows_past_four_gigabytes():
    # 300000 rows of 16 KiB: byte offsets pass 2^32; codes 2^31
    rows, inner = 300000, 4096
    h = torch.empty((rows, 2 * inner), dtype=torch.bfloat16, device=DEV)
    h.copy_(((torch.arange(rows, device=DEV) % 251) - 125)[:, None].expand(-1, 2 * inner) * 0.03125)
    assert h.numel() * 2 > 2 ** 32 and h.numel() > 2 ** 31
    y, _, saved, scales = kgw.kgw_moe_act_fp8(h)
    dh = kgw.kgw_moe_act_fp8_grad(y, saved, scales)[0]
    few = kgw.kgw_moe_act_fp8(h[:251])
    few_dh = kgw.kgw_moe_act_fp8_grad(few[0], few[2], few[3])[0]
    for at in (0, 251 * 600, 251 * 1194):
        part = slice(at, at + 251)
        assert torch.equal(y[part], few[0]) and torch.equal(saved[part], few[2]) and torch.equal(scales[:, part], few[3])
        assert torch.equal(dh[part], few_dh)


def test_refusals():
    h = torch.zeros((4, 256), dtype=torch.bfloat16, device=DEV)
    dy = torch.zeros((4, 128), dtype=torch.bfloat16, device=DEV)
    _, _, saved, scales = kgw.kgw_moe_act_fp8(h)
    off = torch.zeros(2, dtype=torch.int32, device=DEV)
    act, grad = kgw.kgw_moe_act_fp8, kgw.kgw_moe_act_fp8_grad
    bad = [lambda: act(h.double()), lambda: act(h[0]), lambda: act(h.t()), lambda: act(h.cpu()), lambda: act(h, act="gelu"),
           lambda: act(h[:, :248]), lambda: act(h[:, :12], act="relu2"), lambda: act(h, offsets=off.long()),
           lambda: act(h, offsets=off.cpu()), lambda: act(h, out=torch.zeros((4, 127), dtype=torch.bfloat16, device=DEV)),
           lambda: act(h, out=torch.zeros((4, 128), device=DEV)), lambda: act(h, fp8=True, out=dy),
           lambda: grad(dy, saved[:, :128], scales), lambda: grad(dy, saved, scales[:1]), lambda: grad(dy, saved, scales, act="relu2"),
           lambda: grad(dy, saved.bfloat16(), scales), lambda: grad(dy.cpu(), saved, scales), lambda: grad(dy, saved.cpu(), scales),
           lambda: grad(dy, saved, scales, dh=dy), lambda: grad(dy, saved, scales, y=dy),
           lambda: grad(dy[:, :100], saved, scales), lambda: grad(dy, saved, scales, offsets=off[:0])]
    for k, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {k} was accepted")
