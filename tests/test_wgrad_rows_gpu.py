"""Weight gradients from 8-bit token rows.  Their values are bf16 values, so the results are bit for bit those of the
bf16 product of the same rows (itself held to the CPU oracle elsewhere) where that takes the counts, and within the
oracle's tolerances otherwise."""
import numpy as np
import pytest
import torch

import grouped_gemm_expert_offsets_amd as kgw
import oracle
from helpers import assert_bf16_close, assert_fp16_close, assert_fp32_close, to_f64

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs an MI355X")]

DEV = "cuda"
SIZES = [([256, 0, 512, 768], 256, 512), ([256, 0, 512, 768], 272, 400), ([512, 256], 16, 16), ([256], 128, 144), ([256] * 5, 1040, 784),
         ([2048] * 3 + [1024], 320, 384), ([4096, 0, 8192, 256], 320, 384), ([0, 0, 256], 144, 528),
         ([1024 + 256 * (e % 5) for e in range(32)], 2048, 2048), ([256, 512], 24, 264), ([512, 256], 264, 776), ([256], 776, 24), ([256, 256], 8, 136), ([256], 136, 8),
         ([256, 256], 1048, 520)]


def rows8(tokens, cols, seed):
    """Random codes (every finite one) and scale bytes within 2^-10 .. 2^10, and the bf16 rows that they stand for."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    codes = torch.randint(0, 256, (tokens, cols), generator=g, device=DEV, dtype=torch.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0x38
    scales = torch.randint(117, 138, (-(-cols // 128), tokens), generator=g, device=DEV, dtype=torch.uint8)
    return codes, scales, decode(codes, scales)


def decode(codes, scales):
    v = codes.view(torch.float8_e4m3fn).bfloat16()
    s = (scales.int() << 7).to(torch.int16).view(torch.bfloat16)
    return v * s.t().repeat_interleave(128, 1)[:, :v.shape[1]]


def offsets_of(counts):
    return torch.cumsum(torch.tensor(counts), 0).int().to(DEV)


@pytest.mark.parametrize("both", [False, True])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("counts,hidden,n", SIZES)
def test_equals_the_bf16_product_of_the_same_rows(counts, hidden, n, out_dtype, both):
    T, E = sum(counts), len(counts)
    A, sa, a = rows8(T, hidden, 1)
    B, sb, b = rows8(T, n, 2)
    off = offsets_of(counts)
    out = torch.full((E, hidden, n), float("nan"), dtype=out_dtype, device=DEV)
    got = kgw.kgw_wgrad_fp8_rows(A, sa, B if both else b, off, sb=sb if both else None, out=out)
    one = kgw.kgw_wgrad_fp8_rows(A.view(torch.float8_e4m3fn), sa, B.view(torch.float8_e4m3fn) if both else b, off,
                                 sb=sb if both else None, out_dtype=out_dtype, split_k=False)
    want = kgw.kgw_wgrad_bf16_ex(a, b, off, a_major="m", out_dtype=out_dtype, split_k=False)
    assert got is out and torch.equal(one, want)
    if kgw.load_library().kgw_wgrad_fp8_rows_workspace_bytes(E, hidden, n, T) <= 256:
        assert torch.equal(got, want)
    else:                                                   # shares of the tokens summed apart: another order of the same sums
        exact = to_f64(kgw.kgw_wgrad_bf16_ex(a, b, off, a_major="m", split_k=False))
        if out_dtype == torch.float32:
            assert_fp32_close(to_f64(got), exact)
        elif out_dtype == torch.bfloat16:
            assert_bf16_close(to_f64(got), exact)
        else:
            past = np.abs(exact) > 6e4                      # (beyond fp16: infinities of the same sign)
            g = to_f64(got)
            assert np.array_equal(np.sign(g[past]), np.sign(exact[past]))
            assert_fp16_close(np.where(past, 0, g), np.where(past, 0, exact))


@pytest.mark.parametrize("both", [False, True])
@pytest.mark.parametrize("counts,hidden,n", [([128], 64, 48), ([128, 384, 0, 640], 272, 160), ([128] * 7, 48, 272)])
def test_counts_of_128(counts, hidden, n, both):
    T = sum(counts)
    A, sa, a = rows8(T, hidden, 3)
    B, sb, b = rows8(T, n, 4)
    off = offsets_of(counts)
    want = oracle.wgrad_bf16(a.t().contiguous().cpu(), b.cpu(), off.cpu())
    call = lambda t: to_f64(kgw.kgw_wgrad_fp8_rows(A, sa, B if both else b, off, sb=sb if both else None, out_dtype=t))  # noqa: E731
    assert_fp32_close(call(torch.float32), want)
    assert_bf16_close(call(torch.bfloat16), want)
    if np.abs(want).max() < 6e4:
        assert_fp16_close(call(torch.float16), want)


@pytest.mark.parametrize("both", [False, True])
def test_accumulate_and_discrete_outputs(both):
    counts, hidden, n = [256, 0, 768], 144, 272
    A, sa, a = rows8(sum(counts), hidden, 5)
    B, sb, b = rows8(sum(counts), n, 6)
    off = offsets_of(counts)
    kw = dict(sb=sb if both else None)
    start = torch.randn((3, hidden, n), generator=torch.Generator().manual_seed(1)).to(DEV)
    got = kgw.kgw_wgrad_fp8_rows(A, sa, B if both else b, off, out=start.clone(), accumulate=True, **kw)
    want = kgw.kgw_wgrad_bf16_ex(a, b, off, a_major="m", out=start.clone(), accumulate=True)
    assert torch.equal(got, want) and torch.equal(got[1], start[1])
    outs = [torch.full((hidden, n), 7.0, device=DEV), torch.full((hidden, n), 7.0, device=DEV), None]
    got = kgw.kgw_wgrad_fp8_rows(A, sa, B if both else b, off, outs=outs, **kw)
    plain = kgw.kgw_wgrad_bf16_ex(a, b, off, a_major="m")
    assert got[2] is None and torch.equal(outs[0], plain[0]) and not outs[1].any()


@pytest.mark.parametrize("both", [False, True])
def test_rows_past_the_last_offset(both):
    counts, hidden, n = [256, 512], 144, 272
    T = 1280
    A, sa, a = rows8(T, hidden, 7)
    B, sb, b = rows8(T, n, 8)
    off = offsets_of(counts)
    want = kgw.kgw_wgrad_bf16_ex(a[:768].contiguous(), b[:768].contiguous(), off, a_major="m")
    A[768:], sa[:, 768:], B[768:], sb[:, 768:], b[768:] = 0x7F, 0xFF, 0x7F, 0xFF, float("nan")
    got = kgw.kgw_wgrad_fp8_rows(A, sa, B if both else b, off, sb=sb if both else None)
    assert torch.equal(got, want)


def test_every_code_and_scale():
    """One token an expert's row: out = a_m b_n shows every value of every code at every scale that bf16 holds; a NaN scale
    or code reaches its own outputs alone."""
    T, hidden = 256, 256
    codes = torch.arange(256, dtype=torch.uint8).repeat(T, 1).to(DEV)
    codes[(codes & 0x7F) == 0x7F] = 0
    scales = torch.arange(2, 258).clamp(max=240).to(torch.uint8).repeat(2, 1).to(DEV)      # token t: 2^(t + 2 - 127)
    b = torch.zeros((T, 256), dtype=torch.bfloat16, device=DEV)
    b[torch.arange(256), torch.arange(256)] = 1.0
    got = kgw.kgw_wgrad_fp8_rows(codes, scales, b, offsets_of([T]))[0]
    want = decode(codes, scales).double()
    exact = codes.view(torch.float8_e4m3fn).double() * torch.exp2(scales[0].double() - 127)[:, None]
    normal = (exact.abs() >= 2.0 ** -126) | (exact == 0)
    assert torch.equal(want[normal], exact[normal])
    assert bool(((got.t().double() - exact).abs()[normal] == 0).all())
    assert bool(((got.t().double() - exact).abs() <= 2.0 ** -126).all())
    sa = torch.full((2, T), 127, dtype=torch.uint8, device=DEV)
    A = torch.full((T, hidden), 0x38, dtype=torch.uint8, device=DEV)
    sa[1, 9], A[20, 3] = 0xFF, 0x7F
    bad = kgw.kgw_wgrad_fp8_rows(A, sa, torch.ones((T, 16), dtype=torch.bfloat16, device=DEV), offsets_of([T]))[0].isnan()
    assert bad[128:].all() and bad[3].all() and int(bad.sum()) == 129 * 16


def test_malformed_offsets_stay_in_bounds():
    A, sa, a = rows8(512, 128, 1)
    _, _, b = rows8(512, 128, 2)
    for bad in ([512, 128, 512], [-128, 256, 100000], [100, 333, 512], [0, 0, 0]):
        off = torch.tensor(bad, dtype=torch.int32, device=DEV)
        got = kgw.kgw_wgrad_fp8_rows(A, sa, b, off)
        assert torch.equal(got, kgw.kgw_wgrad_bf16_ex(a, b, off, a_major="m"))


def test_operands_past_four_gigabytes():
    # 600064 tokens x 7168 codes pass 2^32 bytes; the last expert's rows lie behind them
    T, hidden, n = 600064, 7168, 64
    A = torch.full((T, hidden), 0x38, dtype=torch.uint8, device=DEV)
    sa = torch.full((56, T), 127, dtype=torch.uint8, device=DEV)
    b = torch.zeros((T, n), dtype=torch.bfloat16, device=DEV)
    A[-128:, 5], sa[55, -128:], b[-128:] = 0x40, 128, 1.0
    b[0] = 1.0
    out = kgw.kgw_wgrad_fp8_rows(A, sa, b, torch.tensor([256, T], dtype=torch.int32, device=DEV))
    want = torch.full((hidden,), 128.0, device=DEV)
    want[5], want[55 * 128:] = 256.0, 256.0
    assert torch.equal(out[1], want[:, None].expand(-1, n)) and bool((out[0] == 1).all())


def test_refusals():
    A, sa, _ = rows8(256, 128, 1)
    B, sb, b = rows8(256, 128, 2)
    off = offsets_of([256])
    f = kgw.kgw_wgrad_fp8_rows
    odd = lambda c: (torch.zeros((256, c), dtype=torch.uint8, device=DEV), torch.zeros((-(-c // 128), 256), dtype=torch.uint8, device=DEV))  # noqa: E731
    bad = [lambda: f(b, sa, b, off), lambda: f(A, sa, B, off), lambda: f(A, sa, b, off, sb=sb), lambda: f(A, None, b, off),
           lambda: f(A, sa.int(), b, off), lambda: f(A, sa[:, :255], b, off), lambda: f(A, sa.t(), b, off), lambda: f(A, sa.cpu(), b, off),
           lambda: f(A[:128], sa, b, off), lambda: f(A.t(), sa, b, off), lambda: f(A, sa, b, off.long()), lambda: f(A, sa, b, off.cpu()),
           lambda: f(A[:200].contiguous(), sa[:, :200].contiguous(), b[:200].contiguous(), off), lambda: f(*odd(124), b, off),
           lambda: f(A, sa, odd(124)[0], off, sb=odd(124)[1]), lambda: f(A, sa, b[:, :100].contiguous(), off),
           lambda: f(A, sa, b, off, out_dtype=torch.float64), lambda: f(A, sa, b, off, accumulate=True),
           lambda: f(A, sa, b, off, out=torch.zeros((1, 128, 127), device=DEV)),
           lambda: f(A, sa, b, torch.tensor([100], dtype=torch.int32, device=DEV), validate=True)]
    for k, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {k} was accepted")
