"""Token sort, permute, unpermute and their gradients against plain 64-bit forms.

The sort's results are whole numbers and compared exactly, as are permute's rows (copies).
Sums: a rounding to type t is off by at most finfo(t).eps / 2 of the value, an fp32 operation
by at most 2^-24.
  * unpermute adds k products in fp32 and rounds once:
        |err| <= eps_t / 2 |out| + (k + 2) 2^-24 sum |w y|
  * dy = w dout is one fp32 product rounded once: |err| <= (eps_t / 2 + 2^-24) |w dout|
  * dw sums at most 8 ceil(H / 2048) + 1 products on one thread and then 8 partial sums up a
    tree: |err| <= (H / 256 + 24) 2^-24 sum |dout y|
plus half the type's smallest step where a value falls below its normal range.
"""
import numpy as np
import pytest
import torch

import grouped_gemm_expert_offsets_amd as kgw

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs an MI355X")]

DEV = "cuda"
U32 = 2.0 ** -24
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def half_step(dtype):
    f = torch.finfo(dtype)
    return f.eps / 2, f.tiny * f.eps / 2


def sort_reference(ids, E, align, rows):
    """The definition, one assignment after the other."""
    flat = ids.reshape(-1).cpu().tolist()
    counts = [0] * E
    for e in flat:
        if 0 <= e < E:
            counts[e] += 1
    offsets, start, acc = [], [], 0
    for c in counts:
        start.append(acc)
        acc += -(-c // align) * align
        offsets.append(min(acc, rows))
    nxt, row_of, src_of = list(start), [], [-1] * rows
    for i, e in enumerate(flat):
        row = -1
        if 0 <= e < E:
            if nxt[e] < rows:
                row = nxt[e]
                src_of[row] = i
            nxt[e] += 1
        row_of.append(row)
    return counts, offsets, row_of, src_of


def check_sort(ids, E, align, rows=None):
    got = kgw.kgw_moe_sort(ids, E, alignment=align, rows=rows)
    rows = kgw.kgw_moe_rows(ids.shape[0], ids.shape[1], E, align) if rows is None else rows
    want = sort_reference(ids, E, align, rows)
    for g, w, name in zip(got, want, ("counts", "offsets", "row_of", "src_of")):
        assert g.dtype == torch.int32
        assert g.reshape(-1).cpu().tolist() == w, name


def random_ids(tokens, k, E, seed, dtype=torch.int64, spread=None):
    g = torch.Generator().manual_seed(seed)
    if spread is not None:                      # ids outside [0, E) among them
        return torch.randint(-spread, E + spread, (tokens, k), generator=g).to(dtype).to(DEV)
    return torch.rand((tokens, max(E, k)), generator=g).topk(k, dim=1).indices.to(dtype).to(DEV)


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("tokens,k,E,align", [(1, 1, 1, 128), (1, 8, 8, 128), (7, 3, 5, 1), (63, 1, 2, 256), (64, 8, 256, 128),
                                              (500, 8, 33, 128), (2049, 2, 64, 256), (5000, 3, 7, 128),
                                              (20011, 2, 300, 128), (3000, 4, 2048, 128), (512, 4, 40, 128),
                                              (683, 3, 40, 128), (8192, 8, 70, 128), (8193, 8, 70, 128)])
def test_sort(tokens, k, E, align, dtype):
    check_sort(random_ids(tokens, k, E, tokens + E, dtype), E, align)


@pytest.mark.parametrize("tokens,k,E", [(33, 4, 6), (4099, 3, 20)])
def test_sort_ids_of_other_ranks(tokens, k, E):
    check_sort(random_ids(tokens, k, E, 5, spread=2 * E), E, 128)
    none = torch.full((tokens, k), E, dtype=torch.int64, device=DEV)
    none[::2] = -1
    none[0, 0] = 2 ** 40 + 1                    # not expert 1 once cut to 32 bits
    check_sort(none, E, 128)


@pytest.mark.parametrize("tokens", [100, 6000])
def test_sort_one_expert_takes_all(tokens):
    ids = torch.full((tokens, 1), 3, dtype=torch.int32, device=DEV)
    check_sort(ids, 5, 128)


@pytest.mark.parametrize("tokens,rows", [(100, 0), (100, 128), (100, 384), (6000, 2048)])
def test_sort_fewer_rows_than_assignments(tokens, rows):
    check_sort(random_ids(tokens, 2, 4, 11), 4, 128, rows=rows)


def test_sort_no_tokens():
    ids = torch.empty((0, 2), dtype=torch.int64, device=DEV)
    check_sort(ids, 3, 128)
    check_sort(ids, 3, 128, rows=256)


def test_sort_more_than_one_round_per_workgroup():
    # 128 workgroups of 2048 hold 262144 assignments; more make every workgroup loop
    ids = random_ids(150001, 2, 9, 3, torch.int32)
    counts, offsets, row_of, src_of = kgw.kgw_moe_sort(ids, 9, alignment=128)
    flat = ids.reshape(-1).long()
    order = torch.sort(flat, stable=True).indices
    want_counts = torch.bincount(flat, minlength=9)
    padded = (want_counts + 127) // 128 * 128
    start = torch.cumsum(padded, 0) - padded
    first = torch.cumsum(want_counts, 0) - want_counts
    rows = (start - first)[flat[order]] + torch.arange(flat.numel(), device=DEV)
    want = torch.empty_like(flat)
    want[order] = rows
    assert torch.equal(counts.long(), want_counts)
    assert torch.equal(offsets.long(), torch.cumsum(padded, 0))
    assert torch.equal(row_of.reshape(-1).long(), want)
    src = torch.full((src_of.numel(),), -1, dtype=torch.int64, device=DEV)
    src[want] = torch.arange(flat.numel(), device=DEV)
    assert torch.equal(src_of.long(), src)


def routed(tokens, k, E, held, align, seed):
    ids = random_ids(tokens, k, E, seed)
    _, offsets, row_of, src_of = kgw.kgw_moe_sort(ids, held, alignment=align)
    return offsets, row_of, src_of


def values(shape, dtype, seed, stride_pad=0, offset=0):
    """Normals in `dtype`, as a view of a wider, shifted buffer when asked."""
    g = torch.Generator().manual_seed(seed)
    rows, cols = shape
    wide = torch.randn((rows * (cols + stride_pad) + offset + 1,), generator=g).to(dtype).to(DEV)
    return wide[offset:offset + rows * (cols + stride_pad)].view(rows, cols + stride_pad)[:, :cols]


def f64(t):
    return t.detach().cpu().double().numpy()


SHAPES = [(1, 1, 1, 1, 1), (1, 4, 4, 4, 8), (3, 2, 5, 2, 7), (17, 3, 8, 8, 129), (64, 8, 64, 64, 512), (130, 2, 4, 3, 2056),
          (9, 8, 16, 16, 7168), (5, 4, 8, 8, 8200), (40, 2, 6, 6, 1001)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,k,E,held,hidden", SHAPES)
@pytest.mark.parametrize("pad,offset", [(0, 0), (3, 1)])
def test_permute(tokens, k, E, held, hidden, dtype, pad, offset):
    _, row_of, src_of = routed(tokens, k, E, held, 128, hidden)
    x = values((tokens, hidden), dtype, 1, pad, offset)
    out = torch.full((src_of.numel(), hidden), float("nan"), dtype=dtype, device=DEV)
    got = kgw.kgw_moe_permute(x, row_of, src_of, out)
    assert got is out
    src = src_of.cpu()
    want = torch.zeros((src.numel(), hidden), dtype=dtype)
    want[src >= 0] = x.cpu()[src[src >= 0].long() // k]
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,k,E,held,hidden", SHAPES)
@pytest.mark.parametrize("weighted,pad,offset", [(True, 0, 0), (True, 5, 1), (False, 0, 0)])
def test_unpermute(tokens, k, E, held, hidden, dtype, weighted, pad, offset):
    _, row_of, src_of = routed(tokens, k, E, held, 128, hidden + 1)
    rows = src_of.numel()
    y = values((rows, hidden), dtype, 2, pad, offset)
    y[src_of < 0] = float("nan")                # rows of no assignment are not read into any sum
    w = torch.softmax(values((tokens, k), torch.float32, 3), 1).contiguous() if weighted else None
    got = f64(kgw.kgw_moe_unpermute(y, row_of, w))
    r, yd = row_of.cpu().numpy(), f64(y)
    wd = f64(w) if weighted else np.ones((tokens, k))
    want, size = np.zeros((tokens, hidden)), np.zeros((tokens, hidden))
    for j in range(k):
        at = r[:, j] >= 0
        term = wd[at, j, None] * yd[r[at, j]]
        want[at] += term
        size[at] += np.abs(term)
    rel, tiny = half_step(dtype)
    assert np.all(np.abs(got - want) <= rel * np.abs(want) + (1 + rel) * (k + 2) * U32 * size + tiny)
    lost = (r < 0).all(1)
    assert np.all(got[lost] == 0) and not np.signbit(got[lost]).any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,k,E,held,hidden", SHAPES + [(3, 2, 4, 4, 20000)])
@pytest.mark.parametrize("pad,offset", [(0, 0), (5, 1)])
def test_unpermute_grad(tokens, k, E, held, hidden, dtype, pad, offset):
    _, row_of, src_of = routed(tokens, k, E, held, 128, hidden + 2)
    rows = src_of.numel()
    y = values((rows, hidden), dtype, 4, pad, offset)
    y[src_of < 0] = float("nan")
    dout = values((tokens, hidden), dtype, 5, pad, offset)
    w = torch.softmax(values((tokens, k), torch.float32, 6), 1).contiguous()
    dy = torch.full((rows, hidden), float("nan"), dtype=dtype, device=DEV)
    dw = torch.full((tokens, k), float("nan"), dtype=torch.float32, device=DEV)
    kgw.kgw_moe_unpermute_grad(dout, y, row_of, src_of, w, dy, dw)
    r, yd, dd, wd = row_of.cpu().numpy(), f64(y), f64(dout), f64(w)
    want_dy, want_dw, size = np.zeros((rows, hidden)), np.zeros((tokens, k)), np.zeros((tokens, k))
    for j in range(k):
        at = r[:, j] >= 0
        want_dy[r[at, j]] = wd[at, j, None] * dd[at]
        term = dd[at] * yd[r[at, j]]
        want_dw[at, j], size[at, j] = term.sum(1), np.abs(term).sum(1)
    rel, tiny = half_step(dtype)
    got_dy, got_dw = f64(dy), f64(dw)
    assert np.all(np.abs(got_dy - want_dy) <= (rel + 1.01 * U32) * np.abs(want_dy) + tiny)
    assert np.all(got_dy[src_of.cpu().numpy() < 0] == 0)
    assert np.all(np.abs(got_dw - want_dw) <= (hidden / 256 + 24) * U32 * size)
    assert np.all(got_dw[r < 0] == 0)


def test_gradients_against_differences():
    """<out(y + s) - out(y), dout> = <s, dy>, and the same for the weights and for permute, exactly:
    the maps are linear and small integers stay whole in fp32."""
    tokens, k, E, hidden = 50, 3, 9, 77
    _, row_of, src_of = routed(tokens, k, E, 6, 128, 1)
    g = torch.Generator().manual_seed(0)
    whole = lambda *shape: torch.randint(-4, 5, shape, generator=g).float().to(DEV)  # noqa: E731
    rows = src_of.numel()
    y, s, dout = whole(rows, hidden), whole(rows, hidden), whole(tokens, hidden)
    w, sw = whole(tokens, k), whole(tokens, k)
    dy, dw = kgw.kgw_moe_unpermute_grad(dout, y, row_of, src_of, w)
    base = kgw.kgw_moe_unpermute(y, row_of, w).double()
    assert ((kgw.kgw_moe_unpermute(y + s, row_of, w).double() - base) * dout.double()).sum() == \
        (dy.double() * s.double()).sum()
    assert ((kgw.kgw_moe_unpermute(y, row_of, w + sw).double() - base) * dout.double()).sum() == \
        (dw.double() * sw.double()).sum()
    x, sx, drows = whole(tokens, hidden), whole(tokens, hidden), whole(rows, hidden)
    dx = kgw.kgw_moe_unpermute(drows, row_of)
    moved = kgw.kgw_moe_permute(x + sx, row_of, src_of).double() - kgw.kgw_moe_permute(x, row_of, src_of).double()
    assert (moved * drows.double()).sum() == (dx.double() * sx.double()).sum()


def test_infinities_and_nan_stay_in_their_rows():
    tokens, k, hidden = 6, 2, 40
    _, row_of, src_of = routed(tokens, k, 4, 4, 128, 8)
    y = torch.ones((src_of.numel(), hidden), device=DEV)
    y[row_of[2, 0].long(), 5] = float("inf")
    y[row_of[4, 1].long(), 7] = float("nan")
    w = torch.full((tokens, k), 0.5, device=DEV)
    out = kgw.kgw_moe_unpermute(y, row_of, w)
    want = torch.ones((tokens, hidden), device=DEV)
    want[2, 5], want[4, 7] = float("inf"), float("nan")
    assert torch.equal(torch.nan_to_num(out, nan=-7.0), torch.nan_to_num(want, nan=-7.0))


def test_rows_out_of_range_are_skipped():
    # a row_of that no sort made: rows outside the buffer are neither read nor written
    x = torch.arange(8, dtype=torch.float32, device=DEV).view(4, 2) + 1
    row_of = torch.tensor([[0], [-5], [3], [2]], dtype=torch.int32, device=DEV)
    src_of = torch.tensor([0, -1, 3], dtype=torch.int32, device=DEV)
    out = kgw.kgw_moe_permute(x, row_of, src_of)
    assert out.tolist() == [[1, 2], [0, 0], [7, 8]]
    w = torch.ones((4, 1), device=DEV)
    assert kgw.kgw_moe_unpermute(out, row_of, w).tolist() == [[1, 2], [0, 0], [0, 0], [7, 8]]
    dy, dw = kgw.kgw_moe_unpermute_grad(x, out, row_of, src_of, w)
    assert dy.tolist() == [[1, 2], [0, 0], [7, 8]] and dw[:, 0].tolist() == [5, 0, 0, 113]


def test_empty_sizes():
    none = torch.empty((0, 2), dtype=torch.int32, device=DEV)
    pads = torch.full((128,), -1, dtype=torch.int32, device=DEV)
    assert kgw.kgw_moe_permute(torch.empty((0, 16), device=DEV), none, pads).abs().sum() == 0
    assert kgw.kgw_moe_unpermute(torch.empty((0, 16), device=DEV), torch.full((3, 2), -1, dtype=torch.int32, device=DEV)
                                 ).tolist() == [[0.0] * 16] * 3
    one = torch.zeros((3, 1), dtype=torch.int32, device=DEV)
    dy, dw = kgw.kgw_moe_unpermute_grad(torch.empty((3, 0), device=DEV), torch.empty((128, 0), device=DEV), one, pads,
                                        torch.ones((3, 1), device=DEV))
    assert dy.shape == (128, 0) and dw.tolist() == [[0.0]] * 3


def test_on_another_stream_and_in_a_graph():
    tokens, k, E, hidden = 300, 2, 8, 264
    ids = random_ids(tokens, k, E, 4)
    x = values((tokens, hidden), torch.bfloat16, 1)
    w = torch.softmax(values((tokens, k), torch.float32, 3), 1).contiguous()

    def step(stream=None):
        _, _, row_of, src_of = kgw.kgw_moe_sort(ids, E, stream=stream)
        rows = kgw.kgw_moe_permute(x, row_of, src_of, stream=stream)
        out = kgw.kgw_moe_unpermute(rows, row_of, w, stream=stream)
        return (rows, out) + kgw.kgw_moe_unpermute_grad(x, rows, row_of, src_of, w, stream=stream)

    want = step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for r in range(4):
        for t in held:
            t.fill_(float("nan"))
        ids.copy_(random_ids(tokens, k, E, 10 + r))
        x.mul_(0.5)
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want)), r


def test_rows_past_four_gigabytes():
    # 600000 rows of 8 KiB: byte offsets pass 2^32
    tokens, k, hidden = 300000, 2, 4096
    ids = torch.stack([torch.zeros(tokens, dtype=torch.int32), torch.ones(tokens, dtype=torch.int32)], 1).to(DEV)
    _, offsets, row_of, src_of = kgw.kgw_moe_sort(ids, 2)
    x = torch.empty((tokens, hidden), dtype=torch.bfloat16, device=DEV)
    x.copy_((torch.arange(tokens, device=DEV) % 251)[:, None].expand(-1, hidden))
    rows = kgw.kgw_moe_permute(x, row_of, src_of)
    assert rows.numel() * 2 > 2 ** 32
    at = torch.tensor([0, 1, tokens // 2, tokens - 1], device=DEV)
    for j in range(2):
        assert torch.equal(rows[row_of[at, j].long()], x[at])
    back = kgw.kgw_moe_unpermute(rows, row_of, torch.full((tokens, k), 0.5, device=DEV))
    assert torch.equal(back, x)


def test_refusals():
    ids = torch.zeros((4, 2), dtype=torch.int64, device=DEV)
    _, _, row_of, src_of = kgw.kgw_moe_sort(ids, 3)
    x = torch.zeros((4, 16), device=DEV)
    bad = [lambda: kgw.kgw_moe_sort(ids.float(), 3), lambda: kgw.kgw_moe_sort(ids.t(), 3),
           lambda: kgw.kgw_moe_sort(ids[0], 3), lambda: kgw.kgw_moe_sort(ids, 0),
           lambda: kgw.kgw_moe_sort(ids, 2049), lambda: kgw.kgw_moe_sort(ids, 3, rows=100),
           lambda: kgw.kgw_moe_sort(ids, 3, alignment=0), lambda: kgw.kgw_moe_sort(ids.cpu(), 3),
           lambda: kgw.kgw_moe_permute(x.double(), row_of, src_of), lambda: kgw.kgw_moe_permute(x[:3], row_of, src_of),
           lambda: kgw.kgw_moe_permute(x.t(), row_of, src_of), lambda: kgw.kgw_moe_permute(x, row_of.long(), src_of),
           lambda: kgw.kgw_moe_permute(x, row_of, src_of.cpu()), lambda: kgw.kgw_moe_permute(x.cpu(), row_of, src_of),
           lambda: kgw.kgw_moe_permute(x, row_of, src_of, out=torch.zeros((1, 16), device=DEV)),
           lambda: kgw.kgw_moe_unpermute(x, row_of, torch.zeros((4, 3), device=DEV)),
           lambda: kgw.kgw_moe_unpermute(x, row_of, torch.zeros((4, 2), dtype=torch.float64, device=DEV)),
           lambda: kgw.kgw_moe_unpermute(x[:, None], row_of),
           lambda: kgw.kgw_moe_unpermute_grad(x, x, row_of, src_of, torch.zeros((4, 2), device=DEV)),
           lambda: kgw.kgw_moe_unpermute_grad(x[:2], x, row_of, src_of[:4], torch.zeros((4, 2), device=DEV))]
    for k, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {k} was accepted")
