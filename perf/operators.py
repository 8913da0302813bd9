"""Operators around the expert products: tokens sorted by expert and brought back, with their
gradients, and weight gradients orthogonalised by Newton-Schulz products.

Five calls are covered.  With T tokens, k experts each, E experts held here, H values a token and
R rows sorted by expert (every expert's rows padded to a multiple of `align`, the grouping that
the expert products take):

    sort            ids (T, k)                    -> counts, offsets (E), row_of (T, k), src_of (R)
    permute         x (T, H)                      -> rows (R, H), padding rows zero
    unpermute       y (R, H), weights (T, k)      -> out_t = sum_j w_tj y[row_of_tj]
                    (without weights: the gradient of permute)
    unpermute_grad  dout (T, H), y, weights       -> dy_r = w dout_t, dw_tj = <dout_t, y[row_of_tj]>
    newton_schulz   G (B, m, n), `steps` steps of X <- a X + (b A + c A A) X, A = X X^T,
                    from X = G / (|G| + eps)

An id outside [0, E) names an expert of another rank: its assignment has row_of = -1, takes no row
and no part in the sums, and its dw is 0.

`own = False` computes them from elementary torch operations in 32 bits (sums that decide the
scale of a matrix in 64); `own = True` calls the package.
"""
import math

import torch

own = False

DEV = "cuda"
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
EPS = 1e-7
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def _route(op, name, tokens, k, experts, held, align, hidden=0, dtype="bf16", weights=True):
    """A routed case: `held` of the `experts` are on this rank (held == experts: all of them)."""
    return dict(name=name, op=op, tokens=tokens, k=k, experts=experts, held=held, align=align, hidden=hidden,
                dtype=dtype, weights=weights)


def _ns(name, batch, m, n, dtype, out, steps=5):
    return dict(name=name, op="newton_schulz", batch=batch, m=m, n=n, dtype=dtype, out=out, steps=steps)


def listed():
    return [
        # A step of decoding: 64 sequences, 8 of 256 experts each; one short call, latency counts.
        _route("sort", "sort decode 64x8 E256", 64, 8, 256, 256, 128),
        # A training step of the 32-expert fp8 layer (about 264k rows): 32768 tokens, 8 of 32 experts.
        _route("sort", "sort train 32768x8 E32", 32768, 8, 32, 32, 128),
        # The decoding step's rows; most of what is written is padding, as every touched expert gets 128 rows.
        _route("permute", "permute decode 64x8 H7168", 64, 8, 256, 256, 128, 7168),
        # The training step's rows at the fp8 layer's hidden size.
        _route("permute", "permute train 32768x8 H7168", 32768, 8, 32, 32, 128, 7168),
        # Expert outputs back to their tokens, weighted: the training step again.
        _route("unpermute", "unpermute train 32768x8 H7168", 32768, 8, 32, 32, 128, 7168),
        # The gradient of permute (no weights) on one rank of an expert-parallel group that holds 8 of 32
        # experts, in fp32 with an odd token count and an odd row length.
        _route("unpermute", "permute grad 4099x6 H1001 fp32", 4099, 6, 32, 8, 256, 1001, "fp32", weights=False),
        # Gradients of the weighted sum for the training step of the 8-expert layer of hidden size 4096.
        _route("unpermute_grad", "unpermute grad 16384x2 H4096", 16384, 2, 8, 8, 256, 4096),
        # The same for a short ragged batch in fp16, where some tokens lose assignments to other ranks.
        _route("unpermute_grad", "unpermute grad 777x4 H2056 fp16", 777, 4, 64, 48, 128, 2056, "fp16"),
        # The smallest weight gradients the tests use (E=4, 256 x 512), fp32 throughout: many short products.
        _ns("newton-schulz 4x256x512 fp32", 4, 256, 512, "fp32", "fp32"),
        # Odd sizes, taller than wide, bf16 gradients and a master copy in fp32.
        _ns("newton-schulz 3x1777x1000", 3, 1777, 1000, "bf16", "fp32"),
        # The 8-expert layer's weight gradients.
        _ns("newton-schulz 8x4096x2048 bf16", 8, 4096, 2048, "bf16", "bf16"),
        # Eight experts of the 32-expert fp8 layer: the largest matrices.
        _ns("newton-schulz 8x7168x4096 bf16", 8, 7168, 4096, "bf16", "bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_route(rng, op):
    experts = _log_int(rng, 2, 256)
    held = experts if rng.random() < 0.6 else max(1, experts // rng.choice((2, 4, 8)))
    k = rng.randint(1, min(8, experts))
    align = rng.choice((128, 256))
    least = 16 if held == experts else 64             # enough for other inputs to give other outputs
    if op == "sort":
        return dict(op=op, tokens=_log_int(rng, least, 32768), k=k, experts=experts, held=held, align=align, hidden=0,
                    dtype="bf16", weights=True)
    hidden = _log_int(rng, 64, 7168)
    if rng.random() < 0.7:
        hidden = (hidden + 7) // 8 * 8
    dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
    most = 32768 * 8 * 7168 * 2 // (k * hidden * SIZE[dtype])           # the largest listed case's rows
    tokens = _log_int(rng, least, min(32768, most // 2))
    return dict(op=op, tokens=tokens, k=k, experts=experts, held=held, align=align, hidden=hidden, dtype=dtype,
                weights=op != "unpermute" or rng.random() < 0.7)


def draw(rng):
    op = rng.choice(("sort", "permute", "unpermute", "unpermute_grad", "newton_schulz", "newton_schulz"))
    if op != "newton_schulz":
        return _draw_route(rng, op)
    m, n = _log_int(rng, 24, 7168), _log_int(rng, 24, 4096)
    if rng.random() < 0.5:
        m, n = (m + 7) // 8 * 8, (n + 7) // 8 * 8
    dtype, out = rng.choice((("bf16", "bf16"), ("fp32", "bf16"), ("bf16", "fp32"), ("fp32", "fp32"), ("fp16", "bf16")))
    r, c = min(m, n), max(m, n)
    most = 8 * 4096 * 4096 * 7168 // (r * r * c + r * r * r // 2)
    batch = _log_int(rng, 1, max(1, min(32, most, (1 << 28) // (m * n))))
    return dict(op=op, batch=batch, m=m, n=n, dtype=dtype, out=out, steps=rng.choice((5, 5, 5, 3, 6)))


def _rows(case):
    """Rows that always suffice: every expert that gets a token wastes at most align - 1 of them."""
    assignments = case["tokens"] * case["k"]
    return (assignments + min(case["held"], assignments) * (case["align"] - 1)) // case["align"] * case["align"]


def work(case):
    if case["op"] == "newton_schulz":
        b, r, c = case["batch"], min(case["m"], case["n"]), max(case["m"], case["n"])
        # The two products with a symmetric result need one of its halves; a bf16 result needs one
        # product each, a longer one three products of 16-bit halves.
        flops = case["steps"] * b * (r * r * c + r * r * r + 2.0 * r * r * c) * (1 if case["out"] == "bf16" else 3)
        return {"bytes": b * r * c * (SIZE[case["dtype"]] + SIZE[case["out"]]), "flops": flops}
    t, k, h, rows = case["tokens"], case["k"], case["hidden"], _rows(case)
    n, es = t * k, SIZE[case["dtype"]]
    here = n * case["held"] / case["experts"]         # assignments that stay on this rank, on average
    if case["op"] == "sort":
        return {"bytes": 8 * n + 4 * n + 4 * rows + 8 * case["held"], "flops": 0}
    if case["op"] == "permute":
        return {"bytes": (t + rows) * h * es + 4 * n + 4 * rows, "flops": 0}
    if case["op"] == "unpermute":
        return {"bytes": (here + t) * h * es + (8 if case["weights"] else 4) * n, "flops": 2 * here * h}
    return {"bytes": (t + here + rows) * h * es + 12 * n + 4 * rows, "flops": 3 * here * h}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _ids(case, g):
    """Distinct experts a token, popular ones more often (0.7 to 1.3 times the mean), int64 as topk gives them."""
    t, k, e = case["tokens"], case["k"], case["experts"]
    popular = torch.log(0.7 + 0.6 * torch.rand(e, generator=g, device=DEV))
    gumbel = -torch.log(-torch.log(torch.rand((t, e), generator=g, device=DEV).clamp_(1e-7, 1 - 1e-7)))
    return (gumbel + popular).topk(k, dim=1).indices


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = {"case": case}
    if case["op"] == "newton_schulz":
        # Sums of outer products whose strength falls off along a power law, as gradients have it;
        # of four or more experts one got no token, so its gradient is zero.
        b, m, n = case["batch"], case["m"], case["n"]
        r = min(m, n)
        strength = 0.02 * torch.arange(1, r + 1, device=DEV, dtype=torch.float32) ** -0.75
        G = torch.empty((b, m, n), dtype=DTYPES[case["dtype"]], device=DEV)
        for i in range(b):
            left = torch.randn((m, r), generator=g, device=DEV) * strength
            G[i] = left @ torch.randn((r, n), generator=g, device=DEV)
        if b >= 4:
            G[1] = 0
        s["G"] = G
        return s
    ids = _ids(case, g)
    s["rows"] = _rows(case)
    if case["op"] == "sort":
        s["ids"] = ids
        return s
    _, _, s["row_of"], s["src_of"] = _sort(ids, case["held"], case["align"], s["rows"])
    dt, t, h = DTYPES[case["dtype"]], case["tokens"], case["hidden"]
    if case["op"] in ("permute", "unpermute_grad"):
        s["x"] = torch.randn((t, h), generator=g, device=DEV).to(dt)      # tokens, or the gradient of the sum
    if case["op"] in ("unpermute", "unpermute_grad"):
        s["y"] = torch.empty((s["rows"], h), dtype=dt, device=DEV)
        for part in s["y"].split(1 << 14):
            part.copy_(torch.randn(part.shape, generator=g, device=DEV))
        s["y"].mul_((s["src_of"] >= 0)[:, None])                          # padding rows of an expert product are zero
    s["weights"] = None
    if case["weights"] and case["op"] != "permute":
        s["weights"] = torch.softmax(torch.randn((t, case["k"]), generator=g, device=DEV), dim=1)
    return s


# ----------------------------------------------------------------------------
# the plain forms
# ----------------------------------------------------------------------------
def _sort(ids, held, align, rows):
    flat = ids.reshape(-1).long()
    n = flat.numel()
    key = torch.where((flat >= 0) & (flat < held), flat, held)            # assignments of other ranks come last
    key, order = torch.sort(key, stable=True)
    counts = torch.zeros(held + 1, dtype=torch.int64, device=ids.device).scatter_add_(0, key, torch.ones_like(key))
    padded = (counts + align - 1) // align * align
    ends = torch.cumsum(padded[:held], 0)
    first = torch.cumsum(counts, 0) - counts
    start = torch.cumsum(padded, 0) - padded
    row = start[key] + torch.arange(n, device=ids.device) - first[key]
    row = torch.where((key < held) & (row < rows), row, -1)
    row_of = torch.empty(n, dtype=torch.int32, device=ids.device).scatter_(0, order, row.int())
    src_of = torch.full((rows + 1,), -1, dtype=torch.int32, device=ids.device)
    src_of.scatter_(0, torch.where(row >= 0, row, rows), order.int())
    src_of = src_of[:rows].clone()
    return counts[:held].int(), ends.clamp(max=rows).int(), row_of.reshape(ids.shape), src_of


def _permute(x, src_of, k):
    taken = x[src_of.clamp(min=0).long() // k]
    return torch.where((src_of >= 0)[:, None], taken, torch.zeros((), dtype=x.dtype, device=x.device))


def _unpermute(y, row_of, weights):
    here = row_of >= 0
    terms = y[row_of.clamp(min=0).long()].float()
    if weights is not None:
        terms = terms * weights[..., None]
    return torch.where(here[..., None], terms, 0.0).sum(1).to(y.dtype)


def _unpermute_grad(dout, y, row_of, src_of, weights):
    d, k = dout.float(), row_of.shape[1]
    taken = y[row_of.clamp(min=0).long()].float()
    dw = torch.where(row_of >= 0, (taken * d[:, None]).sum(-1), 0.0)
    del taken
    src = src_of.clamp(min=0).long()
    dy = torch.where((src_of >= 0)[:, None], d[src // k] * weights.reshape(-1)[src][:, None], 0.0)
    return dy.to(y.dtype), dw


def _newton_schulz(G, steps, dtype):
    a, b, c = COEFFICIENTS
    norm = G.double().square().sum((1, 2), keepdim=True).sqrt()
    X = (G.float() / (norm + EPS).float())
    tall = X.shape[1] > X.shape[2]
    if tall:
        X = X.transpose(1, 2).contiguous()
    for _ in range(steps):
        A = torch.bmm(X, X.transpose(1, 2).contiguous())
        X = a * X + torch.bmm(b * A + c * torch.bmm(A, A), X)
    return (X.transpose(1, 2).contiguous() if tall else X).to(dtype)


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import grouped_gemm_expert_offsets_amd as kgw
        if op == "sort":
            return kgw.kgw_moe_sort(s["ids"], case["held"], alignment=case["align"], rows=s["rows"])
        if op == "permute":
            return kgw.kgw_moe_permute(s["x"], s["row_of"], s["src_of"])
        if op == "unpermute":
            return kgw.kgw_moe_unpermute(s["y"], s["row_of"], s["weights"])
        if op == "unpermute_grad":
            return kgw.kgw_moe_unpermute_grad(s["x"], s["y"], s["row_of"], s["src_of"], s["weights"])
        return kgw.kgw_newton_schulz(s["G"], steps=case["steps"], coefficients=COEFFICIENTS, eps=EPS,
                                     out_dtype=DTYPES[case["out"]])
    if op == "sort":
        return _sort(s["ids"], case["held"], case["align"], s["rows"])
    if op == "permute":
        return _permute(s["x"], s["src_of"], case["k"])
    if op == "unpermute":
        return _unpermute(s["y"], s["row_of"], s["weights"])
    if op == "unpermute_grad":
        return _unpermute_grad(s["x"], s["y"], s["row_of"], s["src_of"], s["weights"])
    return _newton_schulz(s["G"], case["steps"], DTYPES[case["out"]])


# ----------------------------------------------------------------------------
# the definition in 64 bits
# ----------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "sort":
        return None
    s = prepare(case, seed)
    if case["op"] == "newton_schulz":
        out = s["G"].double()
        for i in range(out.shape[0]):                 # one matrix at a time, products nested from the inside
            X = out[i] / (torch.linalg.vector_norm(out[i]) + EPS)
            X = X.t().contiguous() if X.shape[0] > X.shape[1] else X
            Xt = None
            for _ in range(case["steps"]):
                Xt = X.t().contiguous()
                AX = X @ (Xt @ X) if X.shape[0] == X.shape[1] else (X @ Xt) @ X
                X = COEFFICIENTS[0] * X + COEFFICIENTS[1] * AX + COEFFICIENTS[2] * (X @ Xt @ AX)
            out[i] = X.t() if case["m"] > case["n"] else X
        return out
    row_of, k, h = s["row_of"], case["k"], case["hidden"]
    token, j = torch.nonzero(row_of >= 0, as_tuple=True)
    row = row_of[token, j].long()
    if case["op"] == "permute":
        out = torch.zeros((s["rows"], h), dtype=torch.float64, device=DEV)
        out[row] = s["x"].double()[token]
        return out
    if case["op"] == "unpermute":
        out = torch.zeros((case["tokens"], h), dtype=torch.float64, device=DEV)
        for q in range(k):
            at = torch.nonzero(row_of[:, q] >= 0)[:, 0]
            w = 1.0 if s["weights"] is None else s["weights"][at, q].double()[:, None]
            out[at] += w * s["y"][row_of[at, q].long()].double()
        return out
    dy = torch.zeros((s["rows"], h), dtype=torch.float64, device=DEV)
    dw = torch.zeros((case["tokens"], k), dtype=torch.float64, device=DEV)
    for q in range(k):
        at = torch.nonzero(row_of[:, q] >= 0)[:, 0]
        to = row_of[at, q].long()
        d = s["x"][at].double()
        dy[to] = s["weights"][at, q].double()[:, None] * d
        dw[at, q] = torch.linalg.vecdot(d, s["y"][to].double())
    return dy, dw
