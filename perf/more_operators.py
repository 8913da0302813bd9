"""Operators of a mixture-of-experts training step around the expert products: the router with its
balance loss, the gated activation whose input is kept in 8 bits, and the weight gradient that reads 8-bit rows.

With T tokens, E experts, k experts a token, R rows sorted by expert, I values of the inner layer:

    route       scores (T, E)  -> ids (T, k) by descending score, weights (T, k), counts c (E,), loss, slope (E,)
                p = softmax(scores) or sigmoid(scores) / sum;  N tokens take part
                slope_e = E c_e / (k N^2),  loss = sum_te slope_e p_te    (1 when the experts are used alike)
                weights = p (sigmoid: sigmoid) at ids, made to sum to one if `renormalize`, times `scale`
    route_grad  scores, ids, dweights, dloss, slope -> dscores (T, E)
    act         h (R, 2I) or (R, I) -> y = silu(g) u or relu(h)^2, and h as e4m3 with a power of two for every 128
                values of a row; then dh from dy and the 8-bit h, and y once more from it where asked
    wgrad_rows  out_e = A_e^T B_e over the rows of expert e; A e4m3 with a power of two for every 128 values
                of a row, B the same or bf16

A score of -inf is an expert that its token may not take; a masked token takes none.  Both leave id -1
and weight 0.

`own = False` computes them from elementary torch operations in 32 bits; `own = True` calls the package.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}
BLOCK = 128
TINY = 1e-20


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def _route(op, name, tokens, k, experts, dtype="fp32", score="softmax", renormalize=True, masked=False):
    return dict(name=name, op=op, tokens=tokens, k=k, experts=experts, dtype=dtype, score=score,
                renormalize=renormalize, masked=masked)


def _act(name, rows, inner, dtype="bf16", act="swiglu", again=False, out8=False, part=False):
    """again: y once more in the backward pass; out8: y and dh as e4m3; part: rows past the last offset exist."""
    return dict(name=name, op="act", rows=rows, inner=inner, dtype=dtype, act=act, again=again, out8=out8, part=part)


def _wgrad(name, experts, hidden, n, tokens, other="bf16", out="fp32"):
    return dict(name=name, op="wgrad_rows", experts=experts, hidden=hidden, n=n, tokens=tokens, other=other, out=out)


def listed():
    return [
        # A step of decoding: 64 sequences, 8 of 256 experts each; one short call, latency counts.
        _route("route", "route decode 64x8 E256", 64, 8, 256),
        # A training step over 256 experts with sigmoid scores, as many tokens as the 32-expert layer sorts.
        _route("route", "route train 32768x8 E256 sigmoid", 32768, 8, 256, score="sigmoid"),
        # A ragged padded batch with bf16 scores (many ties) and forbidden experts, an odd number of both.
        _route("route", "route 5003x2 E61 bf16 masked", 5003, 2, 61, "bf16", masked=True),
        # The gradient for the 32-expert layer's training step, weights not made to sum to one.
        _route("route_grad", "route grad 32768x8 E32", 32768, 8, 32, renormalize=False),
        # The same over 256 experts, fp16 scores and a padded batch.
        _route("route_grad", "route grad 16411x6 E256 fp16 masked", 16411, 6, 256, "fp16", masked=True),
        # The activation of a training step of the 8-expert layer (N = 2048): y, the kept h, dh, and y again.
        _act("act 65536x2048 bf16", 65536, 2048, again=True),
        # A short buffer that is larger than what its experts fill, fp32, an inner size that is no multiple of 128.
        _act("act 1283x712 fp32 relu2 part", 1283, 712, "fp32", "relu2", part=True),
        # 8-bit operands for the products of both directions, at the 32-expert layer's inner size.
        _act("act 8192x4096 8-bit results", 8192, 4096, out8=True),
        # The smallest weight gradients the tests use (E=4, 256 x 512): latency.
        _wgrad("wgrad rows E4 256x512", 4, 256, 512, 1024),
        # Odd sizes.
        _wgrad("wgrad rows E5 1040x776", 5, 1040, 776, 5 * 1152, "e4m3", "fp16"),
        # The 8-expert layer's weight gradients from 8-bit rows and bf16 gradients.
        _wgrad("wgrad rows E8 4096x2048", 8, 4096, 2048, 32768, "bf16", "bf16"),
        # The 32-expert fp8 layer with both operands in 8 bits: the largest.
        _wgrad("wgrad rows E32 7168x4096 8-bit", 32, 7168, 4096, 264320, "e4m3", "bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "route_grad", "act", "act", "wgrad_rows", "wgrad_rows"))
    if op in ("route", "route_grad"):
        experts = _log_int(rng, 4, 512)
        k = rng.randint(1, min(8, experts - 1))
        most = min(32768, 32768 * 256 // experts)
        return dict(op=op, tokens=_log_int(rng, 24, most), k=k, experts=experts,
                    dtype=rng.choice(("fp32", "fp32", "bf16", "fp16")), score=rng.choice(("softmax", "softmax", "sigmoid")),
                    renormalize=rng.random() < 0.6, masked=rng.random() < 0.4)
    if op == "act":
        inner = (_log_int(rng, 64, 4096) + 7) // 8 * 8
        if rng.random() < 0.6:
            inner = (inner + 127) // 128 * 128
        dtype = rng.choice(("bf16", "bf16", "bf16", "fp16", "fp32"))
        rows = _log_int(rng, 24, min(65536, 65536 * 2048 * 2 // (inner * SIZE[dtype])))
        out8 = rng.random() < 0.25
        return dict(op=op, rows=rows, inner=inner, dtype=dtype, act=rng.choice(("swiglu", "swiglu", "relu2")),
                    again=rng.random() < 0.4, out8=out8, part=not out8 and rng.random() < 0.4)
    experts = _log_int(rng, 1, 32)
    hidden, n = _log_int(rng, 64, 7168) // 16 * 16, _log_int(rng, 64, 4096) // 16 * 16
    tokens = experts * _log_int(rng, 1, 64) * BLOCK
    return dict(op=op, experts=experts, hidden=hidden, n=n, tokens=tokens, other=rng.choice(("bf16", "e4m3")),
                out=rng.choice(("fp32", "bf16", "fp16")))


def _wide(case):
    """Values of a row of h."""
    return case["inner"] * (2 if case["act"] == "swiglu" else 1)


def work(case):
    if case["op"] == "wgrad_rows":
        t, h, n = case["tokens"], case["hidden"], case["n"]
        b = t * n * SIZE[case["other"]] + (t * n // BLOCK if case["other"] == "e4m3" else 0)
        return {"bytes": t * h + t * h // BLOCK + b + case["experts"] * h * n * SIZE[case["out"]], "flops": 2.0 * t * h * n}
    if case["op"] == "act":
        # forward: h in, its 8-bit form and y out; backward: the 8-bit form and dy in, dh (and y) out
        r, i, w = case["rows"] * (0.75 if case["part"] else 1.0), case["inner"], _wide(case)
        s = SIZE[case["dtype"]]
        o = 1 + 1 / BLOCK if case["out8"] else s
        kept = 1 + 1 / BLOCK
        return {"bytes": r * (w * s + w * kept + i * o + w * kept + i * s + w * o + (i * o if case["again"] else 0)),
                "flops": 30.0 * r * i}
    t, k, e, s = case["tokens"], case["k"], case["experts"], SIZE[case["dtype"]]
    if case["op"] == "route":
        return {"bytes": t * e * s + 8 * t * k + 8 * e, "flops": 4.0 * t * e}
    return {"bytes": 2 * t * e * s + 8 * t * k + 4 * e, "flops": 8.0 * t * e}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _rows8(x):
    """fp32 rows (r, c) -> e4m3 codes (r, c) and the biased exponents (ceil(c / 128), r) of their scales: the
    smallest power of two that brings the block's largest magnitude to 448 or below."""
    r, c = x.shape
    blocks = -(-c // BLOCK)
    padded = x if c == blocks * BLOCK else torch.nn.functional.pad(x, (0, blocks * BLOCK - c))
    padded = padded.reshape(r, blocks, BLOCK)
    m, e = torch.frexp(padded.abs().amax(2))
    byte = torch.where(m == 0, 127, (e - 9 + (m > 0.875).int() + 127).clamp(1, 254)).int()
    inverse = ((254 - byte) << 23).view(torch.float32)
    codes = (padded * inverse[..., None]).reshape(r, blocks * BLOCK)[:, :c].to(torch.float8_e4m3fn)
    return codes.view(torch.uint8).contiguous(), byte.t().to(torch.uint8).contiguous()


def _values(codes, scales, dtype=torch.float32):
    """What 8-bit rows stand for (exact in bf16 and fp32)."""
    scale = (scales.int() << 23).view(torch.float32).to(dtype).t()
    v = codes.view(torch.float8_e4m3fn).to(dtype)
    r, c = v.shape
    if c % BLOCK == 0:
        return (v.view(r, c // BLOCK, BLOCK) * scale[..., None]).view(r, c)
    return v * scale.repeat_interleave(BLOCK, 1)[:, :c]


def _halves8(x, case):
    """_rows8 of h: the two halves of a gated row have blocks of their own."""
    if case["act"] != "swiglu":
        return _rows8(x)
    (a, sa), (b, sb) = _rows8(x[:, :case["inner"]]), _rows8(x[:, case["inner"]:])
    return torch.cat((a, b), 1), torch.cat((sa, sb), 0)


def _halves_values(codes, scales, case, dtype=torch.float32):
    i = case["inner"]
    if case["act"] != "swiglu" or i % BLOCK == 0:
        return _values(codes, scales, dtype)
    half = scales.shape[0] // 2
    return torch.cat((_values(codes[:, :i], scales[:half], dtype), _values(codes[:, i:], scales[half:], dtype)), 1)


def _randn8(rows, cols, g, spread):
    """Normal rows of different sizes in 8 bits, made a part at a time."""
    codes = torch.empty((rows, cols), dtype=torch.uint8, device=DEV)
    scales = torch.empty((-(-cols // BLOCK), rows), dtype=torch.uint8, device=DEV)
    for at in range(0, rows, 1 << 15):
        part = slice(at, min(rows, at + (1 << 15)))
        x = torch.randn((part.stop - at, cols), generator=g, device=DEV)
        x *= torch.exp(spread * torch.randn((part.stop - at, 1), generator=g, device=DEV))
        codes[part], scales[:, part] = _rows8(x)
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = {"case": case}
    rand = lambda *shape: torch.rand(shape, generator=g, device=DEV)       # noqa: E731
    randn = lambda *shape: torch.randn(shape, generator=g, device=DEV)     # noqa: E731
    if case["op"] == "wgrad_rows":
        t, e = case["tokens"], case["experts"]
        # every expert's share of the 128-row blocks, 0.7 to 1.3 times the mean
        ends = torch.cumsum(0.7 + 0.6 * rand(e).double(), 0)
        ends = (ends / ends[-1] * (t // BLOCK)).round().int() * BLOCK
        s["offsets"] = ends.int().contiguous()
        s["most"] = int(torch.diff(ends, prepend=ends.new_zeros(1)).max())
        s["A"], s["sa"] = _randn8(t, case["hidden"], g, 0.5)
        if case["other"] == "e4m3":
            s["B"], s["sb"] = _randn8(t, case["n"], g, 1.0)
        else:
            s["B"], s["sb"] = torch.empty((t, case["n"]), dtype=torch.bfloat16, device=DEV), None
            for part in s["B"].split(1 << 15):
                part.copy_(randn(*part.shape))
        return s
    if case["op"] == "act":
        dt, r = DTYPES[case["dtype"]], case["rows"]
        s["h"] = torch.empty((r, _wide(case)), dtype=dt, device=DEV)
        s["dy"] = torch.empty((r, case["inner"]), dtype=dt, device=DEV)
        for x in (s["h"], s["dy"]):
            for part in x.split(1 << 14):
                part.copy_(randn(*part.shape) * torch.exp(0.5 * randn(part.shape[0], 1)))
        s["offsets"] = s["out"] = s["dh"] = s["y"] = None
        if case["part"]:
            # four experts fill a part of the buffer; the rows behind them hold anything and are left alone
            s["offsets"] = (torch.cumsum(rand(4) * 0.5 * r / 4 + 0.5 * r / 4, 0)).int().clamp(max=r)
            last = int(s["offsets"][-1])
            s["h"][last:] = float("nan")
            s["out"], s["dh"] = torch.zeros_like(s["dy"]), torch.zeros_like(s["h"])
            s["y"] = torch.zeros_like(s["dy"]) if case["again"] else None
        return s
    t, e, k = case["tokens"], case["experts"], case["k"]
    scores = randn(t, e) + torch.log(0.7 + 0.6 * rand(e))                  # some experts are more popular
    s["mask"] = None
    if case["masked"]:
        scores[rand(t, e) < 0.125] = -math.inf
        scores[rand(t) < 0.02] = -math.inf                                 # tokens that may take no expert
        s["mask"] = rand(t) < 0.9                                          # False: padding, with any scores
        scores[~s["mask"]] = float("nan")
    s["scores"] = scores.to(DTYPES[case["dtype"]])
    s["scale"] = 2.5 if case["score"] == "sigmoid" else 1.0
    if case["op"] == "route_grad":
        s["ids"], _, _, _, s["slope"] = _route_plain(s)
        s["dweights"] = randn(t, k)                                        # gradients scaled by the number of tokens
        s["dloss"] = torch.full((), 0.01 * t, device=DEV)
    return s


# ----------------------------------------------------------------------------
# the plain forms
# ----------------------------------------------------------------------------
def _scores(s):
    x = s["scores"].float()
    if s["mask"] is not None:
        x = torch.where(s["mask"][:, None], x, -math.inf)
    return x, x > -math.inf


def _shares(x, allowed, case):
    """p, and for sigmoid scores the unnormalised ones."""
    if case["score"] == "softmax":
        top = x.amax(1, keepdim=True)
        u = torch.where(allowed, torch.exp(x - torch.where(top > -math.inf, top, 0.0)), 0.0)
        p = u / torch.where(allowed.any(1, keepdim=True), u.sum(1, keepdim=True), 1.0)
        return p, p
    u = torch.where(allowed, 1 / (1 + torch.exp(-x)), 0.0)
    return u / (u.sum(1, keepdim=True) + TINY), u


def _route_plain(s):
    case = s["case"]
    x, allowed = _scores(s)
    k, e = case["k"], case["experts"]
    ordered, ids = torch.sort(x, dim=1, descending=True, stable=True)      # ties go to the lowest index
    here = ordered[:, :k] > -math.inf
    ids = torch.where(here, ids[:, :k], -1)
    p, u = _shares(x, allowed, case)
    w = torch.where(here, u.gather(1, ids.clamp(min=0)), 0.0)
    if case["renormalize"]:
        total = w.sum(1, keepdim=True)
        w = w / (total + TINY if case["score"] == "sigmoid" else torch.where(total > 0, total, 1.0))
    counts = torch.zeros(e + 1, dtype=torch.int64, device=x.device)
    counts.scatter_add_(0, torch.where(here, ids, e).reshape(-1), torch.ones_like(ids.reshape(-1)))
    counts = counts[:e]
    part = allowed.any(1).sum().float()
    slope = torch.where(part > 0, counts * (e / k) / torch.where(part > 0, part * part, 1.0), 0.0)
    loss = (p.sum(0) * slope).sum()
    return ids.int(), w * s["scale"], counts.int(), loss, slope


def _route_grad_plain(s):
    case = s["case"]
    x, allowed = _scores(s)
    p, u = _shares(x, allowed, case)
    here = s["ids"] >= 0
    ids = s["ids"].clamp(min=0).long()
    dw = torch.where(here, s["dweights"], 0.0) * s["scale"]
    chosen = torch.where(here, u.gather(1, ids), 0.0)
    push = s["dloss"] * s["slope"]
    push = push - (p * push).sum(1, keepdim=True)                          # d loss / d scores is p times this (softmax)
    if case["renormalize"]:
        total = chosen.sum(1, keepdim=True)
        total = total + TINY if case["score"] == "sigmoid" else torch.where(total > 0, total, 1.0)
        dw = (dw - (dw * chosen).sum(1, keepdim=True) / total) / total
    dw = torch.zeros_like(x).scatter_add_(1, ids, torch.where(here, dw, 0.0))
    if case["score"] == "softmax":
        d = p * push + p * (dw - (p * dw).sum(1, keepdim=True))
    else:
        d = (push / (u.sum(1, keepdim=True) + TINY) + dw) * u * torch.where(allowed, 1 / (1 + torch.exp(x)), 0.0)
    return torch.where(allowed, d, 0.0).to(s["scores"].dtype)


def _act_plain(h, case):
    if case["act"] == "relu2":
        return torch.relu(h).square()
    gate, up = h[:, :case["inner"]], h[:, case["inner"]:]
    return gate / (1 + torch.exp(-gate)) * up


def _act_grad_plain(h, dy, case):
    if case["act"] == "relu2":
        return 2 * torch.relu(h) * dy
    gate, up = h[:, :case["inner"]], h[:, case["inner"]:]
    share = 1 / (1 + torch.exp(-gate))
    return torch.cat((dy * up * share * (1 + gate * (1 - share)), dy * gate * share), 1)


def _act_step_plain(s):
    case, h, dy = s["case"], s["h"].float(), s["dy"].float()
    dt = s["h"].dtype
    here = None
    if case["part"]:
        here = (torch.arange(case["rows"], device=h.device) < s["offsets"][-1])[:, None]
        h = torch.where(here, h, 0.0)
    kept = _halves_values(*_halves8(h, case), case)
    outs = [_act_plain(h, case), _act_grad_plain(kept, dy, case)]
    if case["again"]:
        outs.append(_act_plain(kept, case))
    if case["out8"]:
        parts = [_rows8, lambda x: _halves8(x, case), _rows8]
        back = [_values, lambda q, c, t: _halves_values(q, c, case, t), _values]
        return tuple(b(*q(x), torch.bfloat16) for x, q, b in zip(outs, parts, back))
    if here is not None:
        outs = [torch.where(here, x, 0.0) for x in outs]
    return tuple(x.to(dt) for x in outs)


def _wgrad_plain(s):
    case = s["case"]
    a = _values(s["A"], s["sa"])
    b = s["B"].float() if s["sb"] is None else _values(s["B"], s["sb"])
    ends = s["offsets"].long()
    begin = torch.cat((ends.new_zeros(1), ends[:-1]))
    at = begin[:, None] + torch.arange(max(s["most"], 1), device=a.device)     # (experts, longest): every expert's rows
    here = at < ends[:, None]
    at = torch.where(here, at, 0)
    b = b[at] * here[..., None]
    a = a[at].transpose(1, 2).contiguous()
    return torch.bmm(a, b).to(DTYPES[case["out"]])


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import grouped_gemm_expert_offsets_amd as kgw
        if op == "route":
            return kgw.kgw_moe_route(s["scores"], case["k"], mask=s["mask"], score=case["score"],
                                     renormalize=case["renormalize"], scale=s["scale"])
        if op == "route_grad":
            return kgw.kgw_moe_route_grad(s["scores"], s["ids"], s["dweights"], dloss=s["dloss"], slope=s["slope"],
                                          mask=s["mask"], score=case["score"], renormalize=case["renormalize"],
                                          scale=s["scale"])
        if op == "act":
            y, sy, kept, sk = kgw.kgw_moe_act_fp8(s["h"], act=case["act"], offsets=s["offsets"], fp8=case["out8"],
                                                  out=s["out"])
            dh, sdh, y2, sy2 = kgw.kgw_moe_act_fp8_grad(s["dy"], kept, sk, act=case["act"], offsets=s["offsets"],
                                                        fp8=case["out8"], again=case["again"], dh=s["dh"], y=s["y"])
            if case["out8"]:
                y, dh = _values(y, sy, torch.bfloat16), _halves_values(dh, sdh, case, torch.bfloat16)
                y2 = _values(y2, sy2, torch.bfloat16) if case["again"] else None
            return (y, dh, y2) if case["again"] else (y, dh)
        return kgw.kgw_wgrad_fp8_rows(s["A"], s["sa"], s["B"], s["offsets"], sb=s["sb"], out_dtype=DTYPES[case["out"]])
    if op == "route":
        return _route_plain(s)
    if op == "route_grad":
        return _route_grad_plain(s)
    if op == "act":
        return _act_step_plain(s)
    return _wgrad_plain(s)


# ----------------------------------------------------------------------------
# the definition in 64 bits
# ----------------------------------------------------------------------------
def _e4m3_rows(x):
    """fp64 rows -> what their 8-bit form stands for, by the definition: a block's power of two, then the nearest
    of the values with four significant bits (and no step below 2^-9), ties to the even one."""
    r, c = x.shape
    out = torch.empty_like(x)
    for at in range(0, c, BLOCK):
        part = x[:, at:at + BLOCK]
        top = part.abs().amax(1, keepdim=True)
        k = torch.ceil(torch.log2(top / 448)).clamp(-126, 127)
        k = torch.where(448 * torch.exp2(k - 1) >= top, k - 1, torch.where(448 * torch.exp2(k) < top, k + 1, k))
        scale = torch.exp2(torch.where(top == 0, 0.0, k.clamp(-126, 127)))
        v = part / scale
        step = torch.exp2(torch.frexp(v)[1].clamp(min=-5).double() - 4)
        out[:, at:at + BLOCK] = torch.round(v / step) * step * scale
    return out


def _exact_act(h, case):
    if case["act"] == "relu2":
        return h.clamp(min=0) ** 2
    return h[:, :case["inner"]] * torch.sigmoid(h[:, :case["inner"]]) * h[:, case["inner"]:]


def _exact_step(s):
    case, i = s["case"], s["case"]["inner"]
    last = int(s["offsets"][-1]) if case["part"] else case["rows"]
    parts = []
    for at in range(0, case["rows"], 1 << 14):                            # a part of the rows at a time
        stop = min(case["rows"], at + (1 << 14))
        live = min(max(last, at), stop)
        h, dy = s["h"][at:live].double(), s["dy"][at:live].double()
        halves = (h[:, :i], h[:, i:]) if case["act"] == "swiglu" else (h,)
        kept = torch.cat([_e4m3_rows(x) for x in halves], 1).requires_grad_()
        y = _exact_act(h, case)
        again = _exact_act(kept, case)
        (again * dy).sum().backward()
        outs = [y, kept.grad, again.detach()]
        if case["out8"]:
            outs[0], outs[2] = _e4m3_rows(outs[0]), _e4m3_rows(outs[2])
            d = outs[1]
            outs[1] = torch.cat([_e4m3_rows(x) for x in ((d[:, :i], d[:, i:]) if case["act"] == "swiglu" else (d,))], 1)
        parts.append([torch.nn.functional.pad(x, (0, 0, 0, stop - live)) for x in outs[:3 if case["again"] else 2]])
    return tuple(torch.cat(x) for x in zip(*parts))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "act":
        return _exact_step(s)
    if case["op"] == "wgrad_rows":
        out = torch.zeros((case["experts"], case["hidden"], case["n"]), dtype=torch.float64, device=DEV)
        start = 0
        for e, end in enumerate(s["offsets"].tolist()):
            for at in range(start, end, 1 << 13):
                rows = slice(at, min(end, at + (1 << 13)))
                pair = []
                for q, c in ((s["A"], s["sa"]), (s["B"], s["sb"])):
                    v = (q[rows] if c is None else q[rows].view(torch.float8_e4m3fn)).double()
                    if c is not None:
                        for b in range(c.shape[0]):
                            v[:, BLOCK * b:BLOCK * (b + 1)] *= torch.exp2(c[b, rows].double() - 127)[:, None]
                    pair.append(v)
                out[e] += pair[0].t().contiguous() @ pair[1]
            start = end
        return out
    # the router: shares and weights by logarithms, gradients by differentiating the definition
    x = s["scores"].double()
    if s["mask"] is not None:
        x[~s["mask"]] = -math.inf
    allowed = x > -math.inf
    x = torch.where(allowed, x, -1e6).requires_grad_()
    rows = allowed.any(1)
    if case["score"] == "softmax":
        u = torch.where(allowed, torch.log_softmax(x, 1).exp(), 0.0)
        p = u
    else:
        u = torch.where(allowed, torch.sigmoid(x), 0.0)
        p = u / (u.sum(1, keepdim=True) + TINY)
    p = p * rows[:, None]
    if case["op"] == "route":
        top = torch.sort(torch.where(allowed, x, -math.inf).detach(), dim=1, descending=True, stable=True)
        ids = torch.where(top.values[:, :case["k"]] > -math.inf, top.indices[:, :case["k"]], -1)
    else:
        ids = s["ids"].long()
    w = torch.where(ids >= 0, u.gather(1, ids.clamp(min=0)), 0.0)
    if case["renormalize"]:
        total = w.sum(1, keepdim=True)
        w = w / (total + TINY if case["score"] == "sigmoid" else torch.where(total > 0, total, 1.0))
    w = w * s["scale"]
    if case["op"] == "route":
        counts = torch.bincount(ids[ids >= 0], minlength=case["experts"]).double()
        n = float(rows.sum())
        slope = counts * case["experts"] / (case["k"] * n * n) if n else counts * 0
        return None, w.detach(), None, (p.detach().sum(0) * slope).sum(), slope
    weighed = torch.where(ids >= 0, s["dweights"].double(), 0.0) * w
    (weighed.sum() + s["dloss"].double() * (p * s["slope"].double()).sum()).backward()
    return torch.where(allowed, x.grad, 0.0)
