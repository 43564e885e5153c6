"""Cases that measure the experts' products in FP8 and bf16 with their gradients, and the
SwiGLU between them whose gates and ups are kept in 8 bits for the backward pass.

`run` takes a state from `prepare` and makes one pass: in plain torch operations, or,
where `own` is true, by the calls a user makes of the library.  `exact` gives the
operator's definition in 64 bits.

Definitions (rows are token rows; those of expert e are [expert_base[e], expert_base[e + 1]);
rows behind the last segment are left as they were, zeros here; sums are real numbers):

  fp8     c[r, n] = sum_b a_scales[r, b] * w_scales[e, n / 128, b] * sum_k a[r, k] * w[e, n, k] over the
          k of block b of 128 columns, codes e4m3; with `swiglu` the first half of n are gates g and the
          second half u, whose blocks of 128 rows are counted apart, and the result is g / (1 + exp(-g)) * u.
  bf16    c[r, n] = sum_k a[r, k] * w[e, n, k], plain or with `swiglu`.
  grads   of c: da[r, k] = sum_n dc[r, n] * w[e, n, k] and dw[e, n, k] = sum_r dc[r, n] * a[r, k].
  keep    inner = weight[r] * g / (1 + exp(-g)) * u of bf16 rows [g, u], and the e4m3 codes of [g, u] nearest
          to value / scale (ties to even) with scale = max / 448 of 128 columns.
  back    of inner, from codes times scales g, u: dg = weight * dy * u * s * (1 + g * (1 - s)) and
          du = weight * dy * g * s with s = 1 / (1 + exp(-g)), inner = weight * g * s * u, and the
          weight's gradient sum(dy * g * s * u).
"""
import math

import torch

own = False


def listed():
    return [
        # decode: one projection of eight tokens (no experts)
        {"name": "fp8_8_rows", "op": "fp8", "tokens": 8, "topk": 1, "experts": 1, "skew": 0.0, "align": 1,
         "k": 4096, "n": 4096, "swiglu": False},
        # a small step whose experts get unequal, odd numbers of rows
        {"name": "fp8_ragged", "op": "fp8", "tokens": 1332, "topk": 2, "experts": 16, "skew": 1.2, "align": 1,
         "k": 1024, "n": 1400, "swiglu": True},
        # a decode batch: many experts with a handful of rows each, where reading the weights is the work
        {"name": "fp8_thin", "op": "fp8", "tokens": 256, "topk": 16, "experts": 512, "skew": 0.0, "align": 1,
         "k": 4096, "n": 1024, "swiglu": False},
        # prefill: gate and up products of 8 ranks x 2048 tokens, aligned segments
        {"name": "fp8_gate_up", "op": "fp8", "tokens": 16384, "topk": 8, "experts": 128, "skew": 0.0, "align": 128,
         "k": 4096, "n": 2048, "swiglu": True},
        # a decode batch of more tokens than the few-token layer takes
        {"name": "bf16_thin", "op": "bf16", "tokens": 96, "topk": 8, "experts": 128, "skew": 0.0, "align": 1,
         "k": 4096, "n": 2048, "swiglu": True},
        # training: gate and up products of 8 ranks x 2048 tokens
        {"name": "bf16_gate_up", "op": "bf16", "tokens": 16384, "topk": 8, "experts": 128, "skew": 0.0, "align": 128,
         "k": 4096, "n": 2048, "swiglu": False},
        # the backward pass of a small, uneven step; gradients of the weights for an optimiser of 32 bits
        {"name": "grads_ragged", "op": "grads", "tokens": 1332, "topk": 2, "experts": 16, "skew": 1.2, "align": 1,
         "k": 1024, "n": 1400, "wide": True},
        # the backward pass of the gate and up products
        {"name": "grads_gate_up", "op": "grads", "tokens": 16384, "topk": 8, "experts": 128, "skew": 0.0, "align": 128,
         "k": 4096, "n": 2048, "wide": False},
        # one token's rows, where the call is the work
        {"name": "keep_8_rows", "op": "keep", "rows": 8, "unused": 0, "inner": 1024, "weights": False},
        # a training step's rows on eight ranks, in a buffer for the largest routing
        {"name": "keep_rows", "op": "keep", "rows": 131072, "unused": 16256, "inner": 1024, "weights": True},
        # a ragged microbatch, no weights in the rows
        {"name": "back_ragged", "op": "back", "rows": 2664, "unused": 37, "inner": 768, "weights": False},
        # the backward pass of keep_rows
        {"name": "back_rows", "op": "back", "rows": 131072, "unused": 16256, "inner": 1024, "weights": True},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["fp8", "bf16", "grads", "keep", "back"])
    if op in ("keep", "back"):
        inner = 128 * _log(rng, 1, 32)
        rows = _log(rng, 1, 131072 * 1024 // inner)
        return {"op": op, "rows": rows, "unused": rng.choice([0, 0, rng.randint(1, 300)]), "inner": inner,
                "weights": rng.random() < 0.5}
    case = {"op": op}
    k = 128 * _log(rng, 1, 56) if op == "fp8" else 8 * _log(rng, 8, 896)
    swiglu = op != "grads" and rng.random() < 0.5
    n = 8 * _log(rng, 4, 256) if op == "grads" else _log(rng, 16, 2048) * (2 if swiglu else 1)
    if rng.random() < 0.25:  # one matrix
        case.update(tokens=_log(rng, 1, 16384), topk=1, experts=1, skew=0.0, align=1)
    else:
        skew = rng.choice([0.0, 0.0, 1.2])
        experts = 2 ** rng.randint(2, 5 if skew else 9)
        while experts * k * n > 2 ** 30:
            experts //= 2
        experts = max(experts, 2)
        case.update(tokens=_log(rng, 1, 2048 if skew else 16384), topk=rng.choice([1, 2, 4, 8]) if experts >= 8 else 2,
                    experts=experts, skew=skew, align=rng.choice([1, 64, 128]))
        while case["tokens"] * case["topk"] * k * n > 2 ** 40:
            case["tokens"] //= 2
    case.update(k=k, n=n)
    if op == "grads":
        case["wide"] = rng.random() < 0.5
    else:
        case["swiglu"] = swiglu
    return case


# ---------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, scale=1.0, dtype=torch.bfloat16):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        part = flat[i:i + (1 << 28)]
        if dtype is torch.bfloat16:
            part.normal_(0.0, scale, generator=g)
        else:  # codes that use the type's range, as a quantiser of blocks leaves them
            v = torch.empty(part.numel(), dtype=torch.bfloat16, device="cuda").normal_(0.0, scale, generator=g)
            part.copy_(v.clamp_(-448, 448))
    return out


def _routing(g, tokens, experts, topk, skew):
    """[tokens, topk] distinct experts: uniform, or with probabilities (e + 1)^-skew."""
    u = torch.rand(tokens, experts, device="cuda", generator=g).clamp_(1e-12, 1 - 1e-7)
    keys = -torch.log(-torch.log(u)) - skew * torch.log(torch.arange(1, experts + 1, device="cuda", dtype=torch.float32))
    return keys.topk(topk, dim=1).indices


def _blocks(n, swiglu):
    """Blocks of 128 rows of a matrix, or of its gates and its ups."""
    return 2 * ((n // 2 + 127) // 128) if swiglu else (n + 127) // 128


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    if case["op"] in ("keep", "back"):
        inner, rows = case["inner"], case["rows"] + case["unused"]
        c = _normal(g, rows, 2 * inner, scale=1.5)
        c[torch.rand(rows, device="cuda", generator=g) < 0.01] *= 20  # outlier tokens
        c[torch.rand(rows, device="cuda", generator=g) < 0.05] = 0     # padding between segments
        s["row_weights"] = torch.rand(rows, device="cuda", generator=g) if case["weights"] else None
        s["used"] = torch.tensor([case["rows"]], dtype=torch.int32, device="cuda")
        if case["op"] == "keep":
            s["c"] = c
            s["codes"] = torch.zeros(rows, 2 * inner, dtype=torch.float8_e4m3fn, device="cuda")
            s["scales"] = torch.zeros(rows, inner // 64, dtype=torch.float32, device="cuda")
        else:
            blocks = c.view(-1, 128)
            top = blocks.abs().amax(1, keepdim=True).float()
            s["scales"] = (top / 448).view(rows, inner // 64)
            s["codes"] = torch.cat([(part.float() * (448 / t.clamp_min(1e-30))).clamp_(-448, 448).to(torch.float8_e4m3fn)
                                    for part, t in zip(blocks.split(1 << 20), top.split(1 << 20))]).view(rows, 2 * inner)
            s["dy"] = _normal(g, rows, inner)
            s["dc"] = torch.zeros(rows, 2 * inner, dtype=torch.bfloat16, device="cuda")
            s["dweights"] = torch.zeros(rows, dtype=torch.float32, device="cuda")
        s["inner_rows"] = torch.zeros(rows, inner, dtype=torch.bfloat16, device="cuda")
        return s
    experts, k, n = case["experts"], case["k"], case["n"]
    counts = torch.bincount(_routing(g, case["tokens"], experts, case["topk"], case["skew"]).flatten(), minlength=experts)
    aligned = (counts + case["align"] - 1) // case["align"] * case["align"]
    base = torch.cat([aligned.new_zeros(1), aligned.cumsum(0)])
    used = int(base[-1])
    # buffers of the largest size that the routing can need, as a program that does not wait for the counts has them
    rows = case["tokens"] * case["topk"] + experts * (case["align"] - 1)
    s["longest"], s["unused"] = int(aligned.max()), rows - used
    s["expert_base"] = base.to(torch.int32) if experts > 1 else None
    owner = torch.repeat_interleave(torch.arange(experts, device="cuda"), aligned)
    padding = torch.arange(used, device="cuda") - base[owner] >= counts[owner]  # rows that no token fills
    if case["op"] == "fp8":
        s["a"] = _normal(g, rows, k, scale=130.0, dtype=torch.float8_e4m3fn)
        s["w"] = _normal(g, experts, n, k, scale=130.0, dtype=torch.float8_e4m3fn)
        s["a_scales"] = torch.rand(rows, k // 128, device="cuda", generator=g) * 0.005 + 0.005
        s["w_scales"] = (torch.rand(experts, _blocks(n, case["swiglu"]), k // 128, device="cuda", generator=g) * 0.005 + 0.005) / math.sqrt(k)
        s["a"][:used].view(torch.uint8)[padding] = 0
        s["a_scales"][:used][padding] = 0
    else:
        s["a"] = _normal(g, rows, k)
        s["a"][:used][padding] = 0
        s["w"] = _normal(g, experts, n, k, scale=1 / math.sqrt(k))
    if case["op"] == "grads":
        s["dc"] = _normal(g, rows, n)
        s["dc"][:used][padding] = 0
        s["da"] = torch.zeros(rows, k, dtype=torch.bfloat16, device="cuda")
        s["dw"] = torch.zeros(experts, n, k, dtype=torch.float32 if case["wide"] else torch.bfloat16, device="cuda")
    else:
        s["out"] = torch.zeros(rows, n // 2 if case["swiglu"] else n, dtype=torch.bfloat16, device="cuda")
    return s


# ---------------------------------------------------------------- plain forms

def _segments(s):
    """Rows of each expert, padded to the longest segment, and which of them there are."""
    base = s["expert_base"].long()
    at = base[:-1, None] + torch.arange(s["longest"], device=base.device)
    inside = at < base[1:, None]
    return at.clamp_max(max(s["a"].shape[0] - 1, 0)), inside


def _to_rows(s, c, inside):
    """Rows in order (the segments lie one after another), and the zeros behind them."""
    c = c[inside] if inside is not None else c
    return torch.cat([c, c.new_zeros(s["unused"], c.shape[1])])


def _plain_product(s):
    a, w = s["a"].float(), s["w"].float()
    if s["op"] == "fp8":
        experts, n, k = w.shape
        parts = 2 if s["swiglu"] else 1
        of_row = s["w_scales"].view(experts, parts, -1, k // 128).repeat_interleave(128, 2)[:, :, :n // parts]
        w = (w.view(experts, n, k // 128, 128) * of_row.reshape(experts, n, k // 128, 1)).view(experts, n, k)
        a = (a.view(-1, k // 128, 128) * s["a_scales"][:, :, None]).view(-1, k)
    if s["expert_base"] is None:
        c, inside = a @ w[0].t(), None
    else:
        at, inside = _segments(s)
        c = torch.bmm(a[at], w.transpose(1, 2))
    if s["swiglu"]:
        g, u = c.chunk(2, dim=-1)
        c = g / (1 + torch.exp(-g)) * u
    return _to_rows(s, c.to(torch.bfloat16), inside)


def _plain_grads(s):
    a, w, dc = s["a"].float(), s["w"].float(), s["dc"].float()
    if s["expert_base"] is None:
        da, inside, dw = dc @ w[0], None, (dc.t() @ a)[None]
    else:
        at, inside = _segments(s)
        d = dc[at] * inside[:, :, None]
        da = torch.bmm(d, w)
        dw = torch.bmm(d.transpose(1, 2), a[at])
    return _to_rows(s, da.to(torch.bfloat16), inside), dw.to(s["dw"].dtype)


def _behind(s, v):
    """The rows that are used, and the zeros behind them."""
    return torch.cat([v, v.new_zeros((s["unused"],) + v.shape[1:])]) if s["unused"] else v


def _plain_keep(s):
    c = s["c"][:s["rows"]]
    g, u = c.float().chunk(2, dim=1)
    y = g / (1 + torch.exp(-g)) * u
    if s["row_weights"] is not None:
        y = y * s["row_weights"][:s["rows"], None]
    blocks = c.double().view(-1, 128)  # codes next to a border between two of them are settled in 64 bits
    top = blocks.abs().amax(1, keepdim=True)
    codes = torch.where(top > 0, blocks * 448 / top, 0.0).float().to(torch.float8_e4m3fn).view(c.shape)
    scales = (top / 448).float().view(c.shape[0], -1)
    return (_behind(s, y.to(torch.bfloat16)), torch.cat([codes.view(torch.uint8), codes.view(torch.uint8).new_zeros(
        s["unused"], c.shape[1])]).view(torch.float8_e4m3fn), _behind(s, scales))


def _plain_back(s):
    rows = s["rows"]
    c = (s["codes"][:rows].float().view(rows, -1, 128) * s["scales"][:rows, :, None]).view(rows, -1)
    g, u = c.chunk(2, dim=1)
    dy = s["dy"][:rows].float()
    sig = 1 / (1 + torch.exp(-g))
    y = g * sig * u
    dweights = (dy * y).sum(1)
    if s["row_weights"] is not None:
        weights = s["row_weights"][:rows, None]
        dy, y = dy * weights, y * weights
    dc = torch.cat([dy * u * sig * (1 + g * (1 - sig)), dy * g * sig], 1)
    return _behind(s, dc.to(torch.bfloat16)), _behind(s, y.to(torch.bfloat16)), _behind(s, dweights)


def run(s):
    if not own:
        return {"fp8": _plain_product, "bf16": _plain_product, "grads": _plain_grads, "keep": _plain_keep, "back": _plain_back}[s["op"]](s)
    from combine_ep_layout_03_gb300 import ep
    if s["op"] == "fp8":
        ep.ep_expert_matmul_fp8(s["a"], s["a_scales"], s["w"], s["w_scales"], s["expert_base"], s["out"], swiglu=s["swiglu"])
        return s["out"]
    if s["op"] == "bf16":
        ep.ep_expert_matmul_bf16(s["a"], s["w"], s["expert_base"], s["out"], swiglu=s["swiglu"])
        return s["out"]
    if s["op"] == "grads":
        ep.ep_expert_matmul_grad_rows(s["dc"], s["w"], s["expert_base"], s["da"])
        ep.ep_expert_matmul_grad_weights(s["dc"], s["a"], s["expert_base"], s["dw"])
        return s["da"], s["dw"]
    if s["op"] == "keep":
        ep.ep_swiglu_keep(s["c"], s["inner_rows"], s["codes"], s["scales"], row_weights=s["row_weights"], rows_used=s["used"])
        return s["inner_rows"], s["codes"], s["scales"]
    ep.ep_swiglu_keep_grad(s["codes"], s["scales"], s["dy"], s["dc"], inner=s["inner_rows"], row_weights=s["row_weights"],
                           row_weights_grad=s["dweights"], rows_used=s["used"])
    return s["dc"], s["inner_rows"], s["dweights"]


# ---------------------------------------------------------------- work

def work(case):
    if case["op"] in ("keep", "back"):
        rows, inner = case["rows"], case["inner"]
        each = (8 if case["op"] == "keep" else 10) * inner + inner / 16 + (4 if case["weights"] else 0)
        return {"bytes": rows * each, "flops": rows * inner * (12 if case["op"] == "keep" else 20)}
    rows, k, n, experts = case["tokens"] * case["topk"], case["k"], case["n"], case["experts"]
    active = experts * (1 - (1 - 1 / experts) ** rows) if case["skew"] == 0 else min(experts, rows)
    if case["op"] == "grads":
        return {"bytes": rows * (2 * n + 4 * k) + active * n * k * 2 + experts * n * k * (4 if case["wide"] else 2),
                "flops": 4 * rows * k * n}
    out = n // 2 if case["swiglu"] else n
    each, weight = (k + k / 32, 1 + 4 / 16384) if case["op"] == "fp8" else (2 * k, 2)
    return {"bytes": rows * (each + 2 * out) + active * n * k * weight, "flops": 2 * rows * k * n}


# ---------------------------------------------------------------- the definitions in 64 bits

def _silu(z):
    return torch.sigmoid(z) * z


def _exact_matrix(s, case, e):
    """Expert e's matrix."""
    w = s["w"][e].double()
    if case["op"] != "fp8":
        return w
    halves = 2 if case["swiglu"] else 1
    size, blocks = case["n"] // halves, s["w_scales"].shape[1] // halves
    for half in range(halves):
        for b in range(blocks):
            rows = slice(half * size + 128 * b, half * size + min(128 * (b + 1), size))
            w[rows] *= torch.repeat_interleave(s["w_scales"][e, half * blocks + b].double(), 128)
    return w


def _exact_products(s, case):
    rows, k, n = s["a"].shape[0], case["k"], case["n"]
    base = [0, case["tokens"]] if s["expert_base"] is None else s["expert_base"].tolist()
    if case["op"] == "grads":
        da = torch.zeros(rows, k, dtype=torch.float64, device="cuda")
        dw = torch.zeros(case["experts"], n, k, dtype=torch.float64, device="cuda")
    else:
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    for e, (first, end) in enumerate(zip(base, base[1:])):
        if first == end:
            continue
        a = s["a"][first:end].double()
        if case["op"] == "grads":
            d = s["dc"][first:end].double()
            torch.mm(d, s["w"][e].double(), out=da[first:end])
            torch.mm(d.t(), a, out=dw[e])
            continue
        if case["op"] == "fp8":
            a = a * torch.repeat_interleave(s["a_scales"][first:end].double(), 128, dim=1)
        c = torch.mm(a, _exact_matrix(s, case, e).t())
        out[first:end] = _silu(c[:, :n // 2]) * c[:, n // 2:] if case["swiglu"] else c
    return (da, dw) if case["op"] == "grads" else out


def _nearest_e4m3(v):
    """The e4m3 value nearest to each |v| <= 464 (ties to even), as a double."""
    _, e = torch.frexp(v)  # v = f * 2^e, 1/2 <= |f| < 1
    step = torch.exp2((e - 1).clamp_min(-6).double() - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _exact_keep(s, case):
    total, inner = case["rows"] + case["unused"], case["inner"]
    y = torch.zeros(total, inner, dtype=torch.float64, device="cuda")
    codes = torch.zeros(total, 2 * inner, dtype=torch.float64, device="cuda")
    scales = torch.zeros(total, inner // 64, dtype=torch.float64, device="cuda")
    for i in range(0, case["rows"], 8192):
        part = slice(i, min(i + 8192, case["rows"]))
        c = s["c"][part].double()
        y[part] = _silu(c[:, :inner]) * c[:, inner:]
        if case["weights"]:
            y[part] *= s["row_weights"][part].double()[:, None]
        blocks = c.reshape(-1, 128)
        top = blocks.abs().max(1, keepdim=True).values
        scales[part] = (top / 448).view(-1, inner // 64)
        codes[part] = _nearest_e4m3(blocks * 448 / torch.where(top > 0, top, 1.0)).view(-1, 2 * inner)
    return y, codes, scales


def _exact_back(s, case):
    total, inner = case["rows"] + case["unused"], case["inner"]
    dc = torch.zeros(total, 2 * inner, dtype=torch.float64, device="cuda")
    y = torch.zeros(total, inner, dtype=torch.float64, device="cuda")
    dweights = torch.zeros(total, dtype=torch.float64, device="cuda")
    for i in range(0, case["rows"], 8192):
        part = slice(i, min(i + 8192, case["rows"]))
        c = s["codes"][part].double() * torch.repeat_interleave(s["scales"][part].double(), 128, dim=1)
        gate, up, dy = c[:, :inner], c[:, inner:], s["dy"][part].double()
        silu, weight = _silu(gate), s["row_weights"][part].double()[:, None] if case["weights"] else 1.0
        slope = torch.sigmoid(gate) + silu * torch.sigmoid(-gate)
        y[part] = silu * up * weight
        dweights[part] = torch.einsum("ri,ri->r", dy, silu * up)
        dc[part, :inner] = dy * up * slope * weight
        dc[part, inner:] = dy * silu * weight
    return dc, y, dweights


def exact(case, seed):
    s = prepare(case, seed)
    return {"keep": _exact_keep, "back": _exact_back}.get(case["op"], _exact_products)(s, case)
