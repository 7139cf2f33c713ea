"""The expert operators under measurement: the routing choice, MXFP4 coding, the grouped MXFP4
product and the MXFP4 expert FFN, as cases with their inputs, one pass in plain torch or through the
library, the work they cannot do without, and their values in 64 bits.

Shapes of the cases: one MoE layer of hidden 2048, 64 experts top-6, inter 1408 over 13312 tokens
(prefill fan-in) or 329 tokens (decode fan-in), a small layer of hidden 1024, 16 experts top-4,
inter 512 over 128 tokens, and generic odd sizes.
"""
import math

import torch

own = False  # set by the tools: the library's operators instead of the plain forms

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---- cases ---------------------------------------------------------------------------------
def _select(name, tokens, experts, topk, score, dtype, bias=False, groups=1, topk_groups=1,
            group_top=1, renorm=False, scaling=1.0, mask=False):
    return {"name": name, "op": "select", "tokens": tokens, "experts": experts, "topk": topk,
            "score": score, "dtype": dtype, "bias": bias, "groups": groups,
            "topk_groups": topk_groups, "group_top": group_top, "renorm": renorm,
            "scaling": scaling, "mask": mask}


def _code(name, tokens, cols, dtype, rule="floor", topk=1):
    return {"name": name, "op": "code", "tokens": tokens, "cols": cols, "dtype": dtype,
            "rule": rule, "topk": topk}


def _product(name, tokens, topk, experts, m, k, swiglu, dtype, skew=False):
    return {"name": name, "op": "product", "tokens": tokens, "topk": topk, "experts": experts,
            "m": m, "k": k, "swiglu": swiglu, "dtype": dtype, "skew": skew}


def _ffn(name, tokens, topk, experts, hidden, inter, skew=False):
    return {"name": name, "op": "ffn", "tokens": tokens, "topk": topk, "experts": experts,
            "hidden": hidden, "inter": inter, "dtype": "bf16", "skew": skew}


def listed():
    return [
        # the gate of one decode step of 16 peers
        _select("select decode", 329, 64, 6, "softmax", "f32"),
        # the gate of a prefill fan-in: sigmoid scores, balance bias, 4 of 8 expert groups
        _select("select prefill groups", 13312, 256, 8, "sigmoid", "f32", bias=True, groups=8,
                topk_groups=4, group_top=2, renorm=True, scaling=2.5),
        # odd sizes, bf16 logits, experts taken out per token (some tokens have none left)
        _select("select masked odd", 4999, 60, 4, "softmax", "bf16", renorm=True, mask=True),
        # one token's activations before a product: latency
        _code("code one token", 1, 2048, "bf16"),
        # a prefill fan-in's tokens
        _code("code prefill", 13312, 2048, "bf16"),
        # fp32 rows of an odd count, gathered once per chosen expert
        _code("code routed odd f32", 1999, 1408, "f32", rule="ceil", topk=4),
        # the gate/up projection of a decode step: the weights' bytes count
        _product("product decode", 329, 6, 64, 2816, 2048, True, "bf16"),
        # the down projection of a prefill fan-in: the tensor cores count
        _product("product prefill", 13312, 6, 64, 2048, 1408, False, "bf16"),
        # a small layer with a skewed gate, outputs in fp32
        _product("product small skewed f32", 128, 4, 16, 1024, 512, False, "f32", skew=True),
        # one token through its six experts
        _ffn("experts one token", 1, 6, 64, 2048, 1408),
        # one decode step
        _ffn("experts decode", 329, 6, 64, 2048, 1408),
        # one prefill fan-in
        _ffn("experts prefill", 13312, 6, 64, 2048, 1408),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["select", "code", "product", "ffn"])
    if op == "select":
        groups = rng.choice([1, 1, 2, 4, 8])
        per = rng.randint(2, 256 // groups)
        if groups == 1:
            per = rng.randint(8, 256)
        experts = groups * per
        topk_groups = rng.randint(1, groups)
        topk = rng.randint(1, min(16, topk_groups * per))
        c = _select("", _log(rng, 1, 40000), experts, topk, rng.choice(["softmax", "sigmoid"]),
                    rng.choice(["f32", "bf16"]), bias=rng.random() < 0.5, groups=groups,
                    topk_groups=topk_groups, group_top=rng.choice([1, 2]),
                    renorm=rng.random() < 0.5, scaling=rng.choice([1.0, 2.5]),
                    mask=rng.random() < 0.25)
    elif op == "code":
        cols = 32 * rng.randint(1, 128)
        topk = rng.choice([1, 1, 2, 6])
        c = _code("", _log(rng, 1, max(1, 27000000 // (cols * topk))), cols,
                  rng.choice(["bf16", "f32"]), rule=rng.choice(["floor", "ceil"]), topk=topk)
    else:
        experts = rng.randint(1, 128)
        topk = rng.randint(1, min(8, experts))
        hidden = 32 * rng.randint(2, 64)
        inter = 32 * rng.randint(2, 44)
        tokens = _log(rng, 1, min(13312, 70000 // topk))
        skew = rng.random() < 0.3
        if op == "ffn":
            c = _ffn("", tokens, topk, experts, hidden, inter, skew)
        else:
            swiglu = rng.random() < 0.5
            m = 2 * inter if swiglu else 8 * rng.randint(8, 256)
            c = _product("", tokens, topk, experts, m, hidden, swiglu,
                         "bf16" if swiglu else rng.choice(["bf16", "f32"]), skew)
    del c["name"]
    return c


# ---- inputs --------------------------------------------------------------------------------
def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _pack_nibbles(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _encode(x, rule):
    """[..., cols] fp32 -> codes uint8 [..., cols / 2], scales uint8 [..., cols / 32]."""
    b = x.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    frac, expo = torch.frexp(amax)  # amax = frac * 2^expo, frac in [0.5, 1)
    shift = expo - 3
    if rule == "ceil":  # the smallest scale whose 6 reaches amax
        shift = shift + (frac > 0.75)
    shift = torch.where(amax > 0, shift, -127).clamp(min=-127)
    fine = torch.isfinite(amax)
    a = torch.ldexp(b.abs(), -shift.unsqueeze(-1))
    mag = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
           + (a >= 3.5) + (a > 5.0))
    code = torch.where(fine.unsqueeze(-1), mag + 8 * torch.signbit(b), 0).to(torch.uint8)
    scale = torch.where(fine, shift + 127, 255).to(torch.uint8)
    return _pack_nibbles(code.flatten(-2)), scale


def _decode(codes, scales):
    """The fp32 values that codes and scales stand for."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    v = lut[n.int()].unflatten(-1, (-1, 32))
    s = torch.ldexp(torch.ones((), device=codes.device), scales.int() - 127)
    s = torch.where(scales == 255, math.nan, s)
    return (v * s.unsqueeze(-1)).flatten(-2)


def _routing(c, g):
    """Rows per expert of a seeded gate: offsets on the device, and the largest group."""
    t, e = c["tokens"], c["experts"]
    logits = torch.randn(t, e, generator=g, device="cuda")
    if c["skew"]:
        logits += 1.5 * torch.log(torch.arange(1, e + 1, device="cuda").float() ** -1.2)
    ids = logits.topk(c["topk"], dim=1).indices.flatten()
    counts = torch.bincount(ids, minlength=e)
    off = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
    off[1:] = counts.cumsum(0)
    return off, int(counts.max())


def _weight(e, m, k, g, swiglu):
    w = torch.randn(e, m, k, generator=g, device="cuda") * (1.0 / math.sqrt(k))
    codes, scales = _encode(w, "floor")
    if own:  # laid out once, when a layer's weights are loaded
        from combine_peer_slot_gb300 import runtime
        return {"codes": codes, "scales": scales,
                "handle": runtime.Mx4Weight(codes, scales, swiglu=swiglu)}
    return {"codes": codes, "scales": scales}


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c}
    if c["op"] == "select":
        t, e = c["tokens"], c["experts"]
        logits = torch.randn(t, e, generator=g, device="cuda")
        if c["mask"]:
            gone = torch.rand(t, e, generator=g, device="cuda") < 0.2
            gone |= torch.rand(t, 1, generator=g, device="cuda") < 0.02
            logits.masked_fill_(gone, -math.inf)
        s["logits"] = logits.to(_dtype(c["dtype"]))
        s["bias"] = 0.1 * torch.randn(e, generator=g, device="cuda") if c["bias"] else None
    elif c["op"] == "code":
        x = torch.randn(c["tokens"], c["cols"], generator=g, device="cuda")
        # tokens of different norm, a few large features, as activations have them
        x *= torch.exp(torch.randn(c["tokens"], 1, generator=g, device="cuda"))
        x *= 1 + 20 * (torch.rand(1, c["cols"], generator=g, device="cuda") < 0.01)
        s["x"] = x.to(_dtype(c["dtype"]))
        s["rows"] = None
        if c["topk"] > 1:  # positions t * topk + j in expert order
            n = c["tokens"] * c["topk"]
            s["rows"] = torch.randperm(n, generator=g, device="cuda").int()
    else:
        s["offsets"], s["most"] = _routing(c, g)
        n, k = c["tokens"] * c["topk"], c["k"] if c["op"] == "product" else c["hidden"]
        s["codes"], s["scales"] = _encode(torch.randn(n, k, generator=g, device="cuda"), "floor")
        if c["op"] == "product":
            s["weight"] = _weight(c["experts"], c["m"], k, g, c["swiglu"])
        else:
            s["w13"] = _weight(c["experts"], 2 * c["inter"], k, g, True)
            s["wd"] = _weight(c["experts"], k, c["inter"], g, False)
    return s


# ---- plain forms ---------------------------------------------------------------------------
def _ranked(v):
    """Indices of the last axis in descending order of v, equal values by index."""
    return v.sort(dim=-1, descending=True, stable=True).indices


def _select_plain(s, c, real=torch.float64):
    """Scores and choice in 64 bits (two scores next to each other decide an id)."""
    l = s["logits"].to(real)
    e, k, groups = c["experts"], c["topk"], c["groups"]
    bad = torch.isnan(l).any(-1, keepdim=True)
    open_ = l > -math.inf
    if c["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-l))
    else:
        top = l.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
        p = torch.exp(l - top)
        score = p / p.sum(-1, keepdim=True).clamp(min=1e-300)
    if s["bias"] is None:
        choice = l  # the score rises with the logit
        by_group = score
    else:
        choice = by_group = score + s["bias"].to(real)
    choice = choice.masked_fill(~open_, -math.inf)
    if groups > 1:
        v = by_group.masked_fill(~open_, -math.inf).unflatten(-1, (groups, -1))
        best = v.sort(dim=-1, descending=True).values[..., :c["group_top"]]
        some = best[..., 0] > -math.inf
        gs = best.masked_fill(best == -math.inf, 0).sum(-1).masked_fill(~some, -math.inf)
        keep = torch.zeros_like(some).scatter(-1, _ranked(gs)[..., :c["topk_groups"]], True)
        choice = choice.masked_fill(~keep.repeat_interleave(e // groups, -1), -math.inf)
    ids = _ranked(choice)[..., :k]
    taken = choice.gather(-1, ids) > -math.inf
    w = score.gather(-1, ids) * taken
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True).clamp(min=1e-300)
    w = (w * c["scaling"]).masked_fill(bad, math.nan)
    ids = ids.masked_fill(~taken | bad, -1)
    return ids.int(), w


def _grouped_plain(x, off, w, most):
    """y[r] = w[expert of r] x[r]: each expert's rows in a block of their own."""
    n, e = x.shape[0], w.shape[0]
    r = torch.arange(n, device=x.device)
    g = torch.searchsorted(off[1:].contiguous(), r.int(), right=True)
    pos = r - off[g]
    b = x.new_zeros(e, most, x.shape[1])
    b[g, pos] = x
    return torch.bmm(b, w.transpose(1, 2))[g, pos]


def _swiglu_plain(y):
    gate, up = y.chunk(2, -1)
    return gate / (1 + torch.exp(-gate)) * up


def _run_plain(s, c):
    if c["op"] == "select":
        ids, w = _select_plain(s, c)
        return {"ids": ids, "weights": w.float()}
    if c["op"] == "code":
        x = s["x"].float()
        if s["rows"] is not None:
            x = x[s["rows"] // c["topk"]]
        return {"values": _decode(*_encode(x, c["rule"])).to(_dtype(c["dtype"]))}
    x = _decode(s["codes"], s["scales"])
    if c["op"] == "product":
        w = _decode(s["weight"]["codes"], s["weight"]["scales"])
        y = _grouped_plain(x, s["offsets"], w, s["most"])
        return {"out": (_swiglu_plain(y) if c["swiglu"] else y).to(_dtype(c["dtype"]))}
    w = _decode(s["w13"]["codes"], s["w13"]["scales"])
    h = _swiglu_plain(_grouped_plain(x, s["offsets"], w, s["most"])).bfloat16().float()
    w = _decode(s["wd"]["codes"], s["wd"]["scales"])
    y = _grouped_plain(_decode(*_encode(h, "floor")), s["offsets"], w, s["most"])
    return {"out": y.to(_dtype(c["dtype"]))}


def _run_own(s, c):
    from combine_peer_slot_gb300 import runtime
    if c["op"] == "select":
        ids, w = runtime.route_select(
            s["logits"], c["topk"], bias=s["bias"], score=c["score"], n_groups=c["groups"],
            topk_groups=c["topk_groups"], group_top=c["group_top"], renorm=c["renorm"],
            routed_scaling=c["scaling"])
        return {"ids": ids, "weights": w}
    if c["op"] == "code":
        q = runtime.mx4_quantize(s["x"], src_rows=s["rows"], topk=c["topk"], rule=c["rule"])
        return {"values": runtime.mx4_dequantize(q, _dtype(c["dtype"]))}
    x = runtime.Mx4(s["codes"], s["scales"])
    if c["op"] == "product":
        return {"out": runtime.mx4_gemm(x, s["offsets"], s["weight"]["handle"],
                                        out_dtype=_dtype(c["dtype"]))}
    return {"out": runtime.mx4_ffn(x, s["offsets"], s["w13"]["handle"], s["wd"]["handle"],
                                   out_dtype=_dtype(c["dtype"]))}


def run(state):
    return (_run_own if own else _run_plain)(state, state["case"])


# ---- work and values -----------------------------------------------------------------------
def _experts_hit(c):
    """Experts that get a row, on average over an even gate."""
    return c["experts"] * (1 - (1 - c["topk"] / c["experts"]) ** c["tokens"])


def work(case):
    c = case
    if c["op"] == "select":
        t, e = c["tokens"], c["experts"]
        size = 2 if c["dtype"] == "bf16" else 4
        return {"bytes": t * e * size + t * c["topk"] * 8 + (4 * e if c["bias"] else 0),
                "flops": 4 * t * e}
    size = 2 if c["dtype"] == "bf16" else 4
    n = c["tokens"] * c["topk"]
    if c["op"] == "code":  # rows in, codes and scales out and in again, values out
        return {"bytes": c["tokens"] * c["cols"] * size + n * c["cols"] * (2 * 17 / 32 + size),
                "flops": 4 * n * c["cols"]}
    code = 17 / 32  # bytes of one MXFP4 value with its share of the scale
    if c["op"] == "product":
        m, k = c["m"], c["k"]
        out = m // 2 if c["swiglu"] else m
        return {"bytes": _experts_hit(c) * m * k * code + n * k * code + n * out * size,
                "flops": 2 * n * m * k}
    h, i = c["hidden"], c["inter"]
    return {"bytes": _experts_hit(c) * 3 * h * i * code + n * h * code + n * h * size,
            "flops": 6 * n * h * i}


def _value64(codes, scales):
    """MXFP4 values in 64 bits, from the format: sign, two exponent bits, one fraction bit."""
    n = torch.stack((codes % 16, codes // 16), -1).flatten(-2).long()
    sign, ex, fr = 1.0 - 2.0 * (n // 8), (n // 2) % 4, (n % 2).double()
    v = torch.where(ex == 0, fr / 2, (1 + fr / 2) * torch.exp2((ex - 1).double())) * sign
    scale = torch.exp2(scales.double() - 127).repeat_interleave(32, -1)
    return v * scale


def _nearest64(x, rule):
    """Each value of x (64 bits) as its MXFP4 block holds it: nearest, ties to an even fraction."""
    b = x.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    # 2^-30: over what log2 may be off at a power of two, under the gap to the next fp32 value
    tiny = 2.0 ** -30
    fit = (torch.floor(torch.log2(amax) + tiny) - 2 if rule == "floor"
           else torch.ceil(torch.log2(amax / 6) - tiny))
    scale = torch.exp2(fit.clamp(min=-127))
    a = (b / scale).abs().clamp(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    return (torch.sign(b) * torch.round(a / step) * step * scale).flatten(-2)


def _grouped64(x, off, w):
    out = x.new_zeros(x.shape[0], w[0].shape[1])
    at = off.tolist()
    for e in range(len(at) - 1):
        if at[e + 1] > at[e]:
            out[at[e]:at[e + 1]] = x[at[e]:at[e + 1]] @ _value64(w[0][e], w[1][e]).T
    return out


def _glu64(y):
    h = y.shape[1] // 2
    return y[:, :h] * torch.sigmoid(y[:, :h]) * y[:, h:]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "select":
        l = s["logits"].double()
        t, e, per = c["tokens"], c["experts"], c["experts"] // c["groups"]
        score = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, -1).nan_to_num(0.0)
        shut = torch.isinf(l)
        value = l.clone() if s["bias"] is None else score + s["bias"].double()
        rank = score.clone() if s["bias"] is None else value.clone()
        value[shut] = -math.inf
        rank[shut] = -math.inf
        if c["groups"] > 1:
            top = torch.topk(rank.view(t, c["groups"], per), min(per, c["group_top"]), -1).values
            total = torch.where(torch.isinf(top), 0.0, top).sum(-1)
            total[torch.isinf(top[..., 0])] = -math.inf
            # a group is in when fewer than topk_groups others are ahead of it
            a, b = total.unsqueeze(-1), total.unsqueeze(-2)
            idx = torch.arange(c["groups"], device="cuda")
            ahead = ((b > a) | ((b == a) & (idx.view(1, 1, -1) < idx.view(1, -1, 1)))).sum(-1)
            value.view(t, c["groups"], per)[ahead >= c["topk_groups"]] = -math.inf
        ids = torch.full((t, c["topk"]), -1, dtype=torch.int32, device="cuda")
        w = torch.zeros(t, c["topk"], dtype=torch.float64, device="cuda")
        for j in range(c["topk"]):
            best = value.amax(-1, keepdim=True)
            i = (value == best).to(torch.uint8).argmax(-1, keepdim=True)
            has = ~torch.isinf(best)
            ids[:, j:j + 1] = torch.where(has, i, -1).int()
            w[:, j:j + 1] = torch.where(has, score.gather(1, i), 0.0)
            value.scatter_(1, i, -math.inf)
        if c["renorm"]:
            total = w.sum(-1, keepdim=True)
            w = torch.where(total > 0, w / total, w)
        return {"ids": ids, "weights": w * c["scaling"]}
    if c["op"] == "code":
        x = s["x"].double()
        if s["rows"] is not None:
            x = x[(s["rows"].long() / c["topk"]).floor().long()]
        return {"values": _nearest64(x, c["rule"])}
    x = _value64(s["codes"], s["scales"])
    if c["op"] == "product":
        y = _grouped64(x, s["offsets"], (s["weight"]["codes"], s["weight"]["scales"]))
        return {"out": _glu64(y) if c["swiglu"] else y}
    h = _glu64(_grouped64(x, s["offsets"], (s["w13"]["codes"], s["w13"]["scales"])))
    h = _nearest64(h.bfloat16().double(), "floor")
    return {"out": _grouped64(h, s["offsets"], (s["wd"]["codes"], s["wd"]["scales"]))}
