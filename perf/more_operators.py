"""The tuned gate and the adapters under measurement: the balance loss with per-expert counts, the
gradient of the routing choice, low-rank adapters of many requests beside a shared projection, and
their gradients, as cases with their inputs, one pass in plain torch or through the library, the work
they cannot do without, and their values in 64 bits.

Shapes of the cases: one MoE layer of hidden 2048, 64 experts top-6, inter 1408 (gate and up 2816)
over 13312 tokens of 4 peers (prefill fan-in) or 329 tokens of 16 (decode fan-in), a small layer of
hidden 1024, inter 512 over 128 tokens, and generic odd sizes.
"""
import math

import torch

own = False  # set by the tools: the library's operators instead of the plain forms

TILE = 64  # tokens of one adapter that the plain form multiplies at a time


# ---- cases ---------------------------------------------------------------------------------
def _balance(name, tokens, experts, topk, seqs, score, dtype, mask=False):
    return {"name": name, "op": "balance", "tokens": tokens, "experts": experts, "topk": topk,
            "seqs": seqs, "score": score, "dtype": dtype, "mask": mask}


def _gate(name, tokens, experts, topk, seqs, score, dtype, mask=False, renorm=False, scaling=1.0):
    return {"name": name, "op": "gate", "tokens": tokens, "experts": experts, "topk": topk,
            "seqs": seqs, "score": score, "dtype": dtype, "mask": mask, "renorm": renorm,
            "scaling": scaling}


def _apply(name, tokens, k, m, rank, adapters, x, y, runs=0, none=0.0, keep=False):
    return {"name": name, "op": "apply", "tokens": tokens, "k": k, "m": m, "rank": rank,
            "adapters": adapters, "x": x, "y": y, "runs": runs, "none": none, "keep": keep}


def _grad(name, tokens, k, m, rank, adapters, x, y, runs=0, none=0.0):
    return {"name": name, "op": "grad", "tokens": tokens, "k": k, "m": m, "rank": rank,
            "adapters": adapters, "x": x, "y": y, "runs": runs, "none": none}


def listed():
    return [
        # the load of one decode step of 16 peers, a loss for each peer, with the logits' gradient
        _balance("balance decode", 329, 64, 6, 16, "softmax", "f32"),
        # a prefill fan-in, a loss for each of its 4 peers
        _balance("balance prefill", 13312, 64, 6, 4, "softmax", "f32"),
        # many experts, sigmoid scores, one loss over the batch
        _balance("balance wide sigmoid", 13312, 256, 8, 1, "sigmoid", "f32"),
        # the whole gradient of a gate step over a prefill fan-in
        _gate("gate grad prefill", 13312, 256, 8, 4, "sigmoid", "f32", renorm=True, scaling=2.5),
        # odd sizes, bf16 logits, experts taken out per token (some tokens have none left)
        _gate("gate grad masked odd", 4999, 60, 4, 7, "softmax", "bf16", mask=True, renorm=True),
        # one token of one request beside the gate and up projection: latency
        _apply("adapters one token", 1, 2048, 2816, 16, 8, "bf16", "bf16"),
        # a decode step: every row a request of its own, 64 adapters loaded, some rows without one
        _apply("adapters decode", 329, 2048, 2816, 16, 64, "bf16", "bf16", none=0.1),
        # a prefill fan-in of 24 requests over 8 adapters
        _apply("adapters prefill", 13312, 2048, 2816, 16, 8, "bf16", "bf16", runs=24),
        # beside the gate's own product: fp32 logits, the inner products kept for the gradients
        _apply("adapters gate logits", 13312, 2048, 64, 8, 8, "bf16", "f32", runs=24, keep=True),
        # a small layer's training step, mixed rows
        _grad("adapters grad small", 128, 1024, 1024, 8, 4, "bf16", "bf16"),
        # a training step over a prefill fan-in: gate and up projection, larger rank
        _grad("adapters grad prefill", 13312, 2048, 2816, 64, 8, "bf16", "bf16", runs=24),
        # the gradient of gate logits in fp32, odd sizes, some rows without an adapter
        _grad("adapters grad gate odd", 1999, 1408, 60, 13, 5, "bf16", "f32", runs=11, none=0.2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["balance", "gate", "apply", "grad"])
    if op in ("balance", "gate"):
        experts = rng.randint(2, 256)
        args = (_log(rng, 1, 13312), experts, rng.randint(1, min(16, max(1, experts // 2))), _log(rng, 1, 64),
                rng.choice(["softmax", "sigmoid"]), rng.choice(["f32", "bf16"]),
                rng.random() < 0.25)
        if op == "balance":
            c = _balance("", *args)
        else:
            c = _gate("", *args, renorm=rng.random() < 0.5, scaling=rng.choice([1.0, 2.5]))
    else:
        k, m = _log(rng, 16, 4096), _log(rng, 16, 4096)
        if rng.random() < 0.7:  # most projections have sizes of whole eights
            k, m = max(16, k // 8 * 8), max(16, m // 8 * 8)
        rank = rng.choice([4, 8, 16, 32, 64, rng.randint(1, 64)])
        adapters = min(_log(rng, 1, 128), max(1, 20000000 // (rank * (k + m))))
        tokens = _log(rng, 1, max(1, min(13312, 50000000 // (k + m))))
        x, y = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
        runs = rng.choice([0, _log(rng, 1, 40)])
        none = rng.choice([0.0, 0.1, 0.5])
        if op == "apply":
            c = _apply("", tokens, k, m, rank, adapters, x, y, runs, none, rng.random() < 0.5)
        else:
            c = _grad("", tokens, k, m, rank, adapters, x, y, runs, none)
    del c["name"]
    return c


# ---- inputs --------------------------------------------------------------------------------
def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _offsets(n, parts, g):
    """parts + 1 ascending offsets from 0 to n, drawn; parts may be empty."""
    cut = torch.randint(0, n + 1, (parts - 1,), generator=g, device="cuda").sort().values
    off = torch.zeros(parts + 1, dtype=torch.int32, device="cuda")
    off[1:parts] = cut
    off[parts] = n
    return off


def _gate_inputs(c, s, g):
    t, e, k = c["tokens"], c["experts"], c["topk"]
    # some experts are liked better, as by a gate in training
    logits = 1.5 * torch.randn(t, e, generator=g, device="cuda")
    logits += 0.7 * torch.randn(1, e, generator=g, device="cuda")
    if c["mask"]:
        gone = torch.rand(t, e, generator=g, device="cuda") < 0.2
        gone |= torch.rand(t, 1, generator=g, device="cuda") < 0.02
        logits.masked_fill_(gone, -math.inf)
    s["logits"] = logits.to(_dtype(c["dtype"]))
    best = s["logits"].float().sort(dim=-1, descending=True, stable=True)
    s["ids"] = best.indices[:, :k].masked_fill(best.values[:, :k] == -math.inf, -1).int()
    s["offsets"] = _offsets(t, c["seqs"], g)
    s["d_loss"] = 0.01 * (0.5 + torch.rand(c["seqs"], generator=g, device="cuda"))
    if c["op"] == "gate":
        s["d_weights"] = torch.randn(t, k, generator=g, device="cuda") / t
        s["counts"] = _counts(s, c)


def _adapter_inputs(c, s, g):
    t, k, m, r, n = c["tokens"], c["k"], c["m"], c["rank"], c["adapters"]
    few = c["runs"] or t  # requests: runs of neighbouring rows, or every row its own
    ids = torch.randint(0, n, (few,), generator=g, device="cuda")
    ids[torch.rand(few, generator=g, device="cuda") < c["none"]] = -1
    if c["runs"]:
        off = _offsets(t, few, g)
        ids = ids[torch.searchsorted(off[1:].contiguous(), torch.arange(t, device="cuda").int(), right=True)]
    s["ids"] = ids.int()
    s["x"] = torch.randn(t, k, generator=g, device="cuda").to(_dtype(c["x"]))
    s["a"] = (torch.randn(n, r, k, generator=g, device="cuda") / math.sqrt(k)).bfloat16()
    s["b"] = (torch.randn(n, r, m, generator=g, device="cuda") / math.sqrt(r)).bfloat16()
    s["scale"] = 0.5 + torch.rand(n, generator=g, device="cuda")
    # the rows in adapter order, TILE at a time: what the plain form multiplies
    key = torch.where(s["ids"] < 0, n, s["ids"]).long()
    order = key.argsort(stable=True)
    count = torch.bincount(key, minlength=n + 1)[:n]
    tiles = (count + TILE - 1) // TILE
    first, at = tiles.cumsum(0) - tiles, count.cumsum(0) - count
    order = order[:int(count.sum())]
    l = key[order]
    s["order"] = order
    s["slot"] = first[l] * TILE + torch.arange(order.numel(), device="cuda") - at[l]
    s["tile_adapter"] = torch.repeat_interleave(torch.arange(n, device="cuda"), tiles)
    if own:  # made once for a batch, for all its layers' projections
        from combine_peer_slot_gb300 import runtime
        s["batch"] = runtime.LoraBatch(s["ids"], n)
    if c["op"] == "apply":
        s["base"] = torch.randn(t, m, generator=g, device="cuda").to(_dtype(c["y"]))
    else:
        s["dy"] = (torch.randn(t, m, generator=g, device="cuda") / math.sqrt(t)).to(_dtype(c["y"]))
        s["d_base"] = (torch.randn(t, k, generator=g, device="cuda") / math.sqrt(t)).to(_dtype(c["x"]))
        s["u"] = _inner(s, s["x"], s["a"])  # kept by the forward pass


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}
    (_gate_inputs if case["op"] in ("balance", "gate") else _adapter_inputs)(case, s, g)
    return s


# ---- plain forms ---------------------------------------------------------------------------
def _in_sequence(s, c):
    """[seqs, tokens]: 1 where the token belongs to the sequence."""
    t = torch.arange(c["tokens"], device="cuda")
    return ((t >= s["offsets"][:-1, None]) & (t < s["offsets"][1:, None])).float()


def _counts(s, c):
    hot = (s["ids"].unsqueeze(-1) == torch.arange(c["experts"], device="cuda").int()).sum(1)
    return (_in_sequence(s, c) @ hot.float()).round().int()  # whole numbers under 2^24


def _scores(l, kind):
    """Scores, and their shares of a row's sum."""
    if kind == "sigmoid":
        sc = 1 / (1 + torch.exp(-l))
        return sc, sc / sc.sum(-1, keepdim=True).clamp(min=1e-38)
    top = l.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = torch.exp(l - top)
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-38)
    return p, p


def _balance_factor(s, c, counts):
    """[seqs, 1]: experts / (topk tokens^2), 0 for no tokens."""
    n = (s["offsets"][1:] - s["offsets"][:-1]).float().unsqueeze(1)
    return torch.where(n > 0, c["experts"] / (c["topk"] * n * n), 0)


def _d_logits(s, c, counts, sc, p):
    """The gradient of the balance loss and, for a gate, of the chosen weights."""
    member = _in_sequence(s, c)
    # less the mean count, which the shares, adding up to 1, do not feel
    off = counts.float() - counts.sum(1, keepdim=True).float() / c["experts"]
    gp = member.T @ (off * _balance_factor(s, c, counts) * s["d_loss"].unsqueeze(1))
    inner = gp - (p * gp).sum(-1, keepdim=True)
    if c["score"] == "sigmoid":
        d = p * (1 - sc) * inner
    else:
        d = p * inner
    if c["op"] == "gate":
        have = (s["ids"] >= 0).float()
        at = s["ids"].clamp(min=0).long()
        chosen, dw = sc.gather(1, at) * have, s["d_weights"] * have * c["scaling"]
        if c["renorm"]:
            share = chosen / chosen.sum(-1, keepdim=True).clamp(min=1e-38)
            dw = dw - (share * dw).sum(-1, keepdim=True)
            if c["score"] == "sigmoid":
                share = share * (1 - chosen)
            part = share * dw * have
            d = d.scatter_add(1, at, part)
        elif c["score"] == "sigmoid":
            d = d.scatter_add(1, at, chosen * (1 - chosen) * dw)
        else:
            part = chosen * dw
            d = d.scatter_add(1, at, part) - p * part.sum(-1, keepdim=True)
    return d.to(_dtype(c["dtype"]))


def _tiles(s, v):
    """Rows in adapter order, as tiles of one adapter each, in 32 bits."""
    n = s["tile_adapter"].numel()
    out = torch.zeros(n * TILE, v.shape[1], device=v.device)
    out[s["slot"]] = v[s["order"]].float()
    return out.view(n, TILE, v.shape[1])


def _rows(s, tiles, like):
    """Back to the rows' own order, zero where no adapter is."""
    out = torch.zeros(like.shape[0], tiles.shape[2], device=tiles.device)
    out[s["order"]] = tiles.reshape(-1, tiles.shape[2])[s["slot"]]
    return out


def _inner(s, v, w):
    """w[l] v_t of each row: [tokens, rank]."""
    return _rows(s, torch.bmm(_tiles(s, v), w[s["tile_adapter"]].float().transpose(1, 2)), v)


def _outer(s, u, w):
    """scale[l] w[l]^T u_t of each row."""
    t = torch.bmm(_tiles(s, u), w[s["tile_adapter"]].float())
    return _rows(s, t * s["scale"][s["tile_adapter"]].view(-1, 1, 1), u)


def _weight_grad(s, u, v, n):
    """scale[l] sum over l's rows of u_t v_t^T: [adapters, rank, columns]."""
    t = torch.bmm(_tiles(s, u).transpose(1, 2), _tiles(s, v))
    hot = (torch.arange(n, device="cuda").unsqueeze(1) == s["tile_adapter"]).float()
    return (hot @ t.flatten(1)).view(n, u.shape[1], -1) * s["scale"].view(-1, 1, 1)


def _run_plain(s, c):
    if c["op"] in ("balance", "gate"):
        sc, p = _scores(s["logits"].float(), c["score"])
        counts = _counts(s, c) if c["op"] == "balance" else s["counts"]
        d = _d_logits(s, c, counts, sc, p)
        if c["op"] == "gate":
            return {"d_logits": d}
        share = _in_sequence(s, c) @ p
        loss = (counts.float() * share * _balance_factor(s, c, counts)).sum(1)
        return {"loss": loss, "counts": counts, "d_logits": d}
    if c["op"] == "apply":
        u = _inner(s, s["x"], s["a"])
        y = (s["base"].float() + _outer(s, u, s["b"])).to(s["base"].dtype)
        return {"y": y, "u": u} if c["keep"] else {"y": y}
    v = _inner(s, s["dy"], s["b"])
    dx = (s["d_base"].float() + _outer(s, v, s["a"])).to(s["d_base"].dtype)
    n = c["adapters"]
    return {"dx": dx, "da": _weight_grad(s, v, s["x"], n), "db": _weight_grad(s, s["u"], s["dy"], n)}


def _run_own(s, c):
    from combine_peer_slot_gb300 import runtime
    if c["op"] == "balance":
        loss, counts = runtime.balance_loss(s["logits"], s["ids"], score=c["score"],
                                            seq_offsets=s["offsets"])
        d = runtime.route_backward(s["logits"], s["ids"], score=c["score"], counts=counts,
                                   d_loss=s["d_loss"], seq_offsets=s["offsets"])
        return {"loss": loss, "counts": counts, "d_logits": d}
    if c["op"] == "gate":
        return {"d_logits": runtime.route_backward(
            s["logits"], s["ids"], d_weights=s["d_weights"], score=c["score"], renorm=c["renorm"],
            routed_scaling=c["scaling"], counts=s["counts"], d_loss=s["d_loss"],
            seq_offsets=s["offsets"])}
    if c["op"] == "apply":
        if c["keep"]:
            y, u = runtime.lora_apply(s["batch"], s["x"], s["a"], s["b"], s["base"], scale=s["scale"],
                                      keep=True)
            return {"y": y, "u": u}
        return {"y": runtime.lora_apply(s["batch"], s["x"], s["a"], s["b"], s["base"],
                                        scale=s["scale"])}
    dx, da, db = runtime.lora_backward(s["batch"], s["x"], s["dy"], s["u"], s["a"], s["b"],
                                       d_base=s["d_base"], scale=s["scale"])
    return {"dx": dx, "da": da, "db": db}


def run(state):
    return (_run_own if own else _run_plain)(state, state["case"])


# ---- work and values -----------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] in ("balance", "gate"):
        t, e, k = c["tokens"], c["experts"], c["topk"]
        size = 2 if c["dtype"] == "bf16" else 4
        return {"bytes": 2 * t * e * size + 4 * t * k + 4 * c["seqs"] * (e + 2)
                + (4 * t * k if c["op"] == "gate" else 0),
                "flops": 10 * t * e}
    t, k, m, r, n = c["tokens"] * (1 - c["none"]), c["k"], c["m"], c["rank"], c["adapters"]
    sx, sy = (2 if c[v] == "bf16" else 4 for v in ("x", "y"))
    few = (c["runs"] or c["tokens"]) * (1 - c["none"])
    used = n * (1 - (1 - 1 / n) ** few)  # adapters that get a row, on average
    w = used * r * (k + m) * 2
    if c["op"] == "apply":
        return {"bytes": t * k * sx + 2 * c["tokens"] * m * sy + w + (4 * c["tokens"] * r if c["keep"] else 0),
                "flops": 2 * t * r * (k + m)}
    return {"bytes": t * k * sx + t * m * sy + 2 * c["tokens"] * k * sx + w + 4 * t * r
            + 4 * n * r * (k + m),
            "flops": 4 * t * r * (k + m)}


def _exact_gate(c, s):
    l, off = s["logits"].double(), s["offsets"].tolist()
    e, k = c["experts"], c["topk"]
    if c["score"] == "sigmoid":
        sc = torch.sigmoid(l)
        total = sc.sum(-1, keepdim=True)
        p = torch.where(total > 0, sc / total, 0.0)
    else:
        sc = p = torch.softmax(l, -1).nan_to_num(0.0)
    rest = 1 - sc if c["score"] == "sigmoid" else 1.0
    d = torch.zeros_like(l)
    losses, counted = [], []
    for i in range(c["seqs"]):
        lo, hi = off[i], off[i + 1]
        ids = s["ids"][lo:hi].flatten()
        cnt = torch.bincount(ids[ids >= 0].long(), minlength=e).double()
        if c["op"] == "gate":
            cnt = s["counts"][i].double()
        f = e / (k * max(1, hi - lo))  # f cnt: 1 for an even gate
        mean = p[lo:hi].sum(0) / max(1, hi - lo)
        losses.append((f * cnt * mean).sum())
        counted.append(cnt)
        # (less the mean, exactly 0 for an even gate; the shares add up to 1)
        v = s["d_loss"][i].double() * f * (cnt - cnt.mean()) / max(1, hi - lo)
        q = p[lo:hi]
        d[lo:hi] += q * (v - (q @ v).unsqueeze(1)) * (rest if c["score"] != "sigmoid" else rest[lo:hi])
    if c["op"] == "balance":
        return {"loss": torch.stack(losses), "counts": torch.stack(counted).int(), "d_logits": d}
    hot = torch.zeros_like(l)  # dL / d score of each expert
    have = s["ids"] >= 0
    dw = torch.where(have, s["d_weights"].double(), 0.0) * c["scaling"]
    at = s["ids"].clamp(min=0).long()
    if c["renorm"]:
        picked = torch.where(have, sc.gather(1, at), 0.0)
        total = picked.sum(1, keepdim=True)
        mean = (picked * dw).sum(1, keepdim=True) / total.clamp(min=1e-300)
        dw = torch.where(have & (total > 0), (dw - mean) / total.clamp(min=1e-300), 0.0)
    hot.scatter_add_(1, at, dw)
    if c["score"] == "sigmoid":
        d += sc * (1 - sc) * hot
    else:
        d += sc * (hot - (sc * hot).sum(1, keepdim=True))
    return {"d_logits": d}


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] in ("balance", "gate"):
        return _exact_gate(c, s)
    apply = c["op"] == "apply"
    src, w1, w2 = (s["x"], s["a"], s["b"]) if apply else (s["dy"], s["b"], s["a"])
    out = (s["base"] if apply else s["d_base"]).double()
    inner = torch.zeros(c["tokens"], c["rank"], dtype=torch.float64, device="cuda")
    da, db = (torch.zeros(v.shape, dtype=torch.float64, device="cuda") for v in (s["a"], s["b"]))
    for l in range(c["adapters"]):
        rows = (s["ids"] == l).nonzero().flatten()
        if rows.numel() == 0:
            continue
        sl = s["scale"][l].double()
        v = src[rows].double() @ w1[l].double().T
        inner[rows] = v
        out[rows] += sl * (v @ w2[l].double())
        if not apply:
            da[l] = sl * (v.T @ s["x"][rows].double())
            db[l] = sl * (s["u"][rows].double().T @ s["dy"][rows].double())
    if apply:
        return {"y": out, "u": inner} if c["keep"] else {"y": out}
    return {"dx": out, "da": da, "db": db}
