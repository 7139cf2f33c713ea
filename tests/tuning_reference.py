"""Plain 64-bit forms of the expert load, the routing choice's gradient and the
low-rank adapters, with bounds on what fp32 arithmetic may be off."""
import math

import torch

U = 2.0 ** -24                                              # half a step of fp32
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # half a step of the outputs


def shares(l, score):
    """(scores, shares of a row's sum) of fp64 logits"""
    if score == "sigmoid":
        s = torch.sigmoid(l)
        t = s.sum(-1, keepdim=True)
        return s, torch.where(t > 0, s / t, 0.0 * t)
    top = l.amax(-1, keepdim=True)
    e = torch.exp(l - torch.where(top == -math.inf, 0.0, top))
    t = e.sum(-1, keepdim=True)
    p = torch.where(t > 0, e / t, 0.0 * t)
    return p, p


def sequences(n, offsets):
    off = [0, n] if offsets is None else [min(max(int(v), 0), n) for v in offsets]
    return list(zip(off[:-1], off[1:]))


def hits(ids, E):
    """[T, E] fp64: how often each row chose each expert"""
    h = torch.zeros(ids.shape[0], E, dtype=torch.float64, device=ids.device)
    ok = (ids >= 0) & (ids < E)
    return h.scatter_add_(1, torch.where(ok, ids, 0).long(), ok.double())


def balance(logits, ids, score, offsets=None):
    """(loss [S], counts [S, E])"""
    l = logits.double()
    E, k = l.shape[1], ids.shape[1]
    _, p = shares(l, score)
    h = hits(ids, E)
    loss, counts = [], []
    for lo, hi in sequences(l.shape[0], offsets):
        n = hi - lo
        c = h[lo:hi].sum(0)
        counts.append(c)
        loss.append((c * p[lo:hi].sum(0)).sum() * E / (k * n * n) if n else c.sum())
    return torch.stack(loss), torch.stack(counts).int()


def weights(logits, ids, score, renorm, scaling):
    """route_select's weights for given ids (differentiable)"""
    s, _ = shares(logits, score)
    ok = (ids >= 0) & (ids < logits.shape[1])
    w = torch.where(ok, s.gather(1, torch.where(ok, ids, 0).long()), 0.0)
    if renorm:
        t = w.sum(1, keepdim=True)
        w = torch.where(t > 0, w / torch.where(t > 0, t, 1.0), 0.0)
    return w * scaling


def route_grad(logits, ids, score, d_weights=None, renorm=False, scaling=1.0, counts=None, d_loss=None, offsets=None):
    """(the gradient in fp64, what fp32 arithmetic may be off in it, in units of U)"""
    l = logits.double()
    T, E = l.shape
    k = ids.shape[1] if ids is not None else 1
    s, p = shares(l, score)
    rest = torch.sigmoid(-l) if score == "sigmoid" else torch.ones_like(s)  # (1 - s without its cancellation)
    g = torch.zeros_like(l)
    if d_loss is not None:
        for i, (lo, hi) in enumerate(sequences(T, offsets)):
            if hi > lo:
                c = counts[i].double()
                g[lo:hi] = d_loss[i].double() * (c * E - c.sum()) / (k * (hi - lo) ** 2)
    d = p * rest * (g - (p * g).sum(-1, keepdim=True))
    size = p * rest * 2 * g.abs().amax(-1, keepdim=True)
    if d_weights is not None:
        ok = (ids >= 0) & (ids < E)
        at = torch.where(ok, ids, 0).long()
        dw = torch.where(ok, d_weights.double(), 0.0) * scaling
        big = dw.abs().amax(1, keepdim=True)
        sc, rc = torch.where(ok, s.gather(1, at), 0.0), rest.gather(1, at)
        if renorm:
            top = torch.where(ok, l.gather(1, at), -math.inf)
            if score == "softmax":  # shares of the chosen: their own softmax
                _, sh = shares(top, "softmax")
                sh = sh * (sc.sum(1, keepdim=True) > 0)  # (all 0 in fp64: route_select's weights are 0)
            else:
                t = sc.sum(1, keepdim=True)
                sh = torch.where(t > 0, sc / torch.where(t > 0, t, 1.0), 0.0)
            part = sh * rc * (dw - (sh * dw).sum(1, keepdim=True))
            psize = sh * rc * 2 * big
        else:
            part, psize = sc * rc * dw, sc * rc * big
            if score == "softmax":
                d = d - p * part.sum(1, keepdim=True)
                size = size + p * big
        d = d.scatter_add(1, at, torch.where(ok, part, 0.0))
        size = size.scatter_add(1, at, torch.where(ok, psize, 0.0))
    bad = torch.isnan(l).any(1) | ((l == math.inf).any(1) if score == "softmax" else False)
    d[bad] = math.nan
    return d, size


def adapters(ids, src, w1, w2, scale, base):
    """(out, u, and what fp32 sums may be off in u, and in out before its rounding, u in `parts` bits)"""
    T, L = src.shape[0], w1.shape[0]
    R, K, M = w1.shape[1], w1.shape[2], w2.shape[2]
    u = torch.zeros(T, R, dtype=torch.float64, device=src.device)
    eu = torch.zeros_like(u)
    out = torch.zeros(T, M, dtype=torch.float64, device=src.device) if base is None else base.double().clone()
    size = torch.zeros_like(out)
    eo = torch.zeros_like(out)
    for l in range(L):
        rows = (ids == l).nonzero().flatten()
        if rows.numel() == 0:
            continue
        x, a, b = src[rows].double(), w1[l].double(), w2[l].double()
        s = float(scale[l]) if scale is not None else 1.0
        u[rows] = x @ a.T
        # sums of the tensor cores may cut instead of round: 2 U a step, a step
        # is sixteen columns of one part
        eu[rows] = (3 * K / 16 + 40) * 2 * U * (x.abs() @ a.abs().T)
        out[rows] += s * (u[rows] @ b)
        size[rows] = abs(s) * (u[rows].abs() @ b.abs())
        eo[rows] = abs(s) * (eu[rows] @ b.abs()) + (3 * R / 16 + 8) * 2 * U * size[rows]
    return out, u, eu, eo, size


def adapter_grads(ids, x, dy, u, a, b, scale, d_base):
    """(dx, da, db, bounds of dx as in adapters, of da, of db)"""
    dx, v, ev, eo, size = adapters(ids, dy, b, a, scale, d_base)
    L, R, K = a.shape
    M = b.shape[2]
    da, db = torch.zeros(L, R, K, dtype=torch.float64, device=x.device), torch.zeros(L, R, M, dtype=torch.float64, device=x.device)
    ea, eb = torch.zeros_like(da), torch.zeros_like(db)
    for l in range(L):
        rows = (ids == l).nonzero().flatten()
        if rows.numel() == 0:
            continue
        s = float(scale[l]) if scale is not None else 1.0
        xr, yr, vr, ur = x[rows].double(), dy[rows].double(), v[rows], u[rows].double()
        n = 6 * rows.numel() / 16 + 24
        da[l], db[l] = s * (vr.T @ xr), s * (ur.T @ yr)
        ea[l] = abs(s) * (n * 2 * U * (vr.abs().T @ xr.abs()) + ev[rows].T @ xr.abs())
        eb[l] = abs(s) * n * 2 * U * (ur.abs().T @ yr.abs())
    return dx, da, db, eo, size, ea, eb
