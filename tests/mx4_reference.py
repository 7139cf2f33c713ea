"""Plain 64-bit implementations of the routing choice and of MXFP4, for the
tests of the library's operators: written from the definitions, on torch
tensors of any device."""
import math

import torch

VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def select(logits, topk, bias=None, score="softmax", n_groups=1, topk_groups=1, group_top=1,
           renorm=False, routed_scaling=1.0):
    """(ids, weights fp64): one row at a time, by sorting (value, index)."""
    rows, E = logits.shape
    L = logits.double().cpu()
    B = None if bias is None else bias.double().cpu()
    ids = torch.full((rows, topk), -1, dtype=torch.int32)
    w = torch.zeros((rows, topk), dtype=torch.float64)
    per = E // n_groups
    for t in range(rows):
        l = L[t]
        if bool(torch.isnan(l).any()) or (B is not None and bool(torch.isnan(B).any())) or (
                score == "softmax" and bool((l == math.inf).any())):
            w[t] = math.nan
            continue
        if score == "sigmoid":
            s = 1.0 / (1.0 + torch.exp(-l))
        else:
            p = torch.exp(l - l.max()) if l.max() > -math.inf else torch.zeros_like(l)
            s = p / p.sum() if p.sum() > 0 else p
        c = (l.clone() if B is None else s + B).tolist()
        g = c if B is not None or group_top == 1 else s.tolist()
        lv, sv = l.tolist(), s.tolist()
        ok = [e for e in range(E) if lv[e] > -math.inf and c[e] > -math.inf]
        if n_groups > 1:
            rank = []
            for q in range(n_groups):
                v = sorted((g[e] for e in ok if e // per == q), reverse=True)[:group_top]
                rank.append((-sum(v) if v else math.inf, q))
            keep = {q for _, q in sorted(rank)[:topk_groups]}
            ok = [e for e in ok if e // per in keep]
        best = sorted(ok, key=lambda e: (-c[e], e))[:topk]
        for j, e in enumerate(best):
            ids[t, j] = e
            w[t, j] = sv[e]
        if renorm and best and float(w[t].sum()) > 0:
            w[t] /= w[t].sum()
        w[t] *= routed_scaling
    return ids, w


def decode(codes, scales):
    """fp64 values of uint8 codes [..., cols / 2] and scales [..., cols / 32]."""
    lut = torch.tensor(VALUES + tuple(-v for v in VALUES), dtype=torch.float64, device=codes.device)
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    s = torch.exp2(scales.double() - 127)
    s = torch.where(scales == 255, math.nan, s)
    return lut[n] * s.repeat_interleave(32, -1)


def encode(x, rule="floor"):
    """codes and scales of x [..., cols]: the nearest of the two e2m1 values
    around each quotient, the even code at a tie."""
    b = x.double().unflatten(-1, (-1, 32))
    fine = torch.isfinite(b).all(-1)
    b = torch.where(fine.unsqueeze(-1), b, 0.0)
    amax = b.abs().amax(-1)
    _, ex = torch.frexp(amax)  # amax = f 2^ex, f in [0.5, 1)
    fit = ex - 3
    if rule == "ceil":
        fit = torch.where(amax > 6 * torch.exp2(fit.double()), fit + 1, fit)
    fit = torch.where(amax > 0, fit, -127).clamp(-127, 125)
    a = (b * torch.exp2(-fit.double()).unsqueeze(-1)).abs().clamp(max=6.0)
    lut = torch.tensor(VALUES, dtype=torch.float64, device=x.device)
    lo = (torch.searchsorted(lut, a.contiguous(), right=True) - 1).clamp(0, 7)
    hi = (lo + 1).clamp(max=7)
    dl, dh = a - lut[lo], lut[hi] - a
    code = torch.where((dh < dl) | ((dh == dl) & (lo % 2 == 1)), hi, lo)
    code = code + 8 * torch.signbit(b)
    code = torch.where(fine.unsqueeze(-1), code, 0).to(torch.uint8).flatten(-2)
    scales = torch.where(fine, fit + 127, 255).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), scales


def grouped(x, offsets, w):
    """y[r] = w[g] x[r] in fp64 and S[r, m] = sum |w| |x|; rows in no group NaN."""
    off = [max(0, min(int(v), x.shape[0])) for v in offsets.tolist()]
    y = torch.full((x.shape[0], w.shape[1]), math.nan, dtype=torch.float64, device=x.device)
    s = torch.zeros_like(y)
    for g in range(len(off) - 1):
        if off[g + 1] > off[g]:
            r = slice(off[g], off[g + 1])
            y[r] = x[r] @ w[g].T
            s[r] = x[r].abs() @ w[g].abs().T
    return y, s


def swiglu(y):
    g, u = y.chunk(2, -1)
    return g / (1 + torch.exp(-g)) * u
