"""Plain float64 forms of routing, the norms around a block and gradient clipping, and their
gradients by formula, written from their definitions, for the tests to compare with."""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24   # half a float32 step, relative
BF = 2.0 ** -8   # half a bfloat16 step
INF = math.inf


# ----------------------------------------------------------------------------- routing
def probabilities(z, score):
    """(s, p) of float64 rows; rows without a logit above -inf hold zeros."""
    if score == "softmax":
        s = torch.nan_to_num(torch.softmax(z, 1), nan=0.0)
        return s, s
    ls = torch.nn.functional.logsigmoid(z)
    return torch.exp(ls), torch.nan_to_num(torch.softmax(ls, 1), nan=0.0)


def choose(z, k, score, bias=None, mask=None):
    """ids [T][k] by walking each token's experts in order of (key, id); finite or -inf logits."""
    key = z if bias is None else probabilities(z, score)[0] + bias.double()
    ids = torch.full((z.shape[0], k), -1, dtype=torch.int64)
    for t in range(z.shape[0]):
        if mask is not None and not mask[t]:
            continue
        row, zr = key[t].tolist(), z[t].tolist()
        # a NaN or -inf is not chosen
        able = [e for e in range(len(row)) if zr[e] > -INF and row[e] > -INF]
        for j, e in enumerate(sorted(able, key=lambda e: (-row[e], e))[:k]):
            ids[t, j] = e
    return ids


def weights(z, ids, score, renormalize, scale):
    """[T][k], zero for slots without an expert; a function of z for autograd."""
    ok = ids >= 0
    zi = torch.gather(z, 1, ids.clamp_min(0))
    if renormalize:  # ratios of the scores, by their logarithms
        ls = zi if score == "softmax" else torch.nn.functional.logsigmoid(zi)
        w = torch.softmax(torch.where(ok, ls, torch.full_like(ls, -INF)), 1)
        w = torch.where(ok, w, torch.zeros_like(w))
    else:
        s = torch.gather(probabilities(z, score)[0], 1, ids.clamp_min(0))
        w = torch.where(ok, s, torch.zeros_like(s))
    return w * scale


def balance(z, ids, score):
    """(counts, loss, dprob)."""
    T, G = z.shape
    k = ids.shape[1]
    routed = (ids >= 0).any(1)
    n = max(1, int(routed.sum()))
    counts = torch.zeros(G, dtype=torch.int64)
    for e in ids.reshape(-1).tolist():
        if e >= 0:
            counts[e] += 1
    dprob = counts.double() * G / (k * n * n)
    p = probabilities(z, score)[1]
    return counts, (torch.where(routed[:, None], p, torch.zeros_like(p)) * dprob).sum(), dprob


def route_backward(z, ids, dw, dprob, dloss, score, renormalize, scale):
    """dlogits by the formula, and the sum of magnitudes that its rounding errors follow."""
    T, G = z.shape
    ok = (ids >= 0) & (ids < G)
    idc = torch.where(ok, ids, torch.zeros_like(ids))
    s, p = probabilities(z, score)
    dw = torch.where(ok, dw, torch.zeros_like(dw)) * scale
    if renormalize:
        v = weights(z, torch.where(ok, ids, torch.full_like(ids, -1)), score, True, 1.0)
        a = v * (dw - (dw * v).sum(1, keepdim=True))
        mag = v * (dw.abs() + (dw.abs() * v).sum(1, keepdim=True))
    else:
        a = dw * torch.gather(s, 1, idc)
        mag = a.abs()
    hit = torch.zeros_like(z).scatter_add_(1, idc, torch.where(ok, a, torch.zeros_like(a)))
    hmag = torch.zeros_like(z).scatter_add_(1, idc, torch.where(ok, mag, torch.zeros_like(a)))
    dp = torch.zeros_like(z) if dprob is None else (dprob * dloss).expand_as(z)
    base = (dp * p).sum(1, keepdim=True)
    bmag = (dp.abs() * p).sum(1, keepdim=True)
    if score == "softmax":
        if not renormalize:
            base = base + hit.sum(1, keepdim=True)
            bmag = bmag + hmag.sum(1, keepdim=True)
        dz, m = hit + p * (dp - base), hmag + p * (dp.abs() + bmag)
    else:
        ns = torch.sigmoid(-z)
        dz, m = ns * (hit + p * (dp - base)), ns * (hmag + p * (dp.abs() + bmag))
    routed = ok.any(1, keepdim=True)
    zero = torch.zeros_like(dz)
    return torch.where(routed, dz, zero), torch.where(routed, m, zero)


def spread(z):
    """How far a row's finite logits lie apart: an exponential's argument z - top is rounded once,
    which moves it by that much of half a step."""
    f = torch.where(torch.isfinite(z), z, torch.full_like(z, -INF))
    top = f.amax(1, keepdim=True)
    low = torch.where(torch.isfinite(z), z, top.expand_as(z)).amin(1, keepdim=True)
    return torch.where(torch.isfinite(top), top - low, torch.zeros_like(top))


# ------------------------------------------------------------------------------- norms
def norm_forward(x, y, weight, post, gate, alpha, eps):
    """(n, r, rstd, rstd_y) and bounds on the float32 errors of n and r before their rounding."""
    H = x.shape[1]
    rel_sum = 64 * U  # 64 additions at most in a row's sum of squares: 32 a thread, two trees of five, the rest
    rstd_y, er = None, torch.zeros_like(x)
    r = x
    if y is not None:
        u, eu = y, torch.zeros_like(y)
        if post is not None:
            rstd_y = ((y * y).mean(1) + eps) ** -0.5
            u = u * rstd_y[:, None] * post
            eu = u.abs() * (rel_sum / 2 + 6 * U)
        if gate is not None:
            u = u * gate
            eu = u.abs() * (rel_sum / 2 + 7 * U) if post is not None else u.abs() * U
        r = alpha * x + u
        er = eu + U * ((alpha * x).abs() + u.abs())
    ss = (r * r).sum(1) + eps * H
    rstd = (ss / H) ** -0.5
    rel = rel_sum / 2 + 3 * U + (r.abs() * er).sum(1) / ss.clamp_min(1e-300)
    n = r * rstd[:, None] * weight
    en = weight.abs() * rstd[:, None] * er + n.abs() * (rel + 3 * U)[:, None]
    return (n, r, rstd, rstd_y), en, er, rel


def norm_backward(dn, dr, r, rstd, y, rstd_y, weight, post, gate, alpha):
    """{name: (value, bound on the float32 error before the output's rounding)}."""
    T, H = r.shape
    c = 64 * U  # a row's sums take fewer additions, an element's value fewer operations
    one = torch.ones(H, dtype=r.dtype, device=r.device)
    zero = torch.zeros_like(r)
    dr = zero if dr is None else dr
    gw, rh = dn * weight, r * rstd[:, None]
    c1, m1 = (gw * rh).mean(1, keepdim=True), (gw * rh).abs().mean(1, keepdim=True)
    g = dr + rstd[:, None] * (gw - rh * c1)
    mg = dr.abs() + rstd[:, None] * (gw.abs() + rh.abs() * m1)
    eg = c * mg
    # a column's sum: at most T / 100 rows a CTA in turn and 80 + 8 of the CTAs' sums after them
    cs = (T / 100 + 100) * U
    out = {"dx": (alpha * g, abs(alpha) * eg + U * (alpha * g).abs()),
           "dweight": ((dn * rh).sum(0), (cs + 3 * U) * (dn * rh).abs().sum(0))}
    if y is None:
        return out
    yh = y if post is None else y * rstd_y[:, None]
    u = yh if post is None else yh * post
    ga = one if gate is None else gate
    if gate is not None:
        out["dgate"] = ((g * u).sum(0), (eg * u.abs()).sum(0) + (cs + 4 * U) * (g * u).abs().sum(0))
    d, ed = g * ga, eg * ga.abs() + U * (g * ga).abs()
    if post is None:
        out["dy"] = (d, ed)
        return out
    out["dpost_weight"] = ((d * yh).sum(0), (ed * yh.abs()).sum(0) + (cs + 4 * U) * (d * yh).abs().sum(0))
    q = ga * post * yh
    c2 = (g * q).mean(1, keepdim=True)
    # as three sums: mean((dr + rstd gw) q) - rstd c1 mean(rh q)
    m2 = ((dr.abs() + rstd[:, None] * gw.abs()) * q.abs()).mean(1, keepdim=True)
    m2 = m2 + rstd[:, None] * m1 * (rh * q).abs().mean(1, keepdim=True)
    gp = d * post
    out["dy"] = (rstd_y[:, None] * (gp - yh * c2),
                 rstd_y[:, None] * (ed * post.abs() + 4 * U * (gp.abs() + yh.abs() * c2.abs()) + yh.abs() * 2 * c * m2))
    return out
