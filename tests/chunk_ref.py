"""The score rule and chunk attention from their definitions, in 64 bits, and
the bounds that the kernels' roundings give."""
from __future__ import annotations

import math

import torch

D = 128


def rule(s, dist, cap, slopes):
    """s [heads, queries, keys] scaled products, dist [queries, keys] >= 0."""
    if cap:
        s = cap * torch.tanh(s / cap)
    if slopes is not None:
        s = s - slopes.double().to(s.device)[:, None, None] * dist
    return s


def score_error(q, k, scale, cap, slopes, far):
    """Bound of a score's error (natural units) for queries [.., 128] and keys
    [.., 128]: float32 sums of 128 exact products that may be cut off instead of
    rounded (128 2^-23 of the absolute sum), a few roundings of the score and of
    the distance term (2^-22 of each), the cap's own."""
    top = float(q.abs().double().amax()) * float(k.abs().double().sum(-1).amax()) * scale
    e = top * (D + 4) * 2.0 ** -23
    if cap:
        e += cap * 2.0 ** -21
    if slopes is not None:
        e += float(slopes.abs().max()) * far * 2.0 ** -22
    return e


def chunk(cu, q, k, v, prefix=None, cap=0.0, slopes=None, prior=None, scale=None):
    """(out, lse, mean |v|) in float64: rows of q [n, hq, 128], k and v [n, hkv, 128]."""
    q, k, v = q.double(), k.double(), v.double()
    hq, hkv = q.shape[1], k.shape[1]
    g = hq // hkv
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    out, lse, size = torch.zeros_like(q), torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device), torch.zeros_like(q)
    for d in range(len(cu) - 1):
        a, e = cu[d], cu[d + 1]
        if a == e:
            continue
        n = e - a
        i = torch.arange(n, device=q.device)
        seen = i[None, :] <= i[:, None]
        if prefix is not None:
            seen = seen | (i < prefix[d])[None, :]
        dist = (i[:, None] - i[None, :]).abs().double()
        kk, vv = k[a:e].repeat_interleave(g, 1), v[a:e].repeat_interleave(g, 1)
        s = rule(torch.einsum("ihc,thc->hit", q[a:e], kk) * scale, dist, cap, slopes)
        s = s.masked_fill(~seen, -math.inf)
        p = torch.softmax(s, -1)
        # a hidden token has no part in the sum, whatever it holds
        bad = ~torch.isfinite(vv)
        o = torch.einsum("hit,thc->ihc", p, vv.masked_fill(bad, 0.0))
        if bad.any():
            for h in range(hq):
                for t in torch.nonzero(bad[:, h].any(-1)).flatten().tolist():
                    rows = torch.nonzero(seen[:, t]).flatten()
                    extra = p[h, rows, t][:, None] * torch.where(bad[t, h], vv[t, h], torch.zeros_like(vv[t, h]))[None]
                    o[rows, h] = o[rows, h] + extra
        out[a:e], lse[a:e] = o, torch.logsumexp(s, -1).T
        size[a:e] = torch.einsum("hit,thc->ihc", p, vv.masked_fill(bad, 0.0).abs())
    if prior is not None:
        po, pl = prior[0].double(), prior[1].double()
        total = torch.logaddexp(lse, pl)
        w1, w0 = torch.exp(lse - total)[..., None], torch.exp(pl - total)[..., None]
        gone = (pl == -math.inf)[..., None]
        out = w1 * out + torch.where(gone, torch.zeros_like(po), w0 * po)
        size = w1 * size + torch.where(gone, torch.zeros_like(po), w0 * po.abs())
        lse = total
    return out, lse, size


def check(got, got_lse, want, want_lse, size, es):
    """bf16 outputs: half a step of the output (2^-8), half a step of every
    weight (2^-8 of the mean |v|), weights off by 2 es (their own score's and the
    sum's) and by 2^-20 (exponential, sums).  Log-sum-exp: es and a few float32
    roundings.  Infinite and NaN outputs in the same places."""
    got, want = got.double(), want
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(want), torch.isnan(got)), "NaN in other places"
    assert torch.equal(want[~fine & ~torch.isnan(want)], got[~fine & ~torch.isnan(want)])
    tol = 2.0 ** -8 * want.abs() + (1.01 * 2.0 ** -8 + 2 * es + 2.0 ** -20) * size + 1e-37
    err = torch.where(fine, (got - want).abs(), torch.zeros_like(want))
    assert bool((err <= torch.where(fine, tol, torch.ones_like(tol)))[fine].all()), float((err / tol)[fine].max())
    if got_lse is not None:
        e = (got_lse.double() - want_lse).abs()
        ok = torch.isfinite(want_lse)
        bound = es + 2.0 ** -20 + 2.0 ** -22 * want_lse.abs()
        assert bool((e <= bound)[ok].all()), float((e / bound)[ok].max())
        same = torch.equal(torch.isnan(got_lse.double()), torch.isnan(want_lse))
        assert same, "lse NaN in other places"
    return float((err / tol)[fine].max()) if fine.any() else 0.0
