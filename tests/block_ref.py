"""The operators around a block in 64 bits, straight from their formulas, with
error bounds for a computation in binary32.

A bound is carried along with each value. ULP = 2^-24 is one rounding of
binary32; EPS = 2^-20 stands for sixteen of them, which covers the few operations
of a formula and a hardware exponential or square root. A sum of m terms of one
sign or both is off by at most DEEP or m roundings, whichever is fewer, of the sum of their
sizes: no summation of these kernels is deeper than 128 + its number of rows.
A result stored in bfloat16 adds half of its unit, 2^-8 of its size.
"""
from __future__ import annotations

import torch

ULP = 2.0 ** -24
EPS = 2.0 ** -20
DEEP = 128 * ULP
TINY = 1e-37  # results below binary32's normal range may be flushed


def half_unit(dtype) -> float:
    return float(torch.finfo(dtype).eps) / 2


def stored(value, err, dtype):
    """The bound after storing in ``dtype``."""
    return err + half_unit(dtype) * (value.abs() + err) + TINY


def check(got, want, err, what=""):
    """Every finite value within its bound, every other one the same."""
    got, want = got.detach().double().cpu(), want.detach().cpu()
    err = err.detach().cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    fine = torch.isfinite(want)
    odd = ~fine & ~torch.isnan(want)
    assert torch.equal(got[odd], want[odd]), what
    off = (got - want).abs()[fine] - err[fine]
    assert off.numel() == 0 or float(off.max()) <= 0, (what, float(off.max()), float((got - want).abs()[fine].max()))


# ------------------------------------------------------------------ embedding

def embed(table, tokens, scale):
    """Rows, and the bound of their error in binary32: one product."""
    v = table.shape[0]
    there = (tokens >= 0) & (tokens < v)
    rows = torch.where(there[..., None], table.double()[tokens.long().clamp(0, v - 1)] * scale, 0.0)
    return rows, ULP * rows.abs()


def embed_grad(drows, tokens, vocab, scale, add=None):
    d = drows.double().reshape(-1, drows.shape[-1])
    t = tokens.reshape(-1).long()
    keep = (t >= 0) & (t < vocab)
    sums = torch.zeros(vocab, d.shape[1], dtype=torch.float64).index_add_(0, t[keep], d[keep])
    sizes = torch.zeros_like(sums).index_add_(0, t[keep], d[keep].abs())
    counts = torch.zeros(vocab, dtype=torch.float64).index_add_(0, t[keep], torch.ones(int(keep.sum()), dtype=torch.float64))
    out = scale * sums + (0.0 if add is None else add.double())
    # as many additions as rows, a product and the sum with add
    err = ULP * (counts[:, None] + 2) * abs(scale) * sizes + ULP * out.abs()
    return out, err


# ------------------------------------------------------------------ norms

def block(x, o=None, w_post=None, gate=None, w_pre=None, r=1.0, eps=1e-6):
    """Forward in 64 bits: a dict of values and, under the same names in ``err``, bounds."""
    n, d = x.shape
    x = x.double()
    u = torch.ones(1, d, dtype=torch.float64)
    s1 = torch.ones(n, 1, dtype=torch.float64)
    groups = 1 if gate is None else gate.shape[0]
    g = torch.ones(n, d, dtype=torch.float64) if gate is None else gate.double().repeat_interleave(n // groups, 0)
    oh = torch.zeros_like(x)
    if o is not None:
        oh = o.double()
        if w_post is not None:
            s1 = 1.0 / torch.sqrt((oh * oh).mean(1, keepdim=True) + eps)
            u = w_post.double()[None]
            oh = oh * s1
    v = {"g": g, "u": g * u, "w1": u, "s1": s1, "oh": oh}
    add = v["u"] * oh if o is not None else torch.zeros_like(x)
    v["x"] = r * x + add
    err = {"oh": (DEEP + EPS) * oh.abs()}
    err["x"] = EPS * (r * x).abs() + (DEEP + 2 * EPS) * add.abs()
    v["s2"] = torch.ones(n, 1, dtype=torch.float64)
    rel = torch.zeros(n, 1, dtype=torch.float64)
    if w_pre is not None:
        square = (v["x"] ** 2).mean(1, keepdim=True) + eps
        v["s2"] = 1.0 / torch.sqrt(square)
        rel = DEEP + EPS + (v["x"].abs() * err["x"]).mean(1, keepdim=True) / square
        v["n"] = v["x"] * v["s2"] * w_pre.double()
        err["n"] = (v["s2"] * err["x"] + (v["x"] * v["s2"]).abs() * (rel + EPS)) * w_pre.double().abs()
    v["xh"] = v["x"] * v["s2"]
    err["xh"] = v["s2"] * err["x"] + v["xh"].abs() * (rel + EPS)
    v["err"], v["rel2"] = err, rel
    return v


def block_grad(x, dn=None, dx_new=None, o=None, w_post=None, gate=None, w_pre=None, r=1.0, eps=1e-6):
    """(dx, do, dw_pre, dw_post, dgate) and the bounds of their errors."""
    f = block(x, o, w_post, gate, w_pre, r, eps)
    n, d = x.shape
    xh, oh, s1, s2, u, exh, eoh = f["xh"], f["oh"], f["s1"], f["s2"], f["u"], f["err"]["xh"], f["err"]["oh"]
    y = torch.zeros_like(xh) if dx_new is None else dx_new.double()
    e = torch.zeros_like(xh) if dn is None else dn.double() * w_pre.double()
    mean = lambda t: t.mean(1, keepdim=True)  # noqa: E731
    c2 = mean(e * xh)
    c2_err = mean(e.abs() * exh) + (DEEP + EPS) * mean((e * xh).abs())
    dX = y + s2 * (e - xh * c2)
    size = y.abs() + s2 * (e.abs() + xh.abs() * mean((e * xh).abs()))
    dX_err = s2 * (exh * c2.abs() + xh.abs() * c2_err) + (2 * EPS + f["rel2"]) * size
    dx, dx_err = r * dX, abs(r) * (dX_err + EPS * dX.abs())
    out = [dx, None, None, None, None]
    errs = [dx_err, None, None, None, None]
    deep = DEEP + n * ULP
    if dn is not None:
        t = dn.double() * xh
        out[2] = t.sum(0)
        errs[2] = (dn.double().abs() * exh).sum(0) + (deep + EPS) * t.abs().sum(0)
    if o is None:
        return out, errs
    if w_post is not None:
        c1 = mean(u * oh * dX)
        # taken from two sums whose terms may be larger than their difference
        parts = mean((u * oh).abs() * (y.abs() + s2 * e.abs())) + s2 * mean((e * xh).abs()) * mean((u * oh * xh).abs())
        c1_err = mean(u.abs() * (oh.abs() * dX_err + eoh * dX.abs())) + (DEEP + 4 * EPS + f["rel2"]) * parts
        c1_err = c1_err + s2 * c2_err * mean((u * oh * xh).abs()) + s2 * c2.abs() * mean((u * oh).abs() * exh)
        out[1] = s1 * (u * dX - oh * c1)
        errs[1] = s1 * (u.abs() * dX_err + eoh * c1.abs() + oh.abs() * c1_err
                        + (DEEP + 4 * EPS) * ((u * dX).abs() + oh.abs() * parts))
    else:
        out[1], errs[1] = u * dX, u.abs() * (dX_err + EPS * dX.abs())
    t = dX * oh
    t_err = dX_err * oh.abs() + dX.abs() * eoh + EPS * t.abs()
    if w_post is not None:
        out[3] = (f["g"] * t).sum(0)
        errs[3] = (f["g"].abs() * (t_err + (deep + 2 * EPS) * t.abs())).sum(0)
    if gate is not None:
        groups = gate.shape[0]
        sums = lambda z: z.view(groups, n // groups, d).sum(1)  # noqa: E731
        out[4] = sums(f["w1"] * t)
        errs[4] = sums(f["w1"].abs() * (t_err + (deep + 2 * EPS) * t.abs()))
    return out, errs


# ------------------------------------------------------------------ policies

def policy(z, tokens, temperature, old=None, adv=None, refl=None, clip=(0.2, 0.2), kl=0.0, scale=1.0, dloss=None):
    """loss, logp, lse, gradient and the bounds of their errors (z float64 on the CPU)."""
    n, v = z.shape
    names = ("loss", "logp", "lse", "grad")
    out = {k: torch.zeros(n, dtype=torch.float64) for k in names[:3]}
    out["grad"] = torch.zeros_like(z)
    err = {k: torch.zeros_like(t) for k, t in out.items()}
    for r in range(n):
        t = int(tokens[r])
        if not 0 <= t < v:
            continue
        row = z[r] / temperature
        lse = torch.logsumexp(row, 0)
        logp = row[t] - lse
        # an exponent's argument carries roundings of its size, as far below the maximum as an
        # exponential of binary32 reaches; the sum's are relative to positive terms
        size = 105.0
        q = torch.exp(row - lse)
        live = row[torch.isfinite(row) & (row > row.max() - size)]
        reach = 1.0 + (row.max() - live.min() if live.numel() else 0.0)
        e_lse = 4 * EPS * reach + ULP * 4 * row.max().abs() + DEEP
        e_logp = 4 * EPS * reach + DEEP + 4 * ULP * logp.abs()
        out["lse"][r], err["lse"][r] = lse, e_lse
        out["logp"][r], err["logp"][r] = logp, e_logp
        if old is None:
            continue
        o, a = old[r].double(), adv[r].double()
        ratio = torch.exp(logp - o)
        e_ratio = ratio * (e_logp + EPS * (1 + (logp - o).abs()))
        low, high = 1.0 - clip[0], 1.0 + clip[1]
        edge = 4 * ULP * high
        assert min(abs(ratio - low), abs(ratio - high)) > e_ratio + edge or a == 0, "a ratio too close to a bound to tell"
        cut = bool((a > 0 and ratio > high) or (a < 0 and ratio < low))
        held = (high if a > 0 else low) if cut else ratio
        loss, slope = -held * a, torch.zeros(()) if cut else -ratio * a
        e_loss = (edge if cut else e_ratio + EPS * ratio) * a.abs()
        e_slope = torch.zeros(()) if cut else (e_ratio + EPS * ratio) * a.abs()
        if refl is not None:
            d = refl[r].double() - logp
            e_d = e_logp + EPS * d.abs()
            loss = loss + kl * (torch.exp(d) - 1 - d)
            slope = slope + kl * (1 - torch.exp(d))
            e_loss = e_loss + abs(kl) * ((torch.exp(d) + 1) * (e_d + EPS) + EPS * d.abs())
            e_slope = e_slope + abs(kl) * torch.exp(d) * (e_d + EPS) + EPS * abs(kl)
        out["loss"][r], err["loss"][r] = loss, e_loss + EPS * loss.abs()
        k = scale * (1.0 if dloss is None else dloss[r].double()) / temperature
        hot = torch.zeros(v, dtype=torch.float64)
        hot[t] = 1.0
        out["grad"][r] = k * slope * (hot - q)
        e_q = q * (4 * EPS * reach + DEEP)
        err["grad"][r] = abs(k) * ((e_slope + EPS * slope.abs()) * (hot - q).abs() + slope.abs() * (e_q + EPS * (hot + q)))
    return [out[k] for k in names], [err[k] for k in names]


# ------------------------------------------------------------------ many gradients

def clip(grads, scale, max_norm, eps):
    """norm, coefficient, clipped gradients and the relative bounds of their errors."""
    norm = torch.sqrt(sum(((g.double() * scale) ** 2).sum() for g in grads))
    coef = torch.clamp(max_norm / (norm + eps), max=1.0) if torch.isfinite(norm) else torch.ones((), dtype=torch.float64)
    rel = DEEP  # a part's squares, in binary32, before 64 bits take over
    return norm, coef, [g.double() * scale * coef for g in grads], rel
