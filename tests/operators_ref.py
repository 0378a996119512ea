"""The training operators in 64 bits, straight from their formulas, with error
bounds for a computation in binary32.

A bound is carried along with each value: EPS = 2^-20 stands for sixteen
roundings of binary32 (2^-24 each) per operation of the formula, which covers
the gate (an exponential and a division of a few units each), the products and
sums, and a regrouping of the recurrence. A result stored in bfloat16 adds
half a unit in the last place, 2^-9 of its size at most.
"""
from __future__ import annotations

import torch

EPS = 2.0 ** -20
BF16 = 2.0 ** -8  # one unit of bfloat16: the stored value is within half of it, the bound may shift a tie
TINY = 1e-37      # results below binary32's normal range may be flushed


def scan(x, f, h0, bounds):
    """x, f: float64 (batch, tokens, channels); bounds: per sequence (row, lo, hi).
    Returns h, h_last, the state before each token, and the bounds of h's error."""
    a, u = torch.sigmoid(f), torch.sigmoid(-f)
    h, err, before, before_err = (torch.zeros_like(x) for _ in range(4))
    last, last_err = h0.clone(), torch.zeros_like(h0)
    for s, (b, lo, hi) in enumerate(bounds):
        now, e = h0[s], torch.zeros_like(h0[s])
        for t in range(lo, hi):
            before[b, t], before_err[b, t] = now, e
            e = a[b, t] * e + EPS * (a[b, t] * now.abs() + u[b, t] * x[b, t].abs())
            now = a[b, t] * now + u[b, t] * x[b, t]
            h[b, t], err[b, t] = now, e
        last[s], last_err[s] = now, e
    return h, last, before, err, last_err, before_err


def scan_grad(x, f, h0, dy, dh_last, bounds):
    """dx, df, dh0 and the bounds of their errors."""
    a, u = torch.sigmoid(f), torch.sigmoid(-f)
    _, _, before, _, _, before_err = scan(x, f, h0, bounds)
    g, ge = torch.zeros_like(x), torch.zeros_like(x)
    dh0, dh0_err = dh_last.clone(), torch.zeros_like(dh_last)
    for s, (b, lo, hi) in enumerate(bounds):
        now, e = dh_last[s], torch.zeros_like(dh_last[s])
        for t in range(hi - 1, lo - 1, -1):
            e = e + EPS * (dy[b, t].abs() + now.abs())
            now = dy[b, t] + now
            g[b, t], ge[b, t] = now, e
            e = a[b, t] * e + EPS * a[b, t] * now.abs()
            now = a[b, t] * now
        dh0[s], dh0_err[s] = now, e
    dx, dx_err = u * g, u * (ge + EPS * g.abs())
    d = before - x
    df = g * d * a * u
    df_err = a * u * (ge * d.abs() + g.abs() * before_err + EPS * g.abs() * (before.abs() + x.abs()))
    return dx, df, dh0, dx_err, df_err, dh0_err


def stored(value, err, dtype):
    """The bound after storing in ``dtype``."""
    return err + TINY + (BF16 * value.abs() if dtype is torch.bfloat16 else EPS * value.abs())


def distill(z, t, index, temperature, scale=1.0, dloss=None):
    """loss, lse, gradient in float64 and the bounds of their errors; z, t float64."""
    n, v = z.shape
    k = t.shape[1]
    loss, lse, loss_err, lse_err = (torch.zeros(n, dtype=torch.float64) for _ in range(4))
    grad, grad_err = torch.zeros_like(z), torch.zeros_like(z)
    dloss = torch.ones(n, dtype=torch.float64) if dloss is None else dloss
    for r in range(n):
        at = [j for j in range(k) if 0 <= int(index[r, j]) < v]
        if not at or bool((t[r, at] == -torch.inf).all()):
            continue
        i = index[r, at].long()
        logp = torch.log_softmax(t[r, at] / temperature, 0)
        p = logp.exp()
        lse[r] = torch.logsumexp(z[r] / temperature, 0)
        logq = z[r] / temperature - lse[r]
        finite = z[r][torch.isfinite(z[r])] / temperature
        # an exponent's argument carries one rounding of its operands' size; the
        # sum over the vocabulary is taken in parts, each rounding of which is
        # relative to a sum of positive terms
        size = 1.0 + (finite.abs().max() if finite.numel() else 0.0)
        tsize = 1.0 + (t[r, at][torch.isfinite(t[r, at])].abs().max() / temperature if bool(torch.isfinite(t[r, at]).any()) else 0.0)
        lse_err[r] = 4 * EPS * size
        live = p > 0
        terms = p[live] * (logp[live] - logq[i][live])
        loss[r] = temperature ** 2 * terms.sum()
        loss_err[r] = temperature ** 2 * 4 * EPS * (p[live] * (tsize + size + logq[i][live].abs())).sum()
        target = torch.zeros(v, dtype=torch.float64).scatter_add_(0, i, p)
        q = logq.exp()
        g = temperature * scale * dloss[r]
        grad[r] = (q - target) * g
        grad_err[r] = (q * 4 * EPS * size + target * 4 * EPS * tsize).abs() * g.abs()
    return loss, lse, grad, loss_err, lse_err, grad_err


def check(got, want, err, what=""):
    """Every finite value within its bound, every other one the same."""
    got = got.detach().double().cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    odd = ~fine & ~torch.isnan(want)
    assert torch.equal(got[odd], want[odd]), what
    off = (got - want).abs()[fine] - err[fine]
    assert off.numel() == 0 or float(off.max()) <= 0, (what, float(off.max()), float((got - want).abs()[fine].max()))
