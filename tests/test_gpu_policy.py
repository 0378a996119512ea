"""Token log-probabilities, the clipped policy loss and its gradient, against the
formulas in 64 bits."""
import ctypes
import math

import numpy as np
import pytest
import torch

import block_ref as ref
from gpu_helpers import Guarded
from zero_sharded_mixed_flat_gb300 import binding as zb

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
CLIP, KL = (0.2, 0.28), 0.04


def rand(shape, seed, scale=1.0):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape) * scale)


def logits_of(n, v, dtype, seed, pad=0, offset=0, scale=2.5):
    flat = torch.zeros(offset + n * (v + pad), dtype=dtype)
    flat[offset:].view(n, v + pad)[:, :v].copy_(rand((n, v), seed, scale).to(dtype))
    return flat.cuda()[offset:].view(n, v + pad)[:, :v]


def sample(z, temperature, seed, padding=True):
    """Tokens, and the values of other policies, of which no ratio is close to a bound."""
    n, v = z.shape
    rng = np.random.default_rng(seed)
    tokens = torch.from_numpy(rng.integers(0, v, n))
    logp = torch.log_softmax(z.double().cpu() / temperature, 1).gather(1, tokens[:, None])[:, 0].nan_to_num(0.0, 0.0, -50.0)
    moved = torch.from_numpy(np.resize([0.05, -0.1, 0.5, -0.6, 0.18, -0.15, 1.5, 0.0], n))
    old, refl = (logp - moved).float(), (logp + rand(n, seed + 1, 0.3)).float()
    adv = torch.from_numpy(np.resize([1.3, -0.7, 0.4, -1.1, 2.0], n)).float()
    if padding:
        tokens[n // 2::5] = -1
        if n > 6:
            tokens[4], tokens[6] = v, -(1 << 31)
    return tokens, old, adv, refl


def check_policy(z, tokens, old, adv, refl, temperature, clip=CLIP, kl=KL, seed=50):
    dt, n = z.dtype, z.shape[0]
    dloss = rand(n, seed).abs().float()
    (loss, logp, lse, grad), (e_loss, e_logp, e_lse, e_grad) = ref.policy(z.double().cpu(), tokens, temperature, old, adv, refl,
                                                                         clip, kl, 64.0, dloss)
    f32 = torch.float32
    how = (tokens.cuda(), old.cuda(), adv.cuda(), None if refl is None else refl.cuda(), clip, kl, temperature)
    got_logp, got_lse = zb.token_logp(z, how[0], temperature)
    ref.check(got_logp, logp, ref.stored(logp, e_logp, f32), "logp alone")
    ref.check(got_lse, lse, ref.stored(lse, e_lse, f32), "lse")
    one_loss, one_logp, one = zb.policy_loss_grad(z, *how, 64.0, dloss.cuda())
    two_loss, two_logp, kept = zb.policy_loss(z, *how)
    two = zb.policy_grad(z, kept, *how, 64.0, dloss.cuda())
    for got in (one_loss, two_loss):
        ref.check(got, loss, ref.stored(loss, e_loss, f32), "loss")
    for got in (one_logp, two_logp):
        ref.check(got, logp, ref.stored(logp, e_logp, f32), "logp")
    for got in (one, two):
        assert got.dtype == dt
        ref.check(got, grad, ref.stored(grad, e_grad, dt), "gradient")
    narrow = (how[0].clamp(-(1 << 31), (1 << 31) - 1).to(torch.int32), *how[1:])
    again = zb.policy_loss_grad(z, *narrow, 64.0, dloss.cuda())
    assert all(torch.equal(p, q) for p, q in zip(again, (one_loss, one_logp, one)))
    # in the logits' own memory: the bits of another output's on the same memory (of a row that lies
    # differently the sum is taken in another order)
    mine = z.clone()
    want = zb.policy_loss_grad(mine, *how, 64.0, dloss.cuda())[2]
    zb.policy_loss_grad(mine, *how, 64.0, dloss.cuda(), out=mine)
    assert torch.equal(mine, want)
    ref.check(mine, grad, ref.stored(grad, e_grad, dt), "gradient in place")
    mine = z.clone()
    zb.policy_grad(mine, kept, *how, 64.0, dloss.cuda(), out=mine)
    assert torch.equal(mine, two)


SIZES = [(1, 1), (1, 2), (3, 7), (9, 31), (40, 255), (9, 1000), (8, 5003), (5, 50257), (3, 131075), (2, 262144)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("temperature", [1.0, 0.7])
@pytest.mark.parametrize("n,v", SIZES)
def test_policy(n, v, temperature, dtype):
    z = logits_of(n, v, DT[dtype], 1)
    tokens, old, adv, refl = sample(z, temperature, 2)
    check_policy(z, tokens, old, adv, refl if n != 8 else None, temperature)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,offset", [(1, 0), (8, 8), (3, 5), (0, 1), (47, 0)])
@pytest.mark.parametrize("v", [37, 1000, 5003, 20011])
def test_rows_of_any_alignment(v, pad, offset, dtype):
    z = logits_of(6, v, DT[dtype], 3, pad, offset)
    tokens, old, adv, refl = sample(z, 1.0, 4)
    tokens[0], tokens[1] = 0, v - 1
    logp = torch.log_softmax(z.double().cpu(), 1).gather(1, tokens.clamp(0, v - 1)[:, None])[:, 0]
    old[:2] = (logp[:2] - 0.05).float()
    check_policy(z, tokens, old, adv, refl, 1.0)
    # a gradient whose rows lie differently from the logits'
    how = (tokens.cuda(), old.cuda(), adv.cuda())
    want = zb.policy_loss_grad(z, *how)[2]
    for p, o in ((0, 0), (2, 1), (5, 3), (8, 8)):
        flat = torch.full((o + 6 * (v + p),), 7.0, dtype=DT[dtype], device="cuda")
        out = flat[o:].view(6, v + p)
        zb.policy_loss_grad(z, *how, out=out[:, :v])
        assert torch.equal(out[:, :v], want) and bool((out[:, v:] == 7.0).all()) and bool((flat[:o] == 7.0).all())
        out.fill_(7.0)
        zb.policy_grad(z, zb.policy_loss(z, *how)[2], *how, out=out[:, :v])
        assert torch.allclose(out[:, :v].float(), want.float(), rtol=2.0 ** -7, atol=1e-30)
        assert bool((out[:, v:] == 7.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,v", [(610, 5003), (1000, 50257), (305, 131075), (5000, 70)])
def test_many_rows(n, v, dtype):
    """More rows than blocks fit at once; the formulas on the GPU in 64 bits."""
    z = torch.randn(n, v, generator=torch.Generator("cuda").manual_seed(5), device="cuda").mul_(2.5).to(DT[dtype])
    tokens = torch.randint(0, v, (n,), generator=torch.Generator("cuda").manual_seed(6), device="cuda")
    logp = torch.cat([torch.log_softmax(p.double(), 1) for p in z[:, :].split(64)]).gather(1, tokens[:, None])[:, 0]
    old = (logp - 0.05).float()
    adv = torch.linspace(-1, 1, n, device="cuda")
    tokens[::7] = -1
    loss, got, grad = zb.policy_loss_grad(z, tokens, old, adv, clip=CLIP)
    two_loss, two_logp, kept = zb.policy_loss(z, tokens, old, adv, clip=CLIP)
    two = zb.policy_grad(z, kept, tokens, old, adv, clip=CLIP)
    there = tokens >= 0
    ratio = torch.exp(logp - old.double())
    bound = ref.DEEP + 4 * ref.EPS * 30  # logits within 30 of each other
    for a, b in ((loss, got), (two_loss, two_logp)):
        ref.check(b, logp * there, bound * (1 + logp.abs()), "logp")
        ref.check(a, -ratio * adv.double() * there, 2 * bound * (1 + logp.abs()) * adv.double().abs() + ref.TINY, "loss")
    for lo in range(0, n, 64):
        cut = slice(lo, min(lo + 64, n))
        q = torch.softmax(z[cut].double(), 1)
        hot = torch.zeros_like(q).scatter_(1, tokens[cut].clamp(min=0)[:, None], 1.0)
        slope = torch.where(there, -ratio * adv.double(), 0.0)[cut][:, None]
        want, err = slope * (hot - q), 4 * bound * slope.abs() * (hot + q)
        for g in (grad, two):
            ref.check(g[cut], want, ref.stored(want, err, DT[dtype]), "gradient")


def on_the_gpu(n, v, dtype, pad=0):
    """Both gradients and all values of n rows against the formulas in 64 bits on the GPU."""
    gen = torch.Generator("cuda").manual_seed(7)
    z = torch.randn(n, v + pad, generator=gen, device="cuda").mul_(2.5).to(DT[dtype])[:, :v]
    tokens = torch.randint(0, v, (n,), generator=gen, device="cuda")
    tokens[0], tokens[n // 2] = v - 1, 0
    logq = torch.cat([torch.log_softmax(p.double(), 1) for p in z.split(8)])
    logp = logq.gather(1, tokens[:, None])[:, 0]
    old, adv = (logp + 0.05).float(), torch.linspace(-1, 1.1, n, device="cuda")
    loss, got, grad = zb.policy_loss_grad(z, tokens, old, adv)
    two_loss, two_logp, kept = zb.policy_loss(z, tokens, old, adv)
    two = zb.policy_grad(z, kept, tokens, old, adv)
    alone = zb.token_logp(z, tokens)[0]
    slope = -torch.exp(logp - old.double()) * adv.double()
    bound = ref.DEEP + 4 * ref.EPS * 30
    for b in (got, two_logp, alone):
        ref.check(b, logp, bound * (1 + logp.abs()), "logp")
    for a in (loss, two_loss):
        ref.check(a, slope, 2 * bound * (1 + logp.abs()) * adv.double().abs() + ref.TINY, "loss")
    for r in range(n):
        q = torch.exp(logq[r])
        hot = torch.zeros_like(q)
        hot[tokens[r]] = 1.0
        want, err = slope[r] * (hot - q), 4 * bound * slope[r].abs() * (hot + q)
        for g in (grad, two):
            ref.check(g[r], want, ref.stored(want, err, DT[dtype]), "gradient")
    mine = z.clone()
    want = zb.policy_loss_grad(mine, tokens, old, adv)[2]
    zb.policy_loss_grad(mine, tokens, old, adv, out=mine)
    assert torch.equal(mine, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 2, 38, 43, 50, 60, 76, 77, 100, 152])
def test_rows_shared_out_over_clusters_of_every_size(n, dtype):
    on_the_gpu(n, 20011, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,v,pad", [(2, 500003, 0), (3, 1000001, 7), (40, 250007, 1), (1, 3000017, 0)])
def test_rows_larger_than_shared_memory(n, v, pad, dtype):
    on_the_gpu(n, v, dtype, pad)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("v", [90, 5003, 50257])
def test_masks_and_rows_far_from_zero(v, dtype):
    """Logits closed by -inf or any large negative number count for nothing; what all logits
    of a row have in common does not matter."""
    dt, n = DT[dtype], 6
    z = logits_of(n, v, dt, 7)
    tokens, old, adv, refl = sample(z, 1.0, 8, padding=False)
    at = torch.arange(v)
    shut = torch.stack([at < v // 2, at >= v // 2, at % 16 < 8, at % 7 != 3, torch.ones(v, dtype=torch.bool), at < 0])
    shut[torch.arange(n), tokens] = False
    same = torch.where(shut, -math.inf, z.double().cpu())
    logp = torch.log_softmax(same, 1).gather(1, tokens[:, None])[:, 0]
    old = (logp + torch.tensor([0.05, -0.05, 0.1, -0.1, 0.4, 0.03])).float()
    (loss, lp, _, grad), (e_loss, e_lp, _, e_grad) = ref.policy(same, tokens, 1.0, old, adv, None, CLIP, 0.0)
    how = (tokens.cuda(), old.cuda(), adv.cuda(), None, CLIP)
    for mask in (-math.inf, -1e4, -1e9, -1e12, -1e20, torch.finfo(dt).min):
        m = z.masked_fill(shut.cuda(), mask)
        a, b, g = zb.policy_loss_grad(m, *how)
        _, c, kept = zb.policy_loss(m, *how)
        two = zb.policy_grad(m, kept, *how)
        for got in (b, c):
            ref.check(got, lp, ref.stored(lp, e_lp, torch.float32), "logp")
        ref.check(a, loss, ref.stored(loss, e_loss, torch.float32), "loss")
        for got in (g, two):
            ref.check(got, grad, ref.stored(grad, e_grad, dt), "gradient")
    for move in (3e3, -1e6, 1e10, -1e30):
        m = (logits_of(n, v, torch.float32, 9) + move).contiguous()
        m[5] = move
        same = m.double().cpu() - m.double().cpu().max(1, keepdim=True).values
        lp = torch.log_softmax(same, 1).gather(1, tokens[:, None])[:, 0]
        old = (lp + 0.05).float()
        (loss, lp, _, grad), (e_loss, e_lp, _, e_grad) = ref.policy(same, tokens, 1.0, old, adv, None, CLIP, 0.0)
        how = (tokens.cuda(), old.cuda(), adv.cuda(), None, CLIP)
        a, b, g = zb.policy_loss_grad(m, *how)
        two = zb.policy_grad(m, zb.policy_loss(m, *how)[2], *how)
        ref.check(b, lp, ref.stored(lp, e_lp, torch.float32), "logp")
        for got in (g, two):
            ref.check(got, grad, ref.stored(grad, e_grad, torch.float32), "gradient")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("v", [90, 50257])
def test_padding_rows_hold_anything_and_bad_rows_stay_alone(v, dtype):
    z = logits_of(7, v, DT[dtype], 10)
    tokens, old, adv, refl = (t.cuda() for t in sample(z, 1.0, 11, padding=False))
    clean = zb.policy_loss_grad(z, tokens, old, adv, refl, CLIP, KL)
    z[1] = math.nan
    old[1] = adv[1] = refl[1] = math.nan
    tokens[1] = -1
    z[3, v // 3] = math.nan
    z[4, v - 1] = math.inf
    z[5] = -math.inf
    got = zb.policy_loss_grad(z, tokens, old, adv, refl, CLIP, KL)
    loss, logp, kept = zb.policy_loss(z, tokens, old, adv, refl, CLIP, KL)
    two = zb.policy_grad(z, kept, tokens, old, adv, refl, CLIP, KL)
    for r in range(7):
        if r in (0, 2, 6):
            assert all(torch.equal(a[r], b[r]) for a, b in zip(got, clean))
        elif r == 1:
            assert all(bool((a[r] == 0).all()) for a in (*got, loss, logp, two))
        else:
            assert bool(torch.isnan(got[1][r])) and bool(torch.isnan(got[2][r]).all()) and bool(torch.isnan(two[r]).all())
    lp, lse = zb.token_logp(z, tokens)
    assert float(lp[1]) == float(lse[1]) == 0.0 and bool(torch.isnan(lp[3]))
    # a token that is masked out: an impossible sample, ratio zero
    z = logits_of(1, v, DT[dtype], 12)
    z[0, 5] = -math.inf
    five, one = torch.tensor([5], device="cuda"), torch.ones(1, device="cuda")
    loss, logp, grad = zb.policy_loss_grad(z, five, -one, one)
    assert float(logp) == -math.inf and float(loss) == 0.0 and bool((grad == 0).all())


def test_bounds_of_the_ratio_and_the_zero_advantage():
    """Slope and loss on either side of both bounds, for advantages of either sign."""
    v = 11
    z = logits_of(1, v, torch.float32, 13).expand(12, v).contiguous()
    tokens = torch.full((12,), 4)
    logp = torch.log_softmax(z.double().cpu(), 1)[:, 4]
    ratio = torch.tensor([0.79, 0.81, 1.0, 1.27, 1.29, 3.0] * 2, dtype=torch.float64)
    old = (logp - torch.log(ratio)).float()
    adv = torch.tensor([1.0] * 6 + [-1.0] * 6)
    check_policy(z, tokens, old, adv, None, 1.0)
    grad = zb.policy_loss_grad(z, tokens.cuda(), old.cuda(), adv.cuda(), None, CLIP)[2]
    assert [bool((g == 0).all()) for g in grad] == [False] * 4 + [True] * 2 + [True] + [False] * 5
    check_policy(z, tokens, old, torch.zeros(12), None, 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("v", [90, 50257])
def test_ratios_and_references_beyond_binary32(v, dtype):
    """e^x alone is infinite in binary32; what it is multiplied by makes it zero, or finite again."""
    n = 8
    z = logits_of(n, v, DT[dtype], 23)
    tokens = torch.arange(n) * 11
    logp = torch.log_softmax(z.double().cpu(), 1).gather(1, tokens[:, None])[:, 0]
    old = (logp - torch.tensor([100.0, 100.0, 95.0, 81.0, 300.0, 0.05, 79.9, 100.0])).float()
    adv = torch.tensor([0.0, 1.0, -1e-9, -1e-3, 0.0, 1.0, -1e-3, 1e-12])
    check_policy(z, tokens, old, adv, None, 1.0)
    old = (logp - 0.05).float()
    refl = (logp + torch.tensor([100.0, 95.0, 81.0, 300.0, 0.3, 79.9, -100.0, 88.9])).float()
    check_policy(z, tokens, old, adv, refl, 1.0, kl=0.0)
    refl[3] = (logp[3] + 90).float()
    # the first row's slope is 1e-6 e^100 = 2.69e37: times 64 it is 1.7e39, beyond the largest binary32 (3.4e38), and
    # a row's gradient is then not finite; the loss is, and the other rows are
    loss, _, grad = zb.policy_loss_grad(z, tokens.cuda(), old.cuda(), adv.cuda(), refl.cuda(), CLIP, 1e-6, 1.0, 64.0)
    want = 1e-6 * math.exp(float(refl[0].double() - logp[0]))
    assert abs(float(loss[0]) - want) <= 400 * ref.EPS * want  # the argument, some 100, carries its logp's error
    assert not math.isfinite(float(grad[0, 0])) and bool(torch.isfinite(grad[1:]).all())
    check_policy(z[1:], tokens[1:], old[1:], adv[1:], refl[1:], 1.0, kl=1e-6)


def test_gradient_against_differences():
    v, n = 301, 5
    z = logits_of(n, v, torch.float32, 14)
    tokens, old, adv, refl = sample(z, 1.3, 15, padding=False)
    w, d, step = rand(n, 16).abs().float(), rand((n, v), 17), 1e-5
    grad = zb.policy_loss_grad(z, tokens.cuda(), old.cuda(), adv.cuda(), refl.cuda(), CLIP, KL, 1.3, 3.0, w.cuda())[2]

    def value(sign):
        out = ref.policy(z.double().cpu() + sign * step * d, tokens, 1.3, old, adv, refl, CLIP, KL)[0][0]
        return 3.0 * float((out * w.double()).sum())

    slope, mine = (value(1) - value(-1)) / (2 * step), grad.double().cpu() * d
    assert abs(slope - float(mine.sum())) <= 1e-5 * float(mine.abs().sum())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("v", [37, 5003, 50257, 131075])
def test_only_outputs_are_written(v, dtype):
    n, dt = 3, DT[dtype]
    z = logits_of(n, v, dt, 18)
    tokens, old, adv, refl = (t.cuda() for t in sample(z, 1.0, 19))
    grad, loss, kept = Guarded(n * v, dt), Guarded(n, torch.float32), Guarded(3 * n, torch.float32)
    a = zb._policy(z, tokens, old, adv, refl, CLIP, KL, 1.0)
    st = torch.cuda.current_stream().cuda_stream
    L = zb.lib()
    assert L.zg_policy_loss_grad(ctypes.byref(a), 1.0, None, loss.view.data_ptr(), None, grad.view.data_ptr(), v, st) == 0
    first = grad.view.clone()
    assert L.zg_policy_loss(ctypes.byref(a), loss.view.data_ptr(), None, kept.view.data_ptr(), st) == 0
    assert L.zg_policy_grad(ctypes.byref(a), kept.view.data_ptr(), 1.0, None, grad.view.data_ptr(), v, st) == 0
    torch.cuda.synchronize()
    assert grad.intact() and loss.intact() and kept.intact()
    assert torch.equal(first.view(n, v), zb.policy_loss_grad(z, tokens, old, adv, refl, CLIP, KL)[2])


def test_no_rows():
    z = torch.empty(0, 100, dtype=torch.bfloat16, device="cuda")
    t, f = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
    assert zb.token_logp(z, t)[0].shape == (0,)
    assert zb.policy_loss(z, t, f, f)[2].shape == (0, 3)
    assert zb.policy_loss_grad(z, t, f, f)[2].shape == (0, 100)


def test_same_bits_streams_and_graphs():
    z = logits_of(400, 20011, torch.bfloat16, 20)
    tokens, old, adv, refl = (t.cuda() for t in sample(z, 1.0, 21))

    def both(z, stream=None):
        how = (tokens, old, adv, refl, CLIP, KL)
        two = zb.policy_loss(z, *how, stream=stream)
        return (*two, zb.policy_grad(z, two[2], *how, stream=stream), *zb.policy_loss_grad(z, *how, stream=stream),
                *zb.token_logp(z, tokens, stream=stream))

    want = both(z)
    torch.cuda.synchronize()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    got = both(z, side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    s = torch.zeros_like(z)
    graphs, kept = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for g in graphs:
        with torch.cuda.graph(g):
            kept.append(both(s))
    s.copy_(z)
    torch.cuda.synchronize()
    for _ in range(3):
        for g, st in zip(graphs, (side, other)):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for got in kept:
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_refusals():
    z, t, f = torch.zeros(4, 100, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda"), \
        torch.zeros(4, device="cuda")
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        zb.token_logp(z.half(), t)
    with pytest.raises(TypeError, match="int32 or int64"):
        zb.token_logp(z, f)
    with pytest.raises(ValueError, match="tokens must have shape"):
        zb.token_logp(z, t[:3])
    with pytest.raises(ValueError, match="contiguous"):
        zb.token_logp(z.t(), torch.zeros(100, dtype=torch.int64, device="cuda"))
    for bad in (0.0, -1.0, math.nan, math.inf, 1e-45):
        with pytest.raises(zb.ZgError, match="temperature"):
            zb.token_logp(z, t, bad)
        with pytest.raises(zb.ZgError, match="temperature"):
            zb.policy_loss(z, t, f, f, temperature=bad)
    for low, high, name in ((-0.1, 0.2, "clip_low"), (1.5, 0.2, "clip_low"), (0.2, -1.0, "clip_high"),
                            (0.2, math.inf, "clip_high"), (math.nan, 0.2, "clip_low")):
        with pytest.raises(zb.ZgError, match=name):
            zb.policy_loss(z, t, f, f, clip=(low, high))
    with pytest.raises(zb.ZgError, match="kl must be finite"):
        zb.policy_loss(z, t, f, f, f, kl=math.inf)
    with pytest.raises(zb.ZgError, match="scale must be finite"):
        zb.policy_loss_grad(z, t, f, f, scale=math.nan)
    with pytest.raises(TypeError, match="old_logp must have dtype"):
        zb.policy_loss(z, t, f.bfloat16(), f)
    with pytest.raises(ValueError, match="advantage must have shape"):
        zb.policy_loss(z, t, f, f[:2])
    with pytest.raises(ValueError, match="kept must have shape"):
        zb.policy_grad(z, f, t, f, f)
    with pytest.raises(zb.ZgError, match="own memory"):
        both = torch.zeros(8, 100, dtype=torch.bfloat16, device="cuda")
        zb.policy_loss_grad(both[::2], t, f, f, out=both[:4])
    with pytest.raises(ValueError, match="out must have shape"):
        zb.policy_loss_grad(z, t, f, f, out=z[:, :50])
