"""The operators around a block, the recurrence and the sharded step together, as the example runs them."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_it_runs():
    import policy_recurrent_blocks as ex

    history = ex.train(steps=3, ranks=2, batch=5, tokens=9, vocab=37, width=24)
    assert len(history) == 3 and all(0.0 <= h <= 1.0 for h in history)


def test_its_gradient_is_that_of_plain_autograd():
    """The whole model's gradient against automatic differentiation of the same model in 64 bits. On the way from
    the parameters to a gradient some 26 values are stored in bf16, one after the other (rows, 5 a block, logits; dlogits, 5 a
    block, the sums, the clipped ones), each off by 2^-8 of its size at most."""
    import policy_recurrent_blocks as ex

    gen = torch.Generator(device="cuda").manual_seed(4)
    lay = ex.Layout(53, 24, 2)
    flat = lay.initial(gen).bfloat16()
    for t, s in zip(lay.tensors(flat), lay.shapes):
        if len(s) == 1:
            t.add_(torch.randn(s, generator=gen, device="cuda").bfloat16() * 0.1)
    batch, steps = 3, 20
    rank = ex.Rank(lay, batch, steps)
    tokens = torch.randint(0, 53, (batch, steps), generator=gen, device="cuda")
    targets = torch.randint(0, 53, (batch, steps), generator=gen, device="cuda")
    targets[0, -4:] = -1  # padding
    adv = torch.randn(batch, steps, generator=gen, device="cuda")

    w = flat.double().requires_grad_()
    table, norm, *rest = lay.tensors(w)
    rms = lambda t: t * torch.rsqrt(t.pow(2).mean(-1, keepdim=True) + 1e-6)  # noqa: E731
    x = table[tokens] * lay.scale
    n = rms(x) * norm
    for into, out, post, gate, pre in zip(*[iter(rest)] * 5):
        u = n @ into
        a, h, ys = torch.sigmoid(u[..., 24:] + 2.0), 0.0, []
        for s in range(steps):
            h = a[:, s] * h + (1 - a[:, s]) * u[:, s, :24]
            ys.append(h)
        x = ex.RESIDUAL * x + gate * (rms(torch.stack(ys, 1) @ out) * post)
        n = rms(x) * pre
    logp = torch.log_softmax(n @ table.t(), -1).gather(-1, targets.clamp(min=0)[..., None])[..., 0]
    # ratios well inside the bounds, and some far outside
    moved = torch.where(torch.arange(steps, device="cuda") % 5 == 4, 0.9, 0.02)
    old, refl = (logp.detach() - moved).float(), (logp.detach() + 0.2).float()
    ratio, d = torch.exp(logp - old), refl - logp
    loss = -torch.minimum(ratio * adv, ratio.clamp(1 - ex.CLIP[0], 1 + ex.CLIP[1]) * adv) + ex.KL * (torch.exp(d) - 1 - d)
    loss = loss * (targets >= 0)
    (loss.mean() * 512.0).backward()

    got, stats = ex.gradient(lay, flat, rank, tokens, targets, old, adv, refl, 512.0, 1e9)
    bound = 26 * 2.0 ** -8
    assert float((got.view(batch, steps).double() - loss.detach()).abs().max()) <= bound * float(loss.detach().abs().max())
    want = float(w.grad.norm())
    assert float((rank.flat.double() - w.grad).norm()) <= bound * want
    assert float(stats[1]) == 1.0 and abs(float(stats[0]) - want) <= bound * want
    # clipped to half of that, the same direction
    _, stats = ex.gradient(lay, flat, rank, tokens, targets, old, adv, refl, 512.0, 0.5 * want / 512.0)
    assert abs(float(stats[1]) - 0.5) <= bound
    assert abs(float(rank.flat.double().norm()) - 0.5 * want) <= bound * want
