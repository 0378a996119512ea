"""The operators and the sharded step together, as the example runs them."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_the_student_learns():
    import distill_recurrent_student as ex

    history = ex.train(steps=40)
    assert all(h == h for h in history)
    assert history[-1] < 0.5 * history[0], (history[0], history[-1])


def test_the_example_gradient_is_that_of_plain_autograd():
    """The whole model's gradient against automatic differentiation of the same
    model in 64 bits (bf16 activations in between: a few hundredths of the norm)."""
    import distill_recurrent_student as ex
    from zero_sharded_mixed_flat_gb300 import binding as zb

    torch.manual_seed(3)
    lay = ex.Layout(61, 16)
    flat = (torch.randn(lay.n, device="cuda") * 0.3).bfloat16()
    tokens = torch.randint(0, 61, (2, 40), device="cuda")
    scan = zb.GatedScan(2, 40, 16)
    t, i = zb.topk_logits(torch.randn(80, 61, device="cuda") * 3, 7)
    grad = torch.empty(lay.n, dtype=torch.bfloat16, device="cuda")
    loss = ex.rank_gradient(lay, flat, tokens, scan, (t, i), 512.0, grad)
    w = flat.double().requires_grad_()
    embed, into, out = lay.matrices(w)
    u = embed[tokens] @ into
    x, a = u[..., :16], torch.sigmoid(u[..., 16:] + 2.0)
    h, ys = torch.zeros(2, 16, dtype=torch.float64, device="cuda"), []
    for s in range(40):
        h = a[:, s] * h + (1 - a[:, s]) * x[:, s]
        ys.append(h)
    z = (torch.stack(ys, 1) @ out).view(80, 61)
    p = torch.softmax(t.double() / ex.TEMPERATURE, 1)
    logq = torch.log_softmax(z / ex.TEMPERATURE, 1).gather(1, i.long())
    want = ex.TEMPERATURE ** 2 * (p * (p.log() - logq)).sum(1)
    (want.mean() * 512.0).backward()
    # every stage stores bf16 (2^-8 of a value): a dozen of them in a row
    assert float((loss.double() - want).abs().max()) <= 12 * 2.0 ** -8 * float(want.abs().max())
    assert float((grad.double() - w.grad).norm()) <= 12 * 2.0 ** -8 * float(w.grad.norm())
