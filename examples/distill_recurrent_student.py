"""A recurrent student learns from a teacher's top logits, by sharded steps.

The student is an embedding, one gated linear recurrence whose candidate and
gate are the halves of one projection, and an output projection: one flat bf16
parameter vector. Each of P ranks runs a micro-batch of its own: the teacher's
top logits are selected, the student's logits turned into a loss and, in the
same pass, into their gradient times the loss scale, which goes back through
the projections (library products) and the recurrence into the rank's flat
bf16 gradient. One step then reduces, clips and applies the P gradients.

    python examples/distill_recurrent_student.py [--steps 60]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from zero_sharded_mixed_flat_gb300 import binding as zb  # noqa: E402

TEMPERATURE = 2.0


class Layout:
    """Where a student of this size keeps its matrices in the flat vector."""

    def __init__(self, vocab: int, width: int):
        self.vocab, self.width = vocab, width
        self.shapes = [(vocab, width), (width, 2 * width), (width, vocab)]
        self.n = sum(a * b for a, b in self.shapes)

    def matrices(self, flat: torch.Tensor) -> list[torch.Tensor]:
        parts = flat[:self.n].split([a * b for a, b in self.shapes])
        return [p.view(s) for p, s in zip(parts, self.shapes)]


def logits_of(layout: Layout, flat: torch.Tensor, tokens: torch.Tensor, scan: zb.GatedScan, keep: bool = False):
    """The logits of every token, and what the backward pass needs."""
    embed, into, out = layout.matrices(flat)
    e = embed[tokens]
    u = e @ into
    x, f = u[..., :layout.width], u[..., layout.width:]
    f.add_(2.0)  # memories of several tokens to begin with
    y, _, kept = scan.forward(x, f, keep=keep)
    return (y @ out).view(-1, layout.vocab), (e, x, f, y, kept)


def rank_gradient(layout, flat, tokens, scan, teacher, loss_scale, grad) -> torch.Tensor:
    """One rank's loss per token, and its gradient times loss_scale into ``grad``."""
    embed, into, out = layout.matrices(flat)
    logits, (e, x, f, y, kept) = logits_of(layout, flat, tokens, scan, keep=True)
    rows = logits.shape[0]
    loss, dlogits = zb.distill_loss_grad(logits, *teacher, TEMPERATURE, loss_scale / rows, out=logits)
    d_embed, d_into, d_out = layout.matrices(grad)
    y2, e2 = y.view(rows, -1), e.view(rows, -1)
    torch.mm(y2.t(), dlogits, out=d_out)
    dy = (dlogits @ out.t()).view_as(y)
    du = torch.empty(*y.shape[:2], 2 * layout.width, dtype=y.dtype, device=y.device)
    scan.backward(x, f, dy, kept, out=(du[..., :layout.width], du[..., layout.width:]))
    du2 = du.view(rows, -1)
    torch.mm(e2.t(), du2, out=d_into)
    sums = torch.zeros(layout.shapes[0], device=grad.device).index_add_(0, tokens.view(-1), (du2 @ into.t()).float())
    d_embed.copy_(sums)
    return loss


def train(steps: int = 60, ranks: int = 4, batch: int = 4, tokens: int = 256, vocab: int = 509, width: int = 128,
          top: int = 32, loss_scale: float = 1024.0, seed: int = 0, report=None) -> list[float]:
    """The mean loss of every step."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def weights(layout):
        w = torch.randn(layout.n, generator=gen, device="cuda")
        for m in layout.matrices(w):
            m.mul_(m.shape[0] ** -0.5 if m.shape[0] != vocab else 1.0)
        return w

    student, master = Layout(vocab, width), Layout(vocab, 2 * width)
    teacher_flat = weights(master)
    master.matrices(teacher_flat)[2].mul_(6.0)  # a teacher that is sure of something
    teacher_flat = teacher_flat.bfloat16()
    opt = zb.ShardedAdamW(student.n, ranks, zb.Hparams(lr=5e-3, weight_decay=0.0), weights(student))
    scan, teacher_scan = zb.GatedScan(batch, tokens, width), zb.GatedScan(batch, tokens, 2 * width)
    grads = [torch.empty(student.n, dtype=torch.bfloat16, device="cuda") for _ in range(ranks)]
    data = torch.randint(0, vocab, (ranks, batch, tokens), generator=gen, device="cuda")
    history = []
    for step in range(steps):
        losses = []
        for r in range(ranks):
            values, index = zb.topk_logits(logits_of(master, teacher_flat, data[r], teacher_scan)[0], top)
            losses.append(rank_gradient(student, opt.params, data[r], scan, (values, index), loss_scale, grads[r])
                          .mean())
        opt.step(grads, loss_scale)
        history.append(float(torch.stack(losses).mean()))
        if report and (step % 10 == 0 or step == steps - 1):
            info = opt.info()
            report(f"step {step:3d}  loss {history[-1]:.4f}  gradient norm {info.norm:.3f}  applied {info.step_t}")
    return history


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    train(ap.parse_args().steps, report=print)
