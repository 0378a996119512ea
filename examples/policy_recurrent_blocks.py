"""A recurrent policy learns from rewards of its own samples, by sharded steps.

The policy is a token embedding, blocks of a gated linear recurrence between two
projections, each with a norm before and after it, a gate and a scaled residual, a
last norm, and the embedding again as the output's projection. It samples tokens one
at a time (the recurrence's and the norms' single-token forms), is paid for every
token that is the last one's successor, and takes the clipped policy loss, with a KL
term to where it began, of what it sampled. The gradients of all tensors are clipped
by their common norm into the rank's flat bf16 gradient, and one step reduces and
applies the P ranks' gradients. That clips each rank by itself, so that no rank's
samples outweigh the others'; the clipping by the norm of the reduced gradient is the
step's own, which follows (`Hparams.max_grad_norm`).

    python examples/policy_recurrent_blocks.py [--steps 30]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from zero_sharded_mixed_flat_gb300 import binding as zb  # noqa: E402

RESIDUAL, CLIP, KL = 0.9, (0.2, 0.28), 0.02


class Layout:
    """Where a policy of this size keeps its tensors in the flat vector."""

    def __init__(self, vocab: int, width: int, blocks: int):
        self.vocab, self.width, self.blocks = vocab, width, blocks
        d = width
        # the embedding, the first norm, and for each block: into, out of, norm after, gate, norm before the next
        self.shapes = [(vocab, d), (d,)] + blocks * [(d, 2 * d), (d, d), (d,), (d,), (d,)]
        self.sizes = [torch.Size(s).numel() for s in self.shapes]
        self.n = sum(self.sizes)
        self.scale = d ** 0.5  # of looked-up rows

    def tensors(self, flat: torch.Tensor) -> list[torch.Tensor]:
        return [p.view(s) for p, s in zip(flat[:self.n].split(self.sizes), self.shapes)]

    def initial(self, gen) -> torch.Tensor:
        flat = torch.randn(self.n, generator=gen, device="cuda")
        for t, s in zip(self.tensors(flat), self.shapes):
            if len(s) == 1:
                t.fill_(1.0)
            else:
                t.mul_(self.width ** -0.5)
        return flat


class Rank:
    """One rank's handles, gradients and flat gradient."""

    def __init__(self, layout: Layout, batch: int, tokens: int):
        self.scans = [zb.GatedScan(batch, tokens, layout.width) for _ in range(layout.blocks)]
        self.grads = [torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in layout.shapes]
        self.flat = torch.zeros(layout.n, dtype=torch.bfloat16, device="cuda")
        self.clip = zb.GradClip(self.grads, out=self.flat)


def sample(layout, flat, scans, first, steps, gen):
    """Tokens (batch, steps + 1) from ``first`` on, one at a time, and the samples' log-probabilities."""
    table, norm, *rest = layout.tensors(flat)
    batch = first.shape[0]
    states = [torch.zeros(batch, layout.width, device="cuda") for _ in range(layout.blocks)]
    tokens, logps = [first], []
    for _ in range(steps):
        x = zb.embed(table, tokens[-1], layout.scale)
        _, n, _ = zb.block_norm(x, norm)
        for i, (into, out, post, gate, pre) in enumerate(zip(*[iter(rest)] * 5)):
            u = n @ into
            a, f = u[:, :layout.width], u[:, layout.width:].add_(2.0)
            y, states[i] = scans[i].step(a, f, states[i], out_state=states[i])
            x, n, _ = zb.block_norm(x, pre, y @ out, post, gate, RESIDUAL)
        logits = n @ table.t()
        noise = -torch.log(-torch.log(torch.rand(logits.shape, generator=gen, device="cuda").clamp_(1e-9, 1 - 1e-7)))
        tokens.append((logits.float() + noise).argmax(1))
        logps.append(zb.token_logp(logits, tokens[-1])[0])
    return torch.stack(tokens, 1), torch.stack(logps, 1)


def forward(layout, flat, tokens, scans, keep=False):
    """The logits after every token, and what the backward pass needs."""
    table, norm, *rest = layout.tensors(flat)
    x = zb.embed(table, tokens, layout.scale)
    _, n, kept = zb.block_norm(x, norm, keep=keep)
    saved = [(x, kept)]
    for scan, (into, out, post, gate, pre) in zip(scans, zip(*[iter(rest)] * 5)):
        u = n @ into
        a, f = u[..., :layout.width], u[..., layout.width:]
        f.add_(2.0)  # memories of several tokens to begin with
        y, _, states = scan.forward(a, f, keep=keep)
        o = y @ out
        x_new, n_new, kept = zb.block_norm(x, pre, o, post, gate, RESIDUAL, keep=keep)
        saved.append((x, n, a, f, states, y, o, kept))
        x, n = x_new, n_new
    return (n @ table.t()).view(-1, layout.vocab), n, saved


def gradient(layout, flat, rank, tokens, targets, old_logp, advantage, ref_logp, loss_scale, max_norm):
    """The loss of every target token, and the clipped gradient of their mean times ``loss_scale`` in ``rank.flat``."""
    table, norm, *rest = layout.tensors(flat)
    d_table, d_norm, *d_rest = rank.grads
    logits, n, saved = forward(layout, flat, tokens, rank.scans, keep=True)
    rows, d = logits.shape[0], layout.width
    loss, _, dlogits = zb.policy_loss_grad(logits, targets.reshape(-1), old_logp.reshape(-1), advantage.reshape(-1),
                                           ref_logp.reshape(-1), CLIP, KL, scale=loss_scale / rows, out=logits)
    torch.mm(dlogits.t(), n.view(rows, d), out=d_table)
    dn, dx = (dlogits @ table).view_as(n), None
    for i in reversed(range(layout.blocks)):
        into, out, post, gate, pre = rest[5 * i:5 * i + 5]
        d_into, d_out, d_post, d_gate, d_pre = d_rest[5 * i:5 * i + 5]
        x, n_in, a, f, states, y, o, kept = saved[i + 1]
        dx, do, w_pre, w_post, w_gate = zb.block_norm_grad(x, kept, dn, dx, pre, o, post, gate, RESIDUAL)
        for to, got in ((d_pre, w_pre), (d_post, w_post), (d_gate, w_gate)):
            to.copy_(got)
        torch.mm(y.view(rows, d).t(), do.view(rows, d), out=d_out)
        dy = do @ out.t()
        du = torch.empty(*y.shape[:2], 2 * d, dtype=y.dtype, device=y.device)
        rank.scans[i].backward(a, f, dy, states, out=(du[..., :d], du[..., d:]))
        torch.mm(n_in.view(rows, d).t(), du.view(rows, 2 * d), out=d_into)
        dn = du @ into.t()
    x, kept = saved[0]
    dx, _, w_norm, _, _ = zb.block_norm_grad(x, kept, dn, dx, norm)
    d_norm.copy_(w_norm)
    # the table is the output's projection too: the lookups' part is added to that one's
    zb.embed_grad(dx, tokens, layout.vocab, layout.scale, add=d_table, out=d_table)
    stats = rank.clip.clip(max_norm * loss_scale)
    return loss, stats


def train(steps: int = 30, ranks: int = 2, batch: int = 16, tokens: int = 32, vocab: int = 61, width: int = 64, blocks: int = 2,
          loss_scale: float = 1024.0, max_norm: float = 1.0, seed: int = 0, report=None) -> list[float]:
    """The mean reward of every step."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    layout = Layout(vocab, width, blocks)
    w0 = layout.initial(gen)
    reference = w0.bfloat16()
    opt = zb.ShardedAdamW(layout.n, ranks, zb.Hparams(lr=1e-2, weight_decay=0.0), w0)
    all_ranks = [Rank(layout, batch, tokens) for _ in range(ranks)]
    history = []
    for step in range(steps):
        rewards = []
        for rank in all_ranks:
            first = torch.randint(0, vocab, (batch,), generator=gen, device="cuda")
            seen, logp = sample(layout, opt.params, rank.scans, first, tokens, gen)
            reward = (seen[:, 1:] == (seen[:, :-1] + 1) % vocab).float()
            inputs, targets = seen[:, :-1].contiguous(), seen[:, 1:].contiguous()
            ref_logits = forward(layout, reference, inputs, rank.scans)[0]
            ref_logp = zb.token_logp(ref_logits, targets.view(-1))[0]
            gradient(layout, opt.params, rank, inputs, targets, logp, reward - reward.mean(), ref_logp, loss_scale, max_norm)
            rewards.append(reward.mean())
        opt.step([rank.flat for rank in all_ranks], loss_scale)
        history.append(float(torch.stack(rewards).mean()))
        if report and (step % 5 == 0 or step == steps - 1):
            info = opt.info()
            report(f"step {step:3d}  reward {history[-1]:.4f}  gradient norm {info.norm:.3f}  applied {info.step_t}")
    return history


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=30)
    train(ap.parse_args().steps, report=print)
