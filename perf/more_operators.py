"""Measured cases of the operators around a trained block and the sharded step:
the token embedding with its gradient, the norms before and after a block with
its gate and residual scale, the clipped policy loss with its gradient, and the
gradient norm over many tensors with clipping into the flat gradient.

``run`` computes a case with elementary torch operations in 32 bits, or, where
``own`` is true, with this package's kernels. ``exact`` gives the same outputs
from the definitions in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
DEV = "cuda"
EPS = 1e-6          # of the norms
CLIP = (0.2, 0.28)  # the policy ratio's bounds below and above one
KL = 0.04
ROOT_WIDTH = 768.0 ** 0.5  # the scale of looked-up rows


# ------------------------------------------------------------------ the cases

def listed() -> list[dict]:
    return [
        # one decoded token for each of 32 requests: latency alone counts
        embed("embed_32x768_bf16", "embed", 32, 50257, 768, "bf16"),
        # a micro-batch of eight GPT-2-small contexts; the whole table's gradient, as the flat vector takes it
        embed("embed_train_8192x768_bf16", "embed_train", 8192, 50257, 768, "bf16"),
        # a table that is the output projection too: its gradient is added to that one's. Odd width, full precision
        embed("embed_train_tied_20011x771_f32", "embed_train", 20011, 50257, 771, "f32", tied=True),
        # one decoded token of 32 requests between two blocks: latency
        norm("norm_32x768_bf16", "norm", 32, 768, "bf16"),
        # a training micro-batch of a wide model, a gate for each of its eight sequences
        norm("norm_train_16384x4096_bf16", "norm_train", 16384, 4096, "bf16", groups=8),
        # ragged, odd width, full precision; the block's output is not normed
        norm("norm_train_9001x771_f32", "norm_train", 9001, 771, "f32", post=False),
        # the behaviour's or the reference policy's log-probabilities of sampled tokens
        policy("logp_1000x50257_bf16", "logp", 1000, 50257, "bf16"),
        # the training step's loss and gradient on four contexts of GPT-2 small, the largest case
        policy("policy_4096x50257_bf16", "policy_train", 4096, 50257, "bf16"),
        # the same on few rows in full precision, without a reference policy
        policy("policy_37x50257_f32", "policy_train", 37, 50257, "f32", ref=False),
        # a multilingual vocabulary, odd and with padded rows; the gradient of a kept forward pass
        policy("policy_two_777x131075_bf16", "policy_two", 777, 131075, "bf16", pad=29),
        # all gradients of a model of GPT-2 small's shape, matrices in bf16 and vectors in binary32, into the
        # flat bf16 gradient that the step takes
        clip("clip_12x768_mixed", 12, 768, 50257, "mixed"),
        # those of a small student: launches
        clip("clip_2x128_f32", 2, 128, 509, "f32"),
    ]


def embed(name, op, tokens, vocab, width, dtype, tied=False) -> dict:
    return {"name": name, "op": op, "tokens": tokens, "vocab": vocab, "width": width, "dtype": dtype, "tied": tied}


def norm(name, op, rows, width, dtype, groups=1, post=True) -> dict:
    return {"name": name, "op": op, "rows": rows, "width": width, "dtype": dtype, "groups": groups, "post": post}


def policy(name, op, rows, vocab, dtype, ref=True, pad=0) -> dict:
    return {"name": name, "op": op, "rows": rows, "vocab": vocab, "dtype": dtype, "ref": ref, "pad": pad}


def clip(name, layers, width, vocab, dtype) -> dict:
    return {"name": name, "op": "clip", "layers": layers, "width": width, "vocab": vocab, "dtype": dtype}


def draw(rng) -> dict:
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    dtype = rng.choice(["bf16", "bf16", "f32"])
    size = SIZE[dtype]
    op = rng.choice(["embed", "embed_train", "norm", "norm_train", "logp", "policy_train", "policy_two", "clip"])
    if op.startswith("embed"):
        width = log(16, 4096)
        vocab = min(log(256, 262144), 200_000_000 // size // width)
        c = embed("", op, min(log(1, 65536), 200_000_000 // size // width), vocab, width, dtype, rng.random() < 0.3)
    elif op.startswith("norm"):
        width = log(16, 8192)
        rows, groups = min(log(1, 65536), 90_000_000 // size // width), rng.choice([1, 1, log(1, 64)])
        c = norm("", op, max(1, rows // groups) * groups, width, dtype, groups, rng.random() < 0.7)
    elif op == "clip":
        c = clip("", log(1, 24), log(32, 1024), log(256, 60000), rng.choice(["bf16", "f32", "mixed"]))
        while sum(math.prod(shape) for shape in shapes(c)) > 100_000_000:
            c["layers"], c["vocab"] = (c["layers"] + 1) // 2, (c["vocab"] + 1) // 2
    else:
        vocab = log(1000, 262144)
        rows = min(log(1, 4096), 400_000_000 // size // vocab)
        c = policy("", op, rows, vocab, dtype, rng.random() < 0.6, rng.choice([0, 0, 1, 31]))
    del c["name"]
    return c


def shapes(case: dict) -> list[tuple]:
    """The tensors of a transformer of this many layers: embeddings, and for each layer the two
    norms, the joint projection of queries, keys and values, the output's, and the two of the MLP."""
    d, out = case["width"], [(case["vocab"], case["width"]), (1024, case["width"])]
    for _ in range(case["layers"]):
        out += [(d,), (d,), (d, 3 * d), (3 * d,), (d, d), (d,), (d,), (d,), (d, 4 * d), (4 * d,), (4 * d, d), (d,)]
    return out + [(d,), (d,)]


def work(case: dict) -> dict:
    op = case["op"]
    if op == "clip":  # every gradient in, the flat one out; the norm and the coefficient
        n, size = 0, 0
        for s in shapes(case):
            n += math.prod(s)
            size += math.prod(s) * tensor_size(case, s)
        return {"bytes": size + (4 if case["dtype"] == "f32" else 2) * n + 8, "flops": 3 * n}
    s = SIZE[case["dtype"]]
    if op.startswith("embed"):
        n, v, d = case["tokens"], case["vocab"], case["width"]
        hit = s * d * v * (1.0 - (1.0 - 1.0 / v) ** n)  # rows of the table that even draws would meet
        look = 8 * n + hit + s * n * d  # tokens and rows in, rows out
        if op == "embed":
            return {"bytes": int(look), "flops": n * d}
        # the rows' gradients in, the table's out (with a tied table's other part in)
        return {"bytes": int(look + s * n * d + (2 if case["tied"] else 1) * s * v * d), "flops": 2 * n * d + v * d}
    n = case["rows"]
    if op.startswith("norm"):
        d, side = case["width"], (1 + case["post"] + case["groups"]) * case["width"] * s
        if op == "norm":  # x, o in; x', n out
            return {"bytes": 4 * s * n * d + side, "flops": 10 * n * d}
        # with dn, dx' in and dx, do out, the weights' gradients
        return {"bytes": 8 * s * n * d + 2 * side, "flops": 36 * n * d}
    v = case["vocab"]
    if op == "logp":  # logits and tokens in; logp and lse out
        return {"bytes": s * n * v + 16 * n, "flops": 4 * n * v}
    # and the old and reference values, advantages, weights in; loss, logp, gradient out
    return {"bytes": 2 * s * n * v + (28 + 4 * case["ref"]) * n, "flops": 8 * n * v}


def tensor_size(case: dict, shape: tuple) -> int:
    return 4 if case["dtype"] == "f32" or (case["dtype"] == "mixed" and len(shape) == 1) else 2


# ------------------------------------------------------------------ inputs

def prepare(case: dict, seed: int) -> dict:
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dt = DTYPES.get(case["dtype"])
    op, s = case["op"], {"case": case}

    def normal(*shape, dtype=dt, scale=1.0, shift=0.0):
        return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32).mul_(scale).add_(shift).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device=DEV)

    if op.startswith("embed"):
        n, v, d = case["tokens"], case["vocab"], case["width"]
        s["table"] = normal(v, d, scale=0.02)
        # words' frequencies fall as one over their rank; ids are dealt out at random, and the
        # last part of a batch is padding
        rank = torch.exp(uniform(n).double() * math.log(v + 1.0)).floor().long().clamp(1, v) - 1
        tokens = torch.randperm(v, generator=gen, device=DEV)[rank]
        if n > 64:
            tokens[n - n // 16:] = -1
        s["tokens"] = tokens
        if op == "embed_train":
            s["drows"] = normal(n, d, scale=1e-3)
            s["other"] = normal(v, d, scale=1e-3) if case["tied"] else None
        return s

    if op.startswith("norm"):
        n, d, groups = case["rows"], case["width"], case["groups"]
        s["x"], s["o"] = normal(n, d, scale=3.0), normal(n, d, scale=0.7)
        s["w_pre"] = normal(d, scale=0.1, shift=1.0)
        s["w_post"] = normal(d, scale=0.1, shift=1.0) if case["post"] else None
        s["gate"] = normal(groups, d, scale=0.3, shift=0.5)
        s["res_scale"] = 0.875
        if op == "norm_train":
            s["dn"], s["dx_new"] = normal(n, d, scale=1e-3), normal(n, d, scale=1e-3)
        return s

    if op == "clip":
        s["grads"] = [normal(*shape, dtype=torch.float32 if tensor_size(case, shape) == 4 else torch.bfloat16, scale=2e-3)
                      for shape in shapes(case)]
        s["flat"] = torch.empty(sum(g.numel() for g in s["grads"]), device=DEV,
                                dtype=torch.float32 if case["dtype"] == "f32" else torch.bfloat16)
        # a loss scale of 1024 is in the gradients
        s["scale"], s["max_norm"] = 1.0 / 1024.0, 1e-4
        if own:
            from zero_sharded_mixed_flat_gb300 import binding
            s["plan"] = binding.GradClip(s["grads"], out=s["flat"])
        return s

    n, v = case["rows"], case["vocab"]
    s["logits"] = normal(n, v + case["pad"], scale=2.5)[:, :v]
    # sampled tokens: of 64 at random, one by its probability
    some = torch.randint(0, v, (n, 64), generator=gen, device=DEV)
    pick = (s["logits"].gather(1, some).float() - torch.log(-torch.log(uniform(n, 64).clamp(1e-9, 1 - 1e-7)))).argmax(1)
    tokens = some.gather(1, pick[:, None])[:, 0]
    s["temperature"] = 1.0
    if op != "logp":
        # the behaviour policy was a little different; no ratio is within 32 bits' error of a bound,
        # where the gradient jumps
        logp = torch.cat([torch.log_softmax(s["logits"][i:i + 256].float(), 1).gather(1, tokens[i:i + 256, None])[:, 0]
                          for i in range(0, n, 256)])
        moved = normal(n, dtype=torch.float32, scale=0.2)
        for bound in (math.log(1.0 - CLIP[0]), math.log(1.0 + CLIP[1])):
            moved = torch.where((moved - bound).abs() < 2e-3, moved + 5e-3, moved)
        s["old_logp"] = logp - moved
        s["ref_logp"] = logp + normal(n, dtype=torch.float32, scale=0.3) if case["ref"] else None
        s["advantage"] = normal(n, dtype=torch.float32)
        s["dloss"] = uniform(n).add_(0.5)
        s["scale"] = 1024.0 / n  # the loss scale over the rows
    tokens[torch.arange(n, device=DEV) % 16 == 15] = -1  # padding rows
    s["tokens"] = tokens
    return s


# ------------------------------------------------------------------ the package's calls and the plain forms

def run(state: dict):
    return (_run_own if own else _run_plain)(state)


def _run_own(s: dict):
    from zero_sharded_mixed_flat_gb300 import binding as zb

    case = s["case"]
    op = case["op"]
    if op.startswith("embed"):
        out = {"rows": zb.embed(s["table"], s["tokens"], ROOT_WIDTH)}
        if op == "embed_train":
            out["dtable"] = zb.embed_grad(s["drows"], s["tokens"], case["vocab"], ROOT_WIDTH, add=s["other"])
        return out
    if op.startswith("norm"):
        block = (s["w_pre"], s["o"], s["w_post"], s["gate"], s["res_scale"], EPS)
        if op == "norm":
            x_new, n, _ = zb.block_norm(s["x"], *block)
            return {"x_new": x_new, "n": n}
        x_new, n, kept = zb.block_norm(s["x"], *block, keep=True)
        dx, do, dw_pre, dw_post, dgate = zb.block_norm_grad(s["x"], kept, s["dn"], s["dx_new"], *block)
        return {"x_new": x_new, "n": n, "dx": dx, "do": do, "dw_pre": dw_pre, "dw_post": dw_post, "dgate": dgate}
    if op == "clip":
        return {"stats": s["plan"].clip(s["max_norm"], EPS, s["scale"]), "flat": s["flat"]}
    if op == "logp":
        logp, lse = zb.token_logp(s["logits"], s["tokens"], s["temperature"])
        return {"logp": logp, "lse": lse}
    how = (s["tokens"], s["old_logp"], s["advantage"], s["ref_logp"], CLIP, KL, s["temperature"])
    if op == "policy_two":
        loss, logp, kept = zb.policy_loss(s["logits"], *how)
        grad = zb.policy_grad(s["logits"], kept, *how, s["scale"], s["dloss"])
    else:
        loss, logp, grad = zb.policy_loss_grad(s["logits"], *how, s["scale"], s["dloss"])
    return {"loss": loss, "logp": logp, "grad": grad}


def _run_plain(s: dict):
    op = s["case"]["op"]
    if op.startswith("embed"):
        return _plain_embed(s)
    if op.startswith("norm"):
        return _plain_norm(s)
    return _plain_clip(s) if op == "clip" else _plain_policy(s)


def _plain_embed(s: dict):
    table, tokens = s["table"], s["tokens"]
    there = (tokens >= 0) & (tokens < table.shape[0])
    at = torch.where(there, tokens, 0)
    out = {"rows": torch.where(there[:, None], table[at].float() * ROOT_WIDTH, 0.0).to(table.dtype)}
    if s["case"]["op"] == "embed":
        return out
    d = torch.where(there[:, None], s["drows"].float() * ROOT_WIDTH, 0.0)
    sums = torch.zeros(table.shape, device=table.device).index_add_(0, at, d)
    if s["other"] is not None:
        sums += s["other"].float()
    return {**out, "dtable": sums.to(table.dtype)}


def _plain_norm(s: dict):
    dt, groups, r = s["x"].dtype, s["case"]["groups"], s["res_scale"]
    x, o, w2 = s["x"].float(), s["o"].float(), s["w_pre"].float()
    n, d = x.shape
    g = s["gate"].float().repeat_interleave(n // groups, 0)
    post = s["w_post"] is not None
    if post:
        w1 = s["w_post"].float()
        s1 = 1.0 / torch.sqrt((o * o).mean(1, keepdim=True) + EPS)
        oh = o * s1
        b = oh * w1
    else:
        b = o
    xn = r * x + g * b
    s2 = 1.0 / torch.sqrt((xn * xn).mean(1, keepdim=True) + EPS)
    xh = xn * s2
    out = {"x_new": xn.to(dt), "n": (xh * w2).to(dt)}
    if s["case"]["op"] == "norm":
        return out
    dn = s["dn"].float()
    dxh = dn * w2
    dxn = s["dx_new"].float() + s2 * (dxh - xh * (dxh * xh).mean(1, keepdim=True))
    db = g * dxn
    out["dx"] = (r * dxn).to(dt)
    if post:
        doh = db * w1
        out["do"] = (s1 * (doh - oh * (doh * oh).mean(1, keepdim=True))).to(dt)
    else:
        out["do"] = db.to(dt)
    out["dw_pre"] = (dn * xh).sum(0).to(dt)
    out["dw_post"] = (db * oh).sum(0).to(dt) if post else None
    out["dgate"] = (dxn * b).view(groups, n // groups, d).sum(1).to(dt)
    return out


def _plain_clip(s: dict):
    total = sum((g.float() * s["scale"]).square().sum() for g in s["grads"])
    norm = torch.sqrt(total)
    coef = torch.clamp(s["max_norm"] / (norm + EPS), max=1.0)
    coef = torch.where(torch.isfinite(norm), coef, 1.0)
    return {"stats": torch.stack([norm, coef]),
            "flat": torch.cat([(g.float() * s["scale"] * coef).to(s["flat"].dtype).view(-1) for g in s["grads"]])}


def _plain_policy(s: dict):
    tau = s["temperature"]
    z = s["logits"].float() / tau
    there = s["tokens"] >= 0
    at = s["tokens"].clamp(min=0)
    zmax = z.max(1, keepdim=True).values
    lse = zmax + torch.log(torch.exp(z - zmax).sum(1, keepdim=True))
    logp = (z.gather(1, at[:, None]) - lse)[:, 0]
    if s["case"]["op"] == "logp":
        return {"logp": torch.where(there, logp, 0.0), "lse": torch.where(there, lse[:, 0], 0.0)}
    a = s["advantage"]
    ratio = torch.exp(logp - s["old_logp"])
    loss = -torch.minimum(ratio * a, ratio.clamp(1.0 - CLIP[0], 1.0 + CLIP[1]) * a)
    cut = ((a > 0) & (ratio > 1.0 + CLIP[1])) | ((a < 0) & (ratio < 1.0 - CLIP[0]))
    slope = torch.where(cut, 0.0, -ratio * a)
    if s["ref_logp"] is not None:
        d = s["ref_logp"] - logp
        loss = loss + KL * (torch.expm1(d) - d)
        slope = slope - KL * torch.expm1(d)
    slope = torch.where(there, s["scale"] * s["dloss"] * slope / tau, 0.0)[:, None]
    grad = (torch.exp(z - lse) * -slope).scatter_add_(1, at[:, None], slope)
    return {"loss": torch.where(there, loss, 0.0), "logp": torch.where(there, logp, 0.0), "grad": grad.to(s["logits"].dtype)}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case: dict, seed: int):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("embed"):
        return _exact_embed(s)
    if op.startswith("norm"):
        return _exact_norm(s)
    return _exact_clip(s) if op == "clip" else _exact_policy(s)


def _exact_embed(s: dict):
    v, d = s["table"].shape
    tokens = s["tokens"]
    keep = torch.nonzero((tokens >= 0) & (tokens < v))[:, 0]
    rows = torch.zeros(tokens.numel(), d, dtype=torch.float64, device=DEV)
    rows[keep] = s["table"].double()[tokens[keep]] * ROOT_WIDTH
    if s["case"]["op"] == "embed":
        return {"rows": rows}
    total = torch.zeros(v, d, dtype=torch.float64, device=DEV) if s["other"] is None else s["other"].double()
    total.index_put_((tokens[keep],), s["drows"].double()[keep] * ROOT_WIDTH, accumulate=True)
    return {"rows": rows, "dtable": total}


def _exact_norm(s: dict):
    """The gradients by automatic differentiation of the forward pass, some rows at a time."""
    train, groups = s["case"]["op"] == "norm_train", s["case"]["groups"]
    n, each = s["x"].shape[0], s["x"].shape[0] // groups
    w2 = s["w_pre"].double().requires_grad_(train)
    w1 = None if s["w_post"] is None else s["w_post"].double().requires_grad_(train)
    gate = s["gate"].double().requires_grad_(train)
    parts = {k: [] for k in (["x_new", "n", "dx", "do"] if train else ["x_new", "n"])}
    for lo in range(0, n, 2048):
        cut = slice(lo, min(n, lo + 2048))
        x, o = (s[k][cut].double().requires_grad_(train) for k in ("x", "o"))
        with torch.set_grad_enabled(train):
            b = o if w1 is None else o * torch.rsqrt(o.pow(2).mean(1, keepdim=True) + EPS) * w1
            at = torch.arange(cut.start, cut.stop, device=DEV) // each
            y = s["res_scale"] * x + gate[at] * b
            m = y * torch.rsqrt(y.pow(2).mean(1, keepdim=True) + EPS) * w2
            if train:
                ((y * s["dx_new"][cut].double()).sum() + (m * s["dn"][cut].double()).sum()).backward()
        for k, value in zip(parts, (y.detach(), m.detach(), x.grad, o.grad)):
            parts[k].append(value)
    out = {k: torch.cat(p) for k, p in parts.items()}
    if train:
        out.update(dw_pre=w2.grad, dw_post=None if w1 is None else w1.grad, dgate=gate.grad)
    return out


def _exact_clip(s: dict):
    norm = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(g.double()) for g in s["grads"]])) * s["scale"]
    coef = (s["max_norm"] / (norm + EPS)).clamp(max=1.0)
    return {"stats": torch.stack([norm, coef]), "flat": torch.cat([g.double().view(-1) * (s["scale"] * coef) for g in s["grads"]])}


def _exact_policy(s: dict):
    tau, op = s["temperature"], s["case"]["op"]
    out = {}
    for i in range(0, s["logits"].shape[0], 256):
        cut = slice(i, i + 256)
        z = s["logits"][cut].double() / tau
        tokens = s["tokens"][cut]
        there = tokens >= 0
        lse = torch.logsumexp(z, 1)
        logp = z[torch.arange(len(tokens), device=DEV), tokens.clamp(min=0)] - lse
        if op == "logp":
            part = {"logp": logp * there, "lse": lse * there}
        else:
            a = s["advantage"][cut].double()
            ratio = torch.exp(logp - s["old_logp"][cut].double())
            high, low = ratio > 1.0 + CLIP[1], ratio < 1.0 - CLIP[0]
            held = torch.where(high, 1.0 + CLIP[1], torch.where(low, 1.0 - CLIP[0], ratio))
            loss = torch.maximum(-ratio * a, -held * a)
            slope = torch.where((high & (a > 0)) | (low & (a < 0)), 0.0, -ratio * a)
            if s["ref_logp"] is not None:
                d = s["ref_logp"][cut].double() - logp
                loss = loss + KL * (torch.exp(d) - d - 1.0)
                slope = slope + KL * (1.0 - torch.exp(d))
            slope = slope * s["dloss"][cut].double() * s["scale"] / tau * there
            grad = torch.exp(z - lse[:, None]) * -slope[:, None]
            grad[torch.arange(len(tokens), device=DEV), tokens.clamp(min=0)] += slope
            part = {"loss": loss * there, "logp": logp * there, "grad": grad}
        for k, value in part.items():
            out.setdefault(k, []).append(value)
    return {k: torch.cat(p) for k, p in out.items()}
