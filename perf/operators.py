"""Measured cases of the training operators: the gated linear recurrence, the
selection of a teacher's top logits, and the distillation loss with its
gradient.

``run`` computes a case with elementary torch operations in 32 bits, or, where
``own`` is true, with this package's kernels. ``exact`` gives the same outputs
from the definitions in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda"


# ------------------------------------------------------------------ the cases

def listed() -> list[dict]:
    return [
        # one decoded token for each of 32 requests through a layer as wide as GPT-2 small: latency alone counts
        scan("step_32x768_bf16", "scan_step", 32, 1, 768, "bf16"),
        # a prefill of eight prompts of GPT-2 small's context length
        scan("scan_8x1024x768_bf16", "scan", 8, 1024, 768, "bf16"),
        # one long document, where only the time axis has work to spread over the GPU
        scan("scan_1x65536x768_bf16", "scan", 1, 65536, 768, "bf16"),
        # a training micro-batch; candidate and gate are the halves of one projection's output
        scan("train_8x4096x1536_bf16", "scan_train", 8, 4096, 1536, "bf16", fused=True),
        # ragged documents packed end to end, odd width, full precision
        scan("train_packed_9001x771_f32", "scan_train", 1, 9001, 771, "f32", seqs=13),
        # top logits of a teacher for a micro-batch of four GPT-2-small contexts
        rows("topk_4096x50257_k64_bf16", "topk", 4096, 50257, 64, "bf16"),
        # a few generated tokens' teacher logits in full precision: few rows, latency
        rows("topk_7x50257_k100_f32", "topk", 7, 50257, 100, "f32"),
        # evaluation of a student: the loss alone, on a ragged number of rows
        rows("loss_1000x50257_k50_bf16", "distill_loss", 1000, 50257, 50, "bf16"),
        # the training step's loss and gradient on four contexts of GPT-2 small, the largest case
        rows("distill_4096x50257_k64_bf16", "distill_train", 4096, 50257, 64, "bf16"),
        # the same on few rows in full precision (a short fine-tuning sample)
        rows("distill_37x50257_k20_f32", "distill_train", 37, 50257, 20, "f32"),
        # a multilingual vocabulary whose rows are larger than one SM's shared memory
        rows("distill_777x131075_k32_bf16", "distill_train", 777, 131075, 32, "bf16"),
        # gradient of a kept forward pass, on logits stored with padded rows
        rows("loss_grad_2048x50257_pad_bf16", "distill_two", 2048, 50257, 64, "bf16", pad=47),
    ]


def scan(name, op, batch, tokens, channels, dtype, fused=False, seqs=0) -> dict:
    return {"name": name, "op": op, "batch": batch, "tokens": tokens, "channels": channels, "dtype": dtype,
            "fused": fused, "seqs": seqs}


def rows(name, op, n, vocab, k, dtype, pad=0) -> dict:
    return {"name": name, "op": op, "rows": n, "vocab": vocab, "k": k, "dtype": dtype, "pad": pad}


def draw(rng) -> dict:
    def log(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    dtype = rng.choice(["bf16", "bf16", "f32"])
    size = 2 if dtype == "bf16" else 4
    op = rng.choice(["scan_step", "scan", "scan_train", "topk", "distill_loss", "distill_train", "distill_two"])
    if op.startswith("scan"):
        channels = log(64, 4096)
        if op == "scan_step":
            c = scan("", op, log(1, 512), 1, channels, dtype)
        else:
            tokens = log(2, 65536)
            most = max(1, 90_000_000 // size // (tokens * channels))
            seqs = rng.choice([0, 0, log(1, 64)])
            c = scan("", op, 1 if seqs else min(most, log(1, 64)), tokens, channels, dtype, rng.random() < 0.5, seqs)
            if tokens * channels * size > 100_000_000:
                c["tokens"] = 100_000_000 // size // channels
    else:
        vocab = log(1000, 262144)
        n = min(log(1, 4096), 400_000_000 // size // vocab)
        c = rows("", op, n, vocab, log(1, 256), dtype, rng.choice([0, 0, 1, 31]))
    del c["name"]
    return c


def work(case: dict) -> dict:
    s = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("scan"):
        elems = case["batch"] * case["tokens"] * case["channels"]
        state = 4 * (case["seqs"] or case["batch"]) * case["channels"]
        if case["op"] == "scan_train":  # x, f, dy, h0, dh_last in; y, h_last, dx, df, dh0 out
            return {"bytes": 6 * s * elems + 5 * state, "flops": 20 * elems}
        return {"bytes": 3 * s * elems + 2 * state, "flops": 8 * elems}  # x, f, h0 in; y, h_last out
    n, v, k = case["rows"], case["vocab"], case["k"]
    if case["op"] == "topk":  # logits in; values and int32 indices out
        return {"bytes": s * n * v + (s + 4) * n * k, "flops": n * v}
    entries = (s + 4) * n * k
    if case["op"] == "distill_loss":  # logits and entries in; loss and lse out
        return {"bytes": s * n * v + entries + 8 * n, "flops": 4 * n * v}
    return {"bytes": 2 * s * n * v + entries + 12 * n, "flops": 8 * n * v}  # and the gradient out, dloss in


# ------------------------------------------------------------------ inputs

def prepare(case: dict, seed: int) -> dict:
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, dtype=dt, scale=1.0, shift=0.0):
        return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32).mul_(scale).add_(shift).to(dtype)

    s = {"case": case}
    if case["op"].startswith("scan"):
        b, t, c, seqs = case["batch"], case["tokens"], case["channels"], case["seqs"]
        if case["fused"]:  # one projection's output, cut in two
            both = normal(b, t, 2 * c)
            s["x"], s["f"] = both[..., :c], both[..., c:]
            s["f"].add_(2.0)
        else:
            s["x"], s["f"] = normal(b, t, c), normal(b, t, c, scale=1.5, shift=2.0)  # memories of a few to hundreds of tokens
        if case["op"] == "scan_step":
            s["x"], s["f"] = s["x"][:, 0], s["f"][:, 0]
        s["seq_start"] = None
        if seqs:  # documents end to end, among them empty ones where two cuts fall together
            cuts = torch.randint(0, t + 1, (seqs - 1,), generator=gen, device=DEV).sort().values
            s["seq_start"] = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), t)])
            s["x"], s["f"] = s["x"][0], s["f"][0]
        s["h0"] = normal(seqs or b, c, dtype=torch.float32)
        if case["op"] == "scan_train":
            s["dy"] = normal(*s["x"].shape, scale=1e-3)
            s["dh_last"] = normal(seqs or b, c, dtype=torch.float32, scale=1e-3)
        if own:
            from zero_sharded_mixed_flat_gb300 import binding
            s["scan"] = binding.GatedScan(b, t, c)
        return s

    n, v, k = case["rows"], case["vocab"], case["k"]
    logits = normal(n, v + case["pad"], scale=2.5)
    if case["op"] == "topk":
        s["logits"] = logits[:, :v]
        return s
    s["logits"] = logits[:, :v]
    s["temperature"] = 2.0
    # the teacher's entries: distinct indices, falling logits; some rows hold
    # fewer entries (absent ones have index -1) and one row in sixteen is padding with none at all
    step = torch.randint(1, v // k + 1, (n, 1), generator=gen, device=DEV)
    first = torch.randint(0, v, (n, 1), generator=gen, device=DEV)
    at = torch.arange(k, device=DEV)
    index = (first + at * step) % v
    count = torch.randint(max(1, k // 2), k + 1, (n, 1), generator=gen, device=DEV)
    count[torch.arange(n, device=DEV) % 16 == 15] = 0
    s["t_index"] = torch.where(at < count, index, -1).to(torch.int32)
    s["t_logits"] = (normal(n, k, dtype=torch.float32).abs_().sort(dim=1, descending=True).values.mul_(3.0).add_(4.0)).to(dt)
    s["dloss"] = torch.rand(n, generator=gen, device=DEV).add_(0.5)
    s["scale"] = 1024.0 / n  # the loss scale over the rows
    return s


# ------------------------------------------------------------------ the plain forms and the package's calls

def run(state: dict):
    return (_run_own if own else _run_plain)(state)


def _run_own(s: dict):
    from zero_sharded_mixed_flat_gb300 import binding as zb

    op = s["case"]["op"]
    if op == "scan_step":
        y, h = s["scan"].step(s["x"], s["f"], s["h0"])
        return {"y": y, "h_last": h}
    if op == "scan":
        y, h, _ = s["scan"].forward(s["x"], s["f"], s["h0"], s["seq_start"])
        return {"y": y, "h_last": h}
    if op == "scan_train":
        y, h, kept = s["scan"].forward(s["x"], s["f"], s["h0"], s["seq_start"], keep=True)
        dx, df, dh0 = s["scan"].backward(s["x"], s["f"], s["dy"], kept, s["h0"], s["dh_last"], s["seq_start"])
        return {"y": y, "h_last": h, "dx": dx, "df": df, "dh0": dh0}
    if op == "topk":
        values, index = zb.topk_logits(s["logits"], s["case"]["k"])
        return {"values": values, "index": index}
    teacher = (s["t_logits"], s["t_index"], s["temperature"])
    if op == "distill_loss":
        loss, lse = zb.distill_loss(s["logits"], *teacher)
        return {"loss": loss, "lse": lse}
    if op == "distill_two":
        loss, lse = zb.distill_loss(s["logits"], *teacher)
        return {"loss": loss, "grad": zb.distill_grad(s["logits"], lse, *teacher, s["scale"], s["dloss"])}
    loss, grad = zb.distill_loss_grad(s["logits"], *teacher, s["scale"], s["dloss"])
    return {"loss": loss, "grad": grad}


def _run_plain(s: dict):
    op = s["case"]["op"]
    if op == "scan_step":
        x, f = s["x"].float(), s["f"].float()
        h = torch.sigmoid(f) * s["h0"] + torch.sigmoid(-f) * x
        return {"y": h.to(s["x"].dtype), "h_last": h}
    if op.startswith("scan"):
        return _plain_scan(s)
    if op == "topk":
        return _plain_topk(s["logits"], s["case"]["k"])
    return _plain_distill(s)


def _doubling(a, b):
    """h_t = a_t h_{t-1} + b_t along dimension 1 (h before the first is zero), in log2(T) passes."""
    d = 1
    while d < a.shape[1]:
        b = torch.cat([b[:, :d], b[:, d:] + a[:, d:] * b[:, :-d]], 1)
        a = torch.cat([a[:, :d], a[:, d:] * a[:, :-d]], 1)
        d *= 2
    return b


def _plain_scan(s: dict):
    start, h0 = s["seq_start"], s["h0"]
    x, f = s["x"].float(), s["f"].float()
    packed = start is not None
    if packed:
        x, f = x[None], f[None]
    t = torch.arange(x.shape[1], device=x.device)
    if packed:
        seq = torch.searchsorted(start, t, right=True) - 1
        first, last = (t == start[seq])[None, :, None], (t + 1 == start[seq + 1])[None, :, None]
        h_in, full = h0[seq][None], (start[1:] > start[:-1])[:, None]
    else:
        first, last = (t == 0)[None, :, None], (t == x.shape[1] - 1)[None, :, None]
        h_in = h0[:, None]
    a, u = torch.sigmoid(f), torch.sigmoid(-f)
    h = _doubling(torch.where(first, 0.0, a), torch.where(first, a * h_in, 0.0) + u * x)
    if packed:
        h_last = torch.where(full, h[0][(start[1:] - 1).clamp(min=0)], h0)
    else:
        h_last = h[:, -1].clone()
    dt = s["x"].dtype
    out = {"y": (h[0] if packed else h).to(dt), "h_last": h_last}
    if s["case"]["op"] == "scan":
        return out
    dy, dh = s["dy"].float(), s["dh_last"]
    if packed:
        dy = dy[None]
    d_in = dh[seq][None] if packed else dh[:, None]
    carry = torch.where(last, 0.0, torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1))
    g = _doubling(carry.flip(1), (dy + torch.where(last, d_in, 0.0)).flip(1)).flip(1)
    before = torch.where(first, h_in, torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1))
    dx, df, back = u * g, g * (before - x) * a * u, a * g
    if packed:
        dh0 = torch.where(full, back[0][start[:-1].clamp(max=x.shape[1] - 1)], dh)
        dx, df = dx[0], df[0]
    else:
        dh0 = back[:, 0].clone()
    return {**out, "dx": dx.to(dt), "df": df.to(dt), "dh0": dh0}


def _plain_topk(logits, k):
    """The k largest of every row, largest first, ties to the lowest index."""
    v = logits.shape[1]
    bits = logits.float().contiguous().view(torch.int32)
    bits = torch.where(bits == -(1 << 31), 0, bits)  # -0 ties with +0
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    key = order * (1 << 32) + torch.arange(v - 1, -1, -1, device=logits.device)
    index = (v - 1) - (torch.topk(key, k, dim=1).values & 0xFFFFFFFF)
    return {"values": logits.gather(1, index), "index": index.to(torch.int32)}


def _plain_distill(s: dict):
    tau, op = s["temperature"], s["case"]["op"]
    z = s["logits"].float() / tau
    there = s["t_index"] >= 0
    none = ~there.any(1)
    at = s["t_index"].clamp(min=0).long()
    t = torch.where(there, s["t_logits"].float() / tau, -math.inf)
    t = t - torch.where(none, 0.0, t.max(1).values)[:, None]
    total = torch.exp(t).sum(1, keepdim=True)
    p = torch.where(there, torch.exp(t) / total, 0.0)
    logp = t - torch.log(total)
    zmax = z.max(1, keepdim=True).values
    lse = zmax + torch.log(torch.exp(z - zmax).sum(1, keepdim=True))
    loss = tau * tau * torch.where(there, p * (logp - (z.gather(1, at) - lse)), 0.0).sum(1)
    if op == "distill_loss":
        return {"loss": loss, "lse": torch.where(none, 0.0, lse[:, 0])}
    g = (tau * s["scale"] * s["dloss"])[:, None]
    grad = (torch.exp(z - lse) * g).scatter_add_(1, at, -p * g)
    return {"loss": loss, "grad": torch.where(none[:, None], 0.0, grad).to(s["logits"].dtype)}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case: dict, seed: int):
    s = prepare(case, seed)
    op = case["op"]
    if op == "topk":
        parts = [s["logits"][i:i + 256].double().sort(dim=1, descending=True).values[:, :case["k"]]
                 for i in range(0, case["rows"], 256)]
        return {"values": torch.cat(parts), "index": None}
    if op.startswith("scan"):
        return _exact_scan(s)
    return _exact_distill(s)


def _exact_scan(s: dict):
    op, start = s["case"]["op"], s["seq_start"]
    x, f = s["x"].double(), s["f"].double()
    if op == "scan_step":
        x, f = x[:, None], f[:, None]
    if start is not None:
        x, f = x[None], f[None]
    n = x.shape[1]
    bounds = [0, n] if start is None else start.tolist()
    h0 = s["h0"].double()
    a = 1.0 / (1.0 + torch.exp(-f))
    u = 1.0 / (1.0 + torch.exp(f))
    b = u * x
    h, before = torch.empty_like(x), torch.empty_like(x)
    h_last, dh0 = h0.clone(), torch.zeros_like(h0)
    for i in range(len(bounds) - 1):
        mine = slice(i, i + 1) if start is not None else slice(None)
        now = h0[mine]
        for t in range(bounds[i], bounds[i + 1]):
            before[:, t] = now
            now = torch.addcmul(b[:, t], a[:, t], now)
            h[:, t] = now
        h_last[mine] = now
    y = h[:, 0] if op == "scan_step" else h[0] if start is not None else h
    out = {"y": y, "h_last": h_last}
    if op != "scan_train":
        return out
    dy, dh = s["dy"].double(), s["dh_last"].double()
    if start is not None:
        dy = dy[None]
    g = torch.empty_like(x)
    for i in range(len(bounds) - 1):
        mine = slice(i, i + 1) if start is not None else slice(None)
        now = dh[mine]
        for t in range(bounds[i + 1] - 1, bounds[i] - 1, -1):
            now = dy[:, t] + now
            g[:, t] = now
            now = a[:, t] * now
        dh0[mine] = now
    dx, df = u * g, g * (before - x) * a * u
    if start is not None:
        dx, df = dx[0], df[0]
    return {**out, "dx": dx, "df": df, "dh0": dh0}


def _exact_distill(s: dict):
    tau, op = s["temperature"], s["case"]["op"]
    losses, lses, grads = [], [], []
    for i in range(0, s["logits"].shape[0], 512):
        cut = slice(i, i + 512)
        logq = torch.log_softmax(s["logits"][cut].double() / tau, 1)
        lse = torch.logsumexp(s["logits"][cut].double() / tau, 1)
        index = s["t_index"][cut].long()
        weight = torch.exp(s["t_logits"][cut].double() / tau) * (index >= 0)
        some = weight.sum(1) > 0
        p = weight / weight.sum(1, keepdim=True).clamp(min=1e-300)
        q_at = logq.gather(1, index.clamp(min=0))
        terms = p * (torch.log(p.clamp(min=1e-300)) - q_at)
        losses.append(tau ** 2 * torch.where(some, terms.sum(1), 0.0))
        lses.append(torch.where(some, lse, 0.0))
        if op != "distill_loss":
            target = torch.zeros_like(logq).scatter_add_(1, index.clamp(min=0), p)
            g = tau * s["scale"] * s["dloss"][cut].double()
            grads.append((torch.exp(logq) - target) * torch.where(some, g, 0.0)[:, None])
    if op == "distill_loss":
        return {"loss": torch.cat(losses), "lse": torch.cat(lses)}
    return {"loss": torch.cat(losses), "grad": torch.cat(grads)}
