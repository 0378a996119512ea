"""The norms around a block with its gate and residual scale, and their gradients,
against the formulas in 64 bits."""
import math

import numpy as np
import pytest
import torch

import block_ref as ref
from zero_sharded_mixed_flat_gb300 import binding as zb

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS, R = 1e-6, 0.875


def rand(shape, seed, dtype, scale=1.0, shift=0.0):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape) * scale + shift).to(dtype)


def strided(t, pad, offset):
    flat = torch.full((offset + t.shape[0] * (t.shape[1] + pad),), 7.0, dtype=t.dtype, device="cuda")
    view = flat[offset:].view(t.shape[0], t.shape[1] + pad)[:, :t.shape[1]]
    view.copy_(t)
    return view


def make(n, d, dtype, groups=1, post=True, gate=True, pre=True, block=True, seed=1):
    dt = DT[dtype]
    c = {"x": rand((n, d), seed, dt, 3.0), "o": rand((n, d), seed + 1, dt, 0.7) if block else None,
         "w_post": rand((d,), seed + 2, dt, 0.1, 1.0) if post and block else None,
         "gate": rand((groups, d), seed + 3, dt, 0.3, 0.5) if gate and block else None,
         "w_pre": rand((d,), seed + 4, dt, 0.1, 1.0) if pre else None}
    up = {"dn": rand((n, d), seed + 5, dt, 1e-3) if pre else None, "dx_new": rand((n, d), seed + 6, dt, 1e-3)}
    return c, up


def cuda(c):
    return {k: None if v is None else v.cuda() for k, v in c.items()}


def formulas(c, up, dt):
    f = ref.block(c["x"], c["o"], c["w_post"], c["gate"], c["w_pre"], R, EPS)
    fwd = {"x_new": (f["x"], ref.stored(f["x"], f["err"]["x"], dt))}
    if c["w_pre"] is not None:
        fwd["n"] = (f["n"], ref.stored(f["n"], f["err"]["n"], dt))
    g, e = ref.block_grad(c["x"], up["dn"], up["dx_new"], c["o"], c["w_post"], c["gate"], c["w_pre"], R, EPS)
    back = [None if a is None else (a, ref.stored(a, b, dt)) for a, b in zip(g, e)]
    return fwd, back


def held(got, want, what):
    assert (got is None) == (want is None), what
    if got is not None:
        ref.check(got, *want, what)


NAMES = ("dx", "do", "dw_pre", "dw_post", "dgate")
SIZES = [(1, 1), (1, 768), (2, 7), (3, 31), (5, 33), (32, 768), (257, 96), (700, 128), (64, 771), (7, 2048), (9, 2050), (4, 4096),
         (3, 4099), (2, 8192), (3, 10007), (2, 16384)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,d", SIZES)
def test_forward_and_gradients(n, d, dtype):
    c, up = make(n, d, dtype)
    fwd, back = formulas(c, up, DT[dtype])
    k, u = cuda(c), cuda(up)
    x_new, nn, kept = zb.block_norm(**k, res_scale=R, eps=EPS, keep=True)
    held(x_new, fwd["x_new"], "x_new")
    held(nn, fwd["n"], "n")
    got = zb.block_norm_grad(k.pop("x"), kept, **u, **k, res_scale=R, eps=EPS)
    for g, w, name in zip(got, back, NAMES):
        held(g, w, name)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,d", [(6, 64), (50, 771), (12, 1536)])
@pytest.mark.parametrize("post,gate,pre,block,stream", [(False, True, True, True, True), (True, False, True, True, True),
                                                        (True, True, False, True, True), (False, False, True, True, False),
                                                        (True, True, True, True, False), (False, False, True, False, True),
                                                        (False, False, True, False, False), (False, False, False, True, True)])
def test_parts_left_out(n, d, post, gate, pre, block, stream, dtype):
    c, up = make(n, d, dtype, 1, post, gate, pre, block, seed=20)
    if not stream:
        up["dx_new"] = None
    fwd, back = formulas(c, up, DT[dtype])
    k, u = cuda(c), cuda(up)
    x_new, nn, kept = zb.block_norm(**k, res_scale=R, eps=EPS, keep=True)
    held(x_new, fwd["x_new"] if block else None, "x_new")
    held(nn, fwd.get("n"), "n")
    if not block:
        out = torch.empty_like(k["x"])
        assert zb.block_norm(**k, res_scale=R, eps=EPS, out=out)[0] is out
        held(out, fwd["x_new"], "x_new asked for")
    got = zb.block_norm_grad(k.pop("x"), kept, **u, **k, res_scale=R, eps=EPS)
    for g, w, name in zip(got, back, NAMES):
        held(g, w, name)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("n,groups,d", [(6, 2, 64), (12, 12, 33), (300, 3, 96), (640, 320, 40), (700, 700, 64), (2000, 1000, 24),
                                        (610, 305, 771), (1301, 1, 520)])
def test_gates_of_groups(n, groups, d, post, dtype):
    c, up = make(n, d, dtype, groups, post, seed=40)
    fwd, back = formulas(c, up, DT[dtype])
    k, u = cuda(c), cuda(up)
    x_new, nn, kept = zb.block_norm(**k, res_scale=R, eps=EPS, keep=True)
    held(x_new, fwd["x_new"], "x_new")
    held(nn, fwd["n"], "n")
    got = zb.block_norm_grad(k.pop("x"), kept, **u, **k, res_scale=R, eps=EPS)
    for g, w, name in zip(got, back, NAMES):
        held(g, w, name)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,offset", [(8, 8), (1, 0), (3, 5), (4, 0)])
@pytest.mark.parametrize("d", [64, 70, 771])
def test_rows_apart_and_in_place(d, pad, offset, dtype):
    n = 21
    c, up = make(n, d, dtype, 3, seed=60)
    fwd, back = formulas(c, up, DT[dtype])
    k, u = cuda(c), cuda(up)
    for name in ("x", "o"):
        k[name] = strided(c[name], pad, offset)
    for name in ("dn", "dx_new"):
        u[name] = strided(up[name], pad, offset)
    x = k.pop("x")
    x_new, nn, kept = zb.block_norm(x, **k, res_scale=R, eps=EPS, keep=True)
    held(x_new, fwd["x_new"], "x_new")
    got = zb.block_norm_grad(x, kept, **u, **k, res_scale=R, eps=EPS, out=(u["dx_new"], u["dn"]))
    assert got[0] is u["dx_new"] and got[1] is u["dn"]
    for g, w, name in zip(got, back, NAMES):
        held(g, w, name)
    o = k["o"]
    got = zb.block_norm(x, **k, res_scale=R, eps=EPS, out=x, n_out=o)
    assert got[0] is x and got[1] is o
    held(x, fwd["x_new"], "x_new in place")
    held(o, fwd["n"], "n in place")
    for t in (x, o, u["dn"], u["dx_new"]):  # the padding between rows stays as it was
        whole = t.as_strided((n, d + pad), (d + pad, 1))
        assert bool((whole[:-1, d:] == 7.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [511, 512, 513, 1021, 1024, 2047, 2048, 4095, 4096, 4100, 8191, 12000, 16383])
def test_widths_that_fill_a_team_at_any_alignment(d, dtype):
    """Rows one element apart from their neighbours, NaN between them, at widths of whole teams and one off."""
    n = 11
    c, up = make(n, d, dtype, seed=70)
    fwd, back = formulas(c, up, DT[dtype])
    k, u = cuda(c), cuda(up)

    def apart(t):
        flat = torch.full((n * (d + 1) + 1,), math.nan, dtype=t.dtype, device="cuda")
        view = flat[1:].view(n, d + 1)[:, :d]
        view.copy_(t)
        return view

    x, k["o"] = apart(k.pop("x")), apart(k["o"])
    u = {name: apart(t) for name, t in u.items()}
    x_new, nn, kept = zb.block_norm(x, **k, res_scale=R, eps=EPS, keep=True)
    held(x_new, fwd["x_new"], "x_new")
    held(nn, fwd["n"], "n")
    for g, w, name in zip(zb.block_norm_grad(x, kept, **u, **k, res_scale=R, eps=EPS), back, NAMES):
        held(g, w, name)


def test_more_dimensions_and_a_gate_of_one():
    c, up = make(24, 48, "f32", seed=80)
    k, u = cuda(c), cuda(up)
    want = zb.block_norm(**k, keep=True)
    want_grad = zb.block_norm_grad(k["x"], want[2], **u, **{a: b for a, b in k.items() if a != "x"})
    shaped = {a: (b.view(2, 3, 4, 48) if a in ("x", "o") else b.view(48) if a == "gate" else b) for a, b in k.items()}
    got = zb.block_norm(**shaped, keep=True)
    assert got[0].shape == (2, 3, 4, 48) and torch.equal(got[0].view(24, 48), want[0])
    x = shaped.pop("x")
    grad = zb.block_norm_grad(x, got[2], *(u[a].view(2, 3, 4, 48) for a in ("dn", "dx_new")), **shaped)
    assert grad[4].shape == (48,)
    assert all(torch.equal(a.reshape(-1), b.reshape(-1)) for a, b in zip(grad, want_grad))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_zero_rows_huge_rows_and_non_finite_ones(dtype):
    c, up = make(9, 768, dtype, seed=90)
    c["x"][1] = 0
    c["o"][1] = 0          # nothing but eps under the roots
    c["o"][2] = 0
    c["x"][3] *= 1e15
    c["o"][4] *= 1e-18     # below eps
    fwd, back = formulas(c, up, DT[dtype])
    k, u = cuda(c), cuda(up)
    x_new, nn, kept = zb.block_norm(**k, res_scale=R, eps=EPS, keep=True)
    held(x_new, fwd["x_new"], "x_new")
    held(nn, fwd["n"], "n")
    x = k.pop("x")
    clean = zb.block_norm_grad(x, kept, **u, **k, res_scale=R, eps=EPS)
    for g, w, name in zip(clean[:2], back[:2], NAMES):
        held(g, w, name)
    x[5, 700], k["o"][7, 3] = math.nan, math.inf
    bad_x, bad_n, kept = zb.block_norm(x, **k, res_scale=R, eps=EPS, keep=True)
    bad = zb.block_norm_grad(x, kept, **u, **k, res_scale=R, eps=EPS)
    rows = torch.tensor([r for r in range(9) if r not in (5, 7)], device="cuda")
    for a, b in ((bad_x, x_new), (bad_n, nn), (bad[0], clean[0]), (bad[1], clean[1])):
        assert torch.equal(a[rows], b[rows])
    assert bool(torch.isnan(bad_n[5]).all()) and bool(torch.isnan(bad_n[7]).any())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,groups,d", [(3001, 1, 64), (3001, 1, 520), (3001, 1, 640), (3000, 1000, 520), (3000, 1000, 1600),
                                        (3001, 1, 1280), (3001, 1, 1600), (2500, 5, 2880), (1200, 1, 5000), (700, 1, 10000)])
def test_non_finite_rows_stay_alone_where_lanes_have_no_column(n, groups, d, dtype):
    """Aligned widths that leave lanes of a team without a column, rows that follow one another in the same shared
    memory: the finite rows have the same bits whatever the others, or an earlier call, held."""
    dt, gen = DT[dtype], torch.Generator("cuda").manual_seed(95)

    def rand_here(*shape, scale=1.0, shift=0.0):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(scale).add_(shift).to(dt)

    x, o = rand_here(n, d, scale=3.0), rand_here(n, d, scale=0.7)
    dn, dy = rand_here(n, d, scale=1e-3), rand_here(n, d, scale=1e-3)
    block = {"w_post": rand_here(d, scale=0.1, shift=1.0), "w_pre": rand_here(d, scale=0.1, shift=1.0),
             "gate": rand_here(groups, d, scale=0.3, shift=0.5), "res_scale": R, "eps": EPS}

    def both(x, o, dn, dy):
        x_new, nn, kept = zb.block_norm(x, o=o, keep=True, **block)
        return [x_new, nn, *zb.block_norm_grad(x, kept, dn, dy, o=o, **block)]

    clean = both(x, o, dn, dy)
    # the first and the last rows of the first and the last gate by the formulas, which take each row by itself
    each = n // groups
    for cut in (slice(0, min(each, 20)), slice(n - min(each, 20), n)):
        g = block["gate"][cut.start // each][None].cpu()
        w1, w2 = block["w_post"].cpu(), block["w_pre"].cpu()
        f = ref.block(x[cut].cpu(), o[cut].cpu(), w1, g, w2, R, EPS)
        want, err = ref.block_grad(x[cut].cpu(), dn[cut].cpu(), dy[cut].cpu(), o[cut].cpu(), w1, g, w2, R, EPS)
        for got, v, e in ((clean[0], f["x"], f["err"]["x"]), (clean[1], f["n"], f["err"]["n"]), (clean[2], want[0], err[0]),
                          (clean[3], want[1], err[1])):
            ref.check(got[cut], v, ref.stored(v, e, dt))
    nan = torch.full_like(x, math.nan)
    for _ in range(3):
        both(nan, nan, nan, nan)
        again = both(x, o, dn, dy)
        assert all(torch.equal(p, q) for p, q in zip(again, clean))
    good = torch.arange(n, device="cuda") % 3 != 1
    spoilt = [t.clone() for t in (x, o, dn, dy)]
    for t, bad in zip(spoilt, (math.nan, math.inf, -math.inf, math.nan)):
        t[1::3, :8] = bad
    for which in ((0,), (1,), (2,), (3,), (0, 1, 2, 3)):
        got = both(*(spoilt[i] if i in which else t for i, t in enumerate((x, o, dn, dy))))
        assert all(torch.equal(p[good], q[good]) for p, q in zip(got[:4], clean)), which


def test_gradient_against_differences():
    c, up = make(5, 24, "f32", 5, seed=100)
    k, u = cuda(c), cuda(up)
    x = k.pop("x")
    _, _, kept = zb.block_norm(x, **k, res_scale=R, eps=EPS, keep=True)
    got = zb.block_norm_grad(x, kept, **u, **k, res_scale=R, eps=EPS)
    step = 1e-5
    for i, name in enumerate(("x", "o", "w_pre", "w_post", "gate")):
        move = rand(c[name].shape, 110 + i, torch.float64)

        def value(sign):
            moved = dict(c, **{name: c[name].double() + sign * step * move})
            f = ref.block(moved["x"], moved["o"], moved["w_post"], moved["gate"], moved["w_pre"], R, EPS)
            return float((f["x"] * up["dx_new"].double()).sum() + (f["n"] * up["dn"].double()).sum())

        slope = (value(1) - value(-1)) / (2 * step)
        mine = got[i].double().cpu() * move
        # the differences' own error is of the order of step^2, 1e-10
        assert abs(slope - float(mine.sum())) <= 1e-5 * float(mine.abs().sum()), name


def test_same_bits_streams_and_graphs():
    c, up = make(1000, 520, "bf16", 4, seed=120)
    k, u = cuda(c), cuda(up)
    x = k.pop("x")

    def both(x, stream=None):
        a = zb.block_norm(x, **k, res_scale=R, keep=True, stream=stream)
        return (*a, *zb.block_norm_grad(x, a[2], **u, **k, res_scale=R, stream=stream))

    want = both(x)
    torch.cuda.synchronize()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    got = both(x, side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    s = torch.zeros_like(x)
    graphs, kept = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for g in graphs:
        with torch.cuda.graph(g):
            kept.append(both(s))
    s.copy_(x)
    torch.cuda.synchronize()
    for _ in range(3):
        for g, st in zip(graphs, (side, other)):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for got in kept:
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_no_rows():
    c, up = make(0, 40, "bf16")
    k, u = cuda(c), cuda(up)
    x_new, n, kept = zb.block_norm(**k, keep=True)
    assert x_new.shape == n.shape == (0, 40)
    got = zb.block_norm_grad(k.pop("x"), kept, **u, **k)
    assert got[0].shape == (0, 40) and all(bool((g == 0).all()) for g in got[2:])


def test_refusals():
    c, up = make(6, 16, "f32", 2)
    k, u = cuda(c), cuda(up)
    x, rest = k["x"], {a: b for a, b in k.items() if a != "x"}
    with pytest.raises(zb.ZgError, match="groups must divide rows"):
        zb.block_norm(x[:5], **dict(rest, o=k["o"][:5]))
    with pytest.raises(ValueError, match="o must have shape"):
        zb.block_norm(x, **dict(rest, o=k["o"][:5]))
    with pytest.raises(TypeError, match="w_pre must have dtype"):
        zb.block_norm(x, **dict(rest, w_pre=k["w_pre"].bfloat16()))
    with pytest.raises(ValueError, match="gate must have shape"):
        zb.block_norm(x, **dict(rest, gate=k["gate"][:, :8]))
    with pytest.raises(zb.ZgError, match="must be NULL where o is"):
        zb.block_norm(x, **dict(rest, o=None))
    with pytest.raises(zb.ZgError, match="neither"):
        zb.block_norm(x)
    with pytest.raises(zb.ZgError, match="eps"):
        zb.block_norm(**k, eps=-1.0)
    with pytest.raises(zb.ZgError, match="res_scale"):
        zb.block_norm(**k, res_scale=math.inf)
    with pytest.raises(zb.ZgError, match="x_new must not overlap"):
        zb.block_norm(**k, out=k["o"])
    with pytest.raises(zb.ZgError, match="n must not overlap"):
        zb.block_norm(**k, n_out=x)
    with pytest.raises(zb.ZgError, match="width"):
        zb.block_norm(torch.zeros(1, 16385, device="cuda"), torch.zeros(16385, device="cuda"))
    kept = zb.block_norm(**k, keep=True)[2]
    with pytest.raises(ValueError, match="kept is None"):
        zb.block_norm_grad(x, None, **u, **rest)
    with pytest.raises(ValueError, match="kept must have shape"):
        zb.block_norm_grad(x, kept[:, :5].contiguous(), **u, **rest)
    with pytest.raises(zb.ZgError, match="dn is NULL"):
        zb.block_norm_grad(x, kept, None, u["dx_new"], **rest)
    with pytest.raises(zb.ZgError, match="dx and d_o overlap"):
        zb.block_norm_grad(x, kept, **u, **rest, out=(x, u["dn"]))
    with pytest.raises(ValueError, match="contiguous"):
        zb.block_norm(torch.zeros(2, 3, 32, device="cuda")[..., :16], k["w_pre"])
