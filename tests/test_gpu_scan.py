"""The gated linear recurrence against its formulas in 64 bits."""
import math

import numpy as np
import pytest
import torch

import operators_ref as ref
from gpu_helpers import Guarded
from zero_sharded_mixed_flat_gb300 import binding as zb

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def rand(shape, seed, scale=1.0, shift=0.0):
    rng = np.random.default_rng(seed)
    return torch.from_numpy(rng.standard_normal(shape) * scale + shift)


def views(b, t, c, dtype, layout, seed):
    """x and f on the GPU in one of the layouts a program has them in."""
    x, f = rand((b, t, c), seed).to(dtype), rand((b, t, c), seed + 1, 1.5, 2.0).to(dtype)
    if layout == "plain":
        return x.cuda(), f.cuda()
    if layout == "fused":  # halves of one projection's output
        both = torch.cat([x, f], -1).cuda()
        return both[..., :c], both[..., c:]
    if layout == "odd":  # one element off every alignment, odd strides
        wide = torch.zeros(2, b, t, c + 3, dtype=dtype)
        wide[0, ..., 1:c + 1], wide[1, ..., 1:c + 1] = x, f
        wide = wide.cuda()
        return wide[0, ..., 1:c + 1], wide[1, ..., 1:c + 1]
    assert layout == "time_major"
    return x.transpose(0, 1).contiguous().cuda().transpose(0, 1), f.transpose(0, 1).contiguous().cuda().transpose(0, 1)


def run_case(b, t, c, dtype, layout="plain", starts=None, seed=0, with_h0=True, f_override=None):
    dtype = DT[dtype]
    x, f = views(b, t, c, dtype, layout, seed)
    if f_override is not None:
        f.copy_(f_override(f))
    seqs = b if starts is None else len(starts) - 1
    bounds = [(r, 0, t) for r in range(b)] if starts is None else [(0, lo, hi) for lo, hi in zip(starts, starts[1:])]
    h0 = rand((seqs, c), seed + 2).float() if with_h0 else None
    dh = rand((seqs, c), seed + 3).float() if with_h0 else None
    dy = rand((b, t, c), seed + 4).to(dtype)
    seq_start = None if starts is None else torch.tensor(starts, dtype=torch.int64).cuda()
    scan = zb.GatedScan(b, t, c)
    gx, gf, gdy = (x, f, dy.cuda()) if starts is None else (x[0], f[0], dy[0].cuda())
    g0, gdh = (h0.cuda(), dh.cuda()) if with_h0 else (None, None)
    y, last, kept = scan.forward(gx, gf, g0, seq_start, keep=True)
    dx, df, dh0 = scan.backward(gx, gf, gdy, kept, g0, gdh, seq_start)
    assert scan.status() == zb.ZG_OK
    X, F = x.double().cpu(), f.double().cpu()
    H0 = h0.double() if with_h0 else torch.zeros(seqs, c, dtype=torch.float64)
    DH = dh.double() if with_h0 else torch.zeros(seqs, c, dtype=torch.float64)
    h, wl, _, he, le, _ = ref.scan(X, F, H0, bounds)
    wx, wf, w0, xe, fe, e0 = ref.scan_grad(X, F, H0, dy.double(), DH, bounds)
    end = t if starts is None else starts[-1]
    for got, want, err, what in ((y, h, he, "y"), (dx, wx, xe, "dx"), (df, wf, fe, "df")):
        got = got[None] if starts is not None else got
        ref.check(got[:, :end], want[:, :end], ref.stored(want, err, dtype)[:, :end], what)
    ref.check(last, wl, ref.stored(wl, le, torch.float32), "h_last")
    ref.check(dh0, w0, ref.stored(w0, e0, torch.float32), "dh0")
    # the same bits again
    y2, last2, kept2 = scan.forward(gx, gf, g0, seq_start, keep=True)
    again = scan.backward(gx, gf, gdy, kept2, g0, gdh, seq_start)
    y, y2 = (y[:end], y2[:end]) if starts is not None else (y, y2)
    assert torch.equal(y, y2) and torch.equal(last, last2) and torch.equal(dh0, again[2])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("b,t,c", [(1, 1, 1), (3, 1, 5), (5, 1, 768), (2, 2, 64), (1, 7, 63), (2, 16, 129), (2, 31, 66),
                                   (1, 127, 65), (2, 128, 64), (1, 129, 130), (2, 255, 32), (3, 257, 96), (1, 1000, 771),
                                   (1, 4099, 40), (2, 2305, 67)])
def test_sizes(b, t, c, dtype):
    run_case(b, t, c, dtype, seed=b * 1000 + t + c)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["fused", "odd", "time_major"])
@pytest.mark.parametrize("b,t,c", [(2, 1, 70), (2, 33, 66), (3, 300, 130)])
def test_layouts(b, t, c, dtype, layout):
    run_case(b, t, c, dtype, layout, seed=7)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("c", [1, 63, 64, 68, 131])
@pytest.mark.parametrize("off", range(8))
def test_every_alignment_among_nans(off, c, dtype):
    """Rows that begin at any place in a 16-byte unit, each operand's at another and with
    another stride, between NaNs: the elements beside a row take no part."""
    b, t, dt = 2, 140, DT[dtype]
    x, f = views(b, t, c, dt, "plain", 70 + off)
    dy = rand((b, t, c), 72).to(dt).cuda()

    def placed(v, first, step):
        wide = torch.full((b * t * step + 32,), math.nan, dtype=dt, device="cuda")
        at = wide[first:first + b * t * step].view(b, t, step)[..., :c]
        at.copy_(v)
        return at

    px, pf, pd = placed(x, off, c + off), placed(f, (3 * off + 1) % 8, c + 5), placed(dy, (5 * off + 2) % 8, c + 8 - off)
    scan = zb.GatedScan(b, t, c)
    y, _, kept = scan.forward(px, pf, keep=True)
    dx, df, _ = scan.backward(px, pf, pd, kept)
    X, F, bounds = x.double().cpu(), f.double().cpu(), [(r, 0, t) for r in range(b)]
    zero = torch.zeros(b, c, dtype=torch.float64)
    h, _, _, he, _, _ = ref.scan(X, F, zero, bounds)
    wx, wf, _, xe, fe, _ = ref.scan_grad(X, F, zero, dy.double().cpu(), zero, bounds)
    for got, want, err, what in ((y, h, he, "y"), (dx, wx, xe, "dx"), (df, wf, fe, "df")):
        ref.check(got, want, ref.stored(want, err, dt), what)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("starts", [[0, 300], [0, 0, 0, 300], [0, 300, 300, 300], [0, 1, 2, 3, 300], [0, 128, 256, 300],
                                    [0, 127, 129, 129, 256, 299, 300], [0, 100, 100, 150], [0, 0, 0], [0, 250, 260],
                                    list(range(301))])
def test_packed_sequences(starts, dtype):
    run_case(1, 300, 71, dtype, starts=starts, seed=11)


def test_packed_many_sequences_over_many_chunks():
    rng = np.random.default_rng(5)
    cuts = sorted(int(v) for v in rng.integers(0, 3001, 40))
    run_case(1, 3000, 66, "bf16", starts=[0, *cuts, 3000], seed=13)
    run_case(1, 3000, 65, "f32", "odd", starts=[0, *cuts, 2900 if cuts[-1] <= 2900 else cuts[-1]], seed=14)


def test_more_empty_sequences_than_tokens_in_a_chunk():
    run_case(1, 200, 33, "f32", starts=[0] * 200 + [70] * 300 + [200] * 150, seed=15)


@pytest.mark.parametrize("t", [1, 64, 700])
def test_no_initial_state(t):
    run_case(2, t, 66, "f32", seed=17, with_h0=False)


@pytest.mark.parametrize("shift", [-200.0, -20.0, 9.0, 30.0, 200.0])
def test_gates_near_and_at_their_ends(shift):
    """From forgetting everything to holding for ever."""
    run_case(2, 400, 66, "f32", seed=19, f_override=lambda f: f * 0.5 + shift)


def test_infinite_gates():
    def some(f):
        g = f.clone()
        g[:, ::5] = math.inf
        g[:, ::7] = -math.inf
        return g
    run_case(2, 300, 66, "f32", seed=23, f_override=some)
    run_case(2, 300, 66, "bf16", seed=23, f_override=some)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_non_finite_values_stay_in_their_sequence_and_channel(dtype):
    t, c = 700, 70
    starts = torch.tensor([0, 200, 450, 600], dtype=torch.int64).cuda()
    x, f = (v[0] for v in views(1, t, c, DT[dtype], "plain", 29))
    x[599:], f[600:] = math.nan, math.nan  # the last token of the third sequence, and all past the end
    x[250, 3], f[300, 4] = math.nan, math.nan
    scan = zb.GatedScan(1, t, c)
    h0 = torch.zeros(3, c, device="cuda")
    dy = torch.ones_like(x)
    dy[600:] = math.nan
    y, last, kept = scan.forward(x, f, h0, starts, keep=True)
    dx, df, dh0 = scan.backward(x, f, dy, kept, h0, None, starts)
    bad = torch.zeros(t, c, dtype=torch.bool, device="cuda")
    bad[250:450, 3] = True
    bad[300:450, 4] = True
    bad[599] = True
    assert torch.equal(torch.isnan(y[:600]), bad[:600])
    assert torch.equal(torch.isnan(last), torch.stack([bad[199], bad[449], bad[599]]))
    bad_dx = torch.zeros_like(bad)
    bad_dx[200:301, 4] = True
    assert torch.equal(torch.isnan(dx[:600]), bad_dx[:600])
    bad_df = bad_dx.clone()
    bad_df[250:450, 3] = True
    bad_df[300:450, 4] = True
    bad_df[599] = True
    assert torch.equal(torch.isnan(df[:600]), bad_df[:600])
    assert torch.isnan(dh0).nonzero().tolist() == [[1, 4]]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t,end", [(5, 4), (300, 290)])
def test_only_the_outputs_are_written(t, end, dtype):
    """Guards around every output, and the rows past the last sequence, keep their bytes."""
    c, dt = 67, DT[dtype]
    x, f = (v[0] for v in views(1, t, c, dt, "plain", 31))
    starts = torch.tensor([0, 2, end], dtype=torch.int64).cuda()
    big = {k: Guarded(t * c, dt) for k in ("y", "dx", "df")}
    last = Guarded(2 * c, torch.float32)
    scan = zb.GatedScan(1, t, c)
    out = {k: g.view.view(t, c) for k, g in big.items()}
    _, _, kept = scan.forward(x, f, None, starts, keep=True, out=out["y"], h_last=last.view.view(2, c))
    scan.backward(x, f, torch.ones_like(x), kept, None, None, starts, out=(out["dx"], out["df"]))
    torch.cuda.synchronize()
    assert last.intact()
    for k, g in big.items():
        assert g.intact(), k
        tail = out[k][end:].contiguous().view(torch.uint8)
        assert bool((tail == 0xA5).all()), k
        assert bool(torch.isfinite(out[k][:end]).all()), k


def test_state_updated_in_place_token_by_token():
    """Decoding one token at a time gives what one call over all tokens gives."""
    b, t, c = 3, 9, 768
    x, f = views(b, t, c, torch.bfloat16, "plain", 37)
    h0 = rand((b, c), 38).float().cuda()
    scan = zb.GatedScan(b, t, c)
    y, last, _ = scan.forward(x, f, h0)
    state = h0.clone()
    for i in range(t):
        yi, s = scan.step(x[:, i], f[:, i], state, out_state=state)
        assert s is state
        ref.check(yi, y[:, i].double().cpu(), ref.BF16 * y[:, i].double().abs().cpu() + 1e-6, i)
    ref.check(state, last.double().cpu(), 1e-6 + ref.EPS * last.double().abs().cpu())
    # in place over many chunks
    x, f = views(b, 700, c, torch.bfloat16, "plain", 39)
    scan = zb.GatedScan(b, 700, c)
    _, want, _ = scan.forward(x, f, h0)
    state = h0.clone()
    scan.forward(x, f, state, h_last=state)
    assert torch.equal(state, want)


def test_gradient_against_differences():
    b, t, c = 1, 150, 9
    x, f = (v.double().cpu() for v in views(b, t, c, torch.float32, "plain", 41))
    h0, w = rand((1, c), 42).float().double(), rand((b, t, c), 43).float().double()
    bounds = [(0, 0, t)]
    scan = zb.GatedScan(b, t, c)
    gx, gf, g0 = x.float().cuda(), f.float().cuda(), h0.float().cuda()
    _, _, kept = scan.forward(gx, gf, g0, keep=True)
    dx, df, dh0 = scan.backward(gx, gf, w.float().cuda(), kept, g0)
    for which, grad in (("x", dx), ("f", df), ("h", dh0)):
        d = rand(grad.shape, 44)
        step = 1e-5

        def value(sign):
            at = {"x": x, "f": f, "h": h0}
            at[which] = at[which] + sign * step * d
            return float((ref.scan(at["x"], at["f"], at["h"], bounds)[0] * w).sum())

        slope = (value(1) - value(-1)) / (2 * step)
        mine = float((grad.double().cpu() * d).sum())
        # the difference's own error is of the order step^2; the gradient's is its rounding
        assert abs(slope - mine) <= 1e-5 * float((grad.double().cpu() * d).abs().sum()), which


def test_another_stream_and_graph_replay():
    b, t, c = 2, 600, 130
    x, f = views(b, t, c, torch.bfloat16, "plain", 47)
    scan = zb.GatedScan(b, t, c)
    want = [v.clone() for v in scan.forward(x, f)[:2]]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = scan.forward(x, f)[:2]
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    sx, sf = torch.zeros_like(x), torch.zeros_like(f)
    out, last = torch.empty_like(x), torch.empty(b, c, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        scan.forward(sx, sf, out=out, h_last=last)
    for _ in range(3):
        sx.copy_(x)
        sf.copy_(f)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(last, want[1])


def test_one_handle_serves_smaller_shapes():
    scan = zb.GatedScan(3, 900, 200)
    for b, t, c in ((3, 900, 200), (1, 1, 1), (2, 300, 64), (3, 129, 200), (1, 900, 33)):
        x, f = views(b, t, c, torch.float32, "plain", 53)
        y, _, _ = scan.forward(x, f)
        h, _, _, e, _, _ = ref.scan(x.double().cpu(), f.double().cpu(), torch.zeros(b, c, dtype=torch.float64),
                                    [(r, 0, t) for r in range(b)])
        ref.check(y, h, ref.stored(h, e, torch.float32))


def test_offsets_past_32_bits():
    """Rows so far apart that element offsets pass 2^31 (the same memory read with a wide stride)."""
    b, t, c = 2, 200, 64
    gap = (1 << 31) + 64
    x = torch.zeros(gap + t * c, dtype=torch.bfloat16, device="cuda")
    dense, f = views(b, t, c, torch.bfloat16, "plain", 59)
    far = x.as_strided((b, t, c), (gap, c, 1))
    far.copy_(dense)
    scan = zb.GatedScan(b, t, c)
    assert torch.equal(scan.forward(far, f)[0], scan.forward(dense, f)[0])


def test_refusals():
    scan = zb.GatedScan(2, 64, 32)
    x = torch.zeros(2, 64, 32, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(zb.ZgError, match="larger than the handle"):
        scan.forward(torch.zeros(2, 65, 32, device="cuda"), torch.zeros(2, 65, 32, device="cuda"))
    with pytest.raises(TypeError, match="f must have dtype"):
        scan.forward(x, x.float())
    with pytest.raises(ValueError, match="f must have shape"):
        scan.forward(x, x[:, :3])
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        scan.forward(x.half(), x.half())
    with pytest.raises(ValueError, match="contiguous"):
        scan.forward(x.transpose(1, 2)[:, :, :32], x.transpose(1, 2)[:, :, :32])
    with pytest.raises(ValueError, match="h0 must have shape"):
        scan.forward(x, x, torch.zeros(3, 32, device="cuda"))
    with pytest.raises(TypeError, match="h0 must have dtype"):
        scan.forward(x, x, torch.zeros(2, 32, device="cuda", dtype=torch.float64))
    with pytest.raises(zb.ZgError, match="batch = 1"):
        scan.forward(x, x, seq_start=torch.tensor([0, 64], device="cuda"))
    with pytest.raises(zb.ZgError, match="overlap"):
        scan.forward(x, x, out=x[:, :1].expand(2, 64, 32))
    with pytest.raises(ValueError, match="kept is None"):
        scan.backward(x, x, x, None)


def test_a_wait_that_runs_out_is_reported_and_forgotten():
    b, t, c = 1, 20000, 130
    x, f = views(b, t, c, torch.bfloat16, "plain", 61)
    scan = zb.GatedScan(b, t, c)
    want = scan.forward(x, f)[0]
    assert scan.status() == zb.ZG_OK
    scan.set_wait_limit(0)  # every first look that finds nothing gives up
    scan.forward(x, f)
    assert scan.status() == zb.ZG_ERR_DEVICE_TIMEOUT
    assert scan.status() == zb.ZG_OK
    scan.set_wait_limit(4000000)
    assert torch.equal(scan.forward(x, f)[0], want)
    assert scan.status() == zb.ZG_OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("c", [70, 64])
def test_a_nan_leaves_the_other_channels_values_alone(c, dtype):
    """What shares a lane, a run or a tile with a NaN has the bits that it has without it."""
    t, dt = 700, DT[dtype]
    starts = torch.tensor([0, 200, 450, 600], dtype=torch.int64).cuda()
    x, f = (v[0] for v in views(1, t, c, dt, "plain", 29))
    dy, h0, dh = rand((t, c), 30).to(dt).cuda(), rand((3, c), 31).float().cuda(), rand((3, c), 32).float().cuda()

    def run(x, f, dy):
        scan = zb.GatedScan(1, t, c)
        y, last, kept = scan.forward(x, f, h0, starts, keep=True)
        dx, df, dh0 = scan.backward(x, f, dy, kept, h0, dh, starts)
        return [v[:600] for v in (y, dx, df)] + [last, kept[0], dh0]

    want = run(x, f, dy)
    for planted, (at, ch) in ((f, (300, 4)), (f, (0, 0)), (f, (211, 8)), (x, (303, 1)), (dy, (333, 12)), (f, (202, 3)),
                              (f, (449, 0)), (f, (320, 32))):
        was = planted[at, ch].clone()
        planted[at, ch] = math.nan
        got = run(x, f, dy)
        planted[at, ch] = was
        others = torch.arange(c, device="cuda") != ch
        for g, w in zip(got, want):
            assert torch.equal(g[:, others], w[:, others]), (at, ch)


def packed_starts(t, seed):
    """Sequences within a run of tokens, across runs, warps and chunks, and empty ones."""
    cuts, at = [0, 7, 9, 9, 18, 33, 128, 128, 140, 267, 300, 300, 301], 301
    rng = np.random.default_rng(seed)
    while at < t - 1:
        at = min(t - 1, at + int(rng.integers(1, 300)))
        cuts.append(at)
    return [c for c in cuts if c < t] + [t]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t,c", [(300, 66), (1500, 771), (5000, 64), (700, 8256)])
def test_packed_states_updated_in_place(t, c, dtype):
    """h_last in h0's own memory: the same bits as apart, wherever a sequence begins and ends."""
    starts = packed_starts(t, t + c)
    x, f = (v[0] for v in views(1, t, c, DT[dtype], "plain", 83))
    seq_start = torch.tensor(starts, dtype=torch.int64).cuda()
    h0 = rand((len(starts) - 1, c), 84, 50.0).float().cuda()
    scan = zb.GatedScan(1, t, c)
    y, last, kept = scan.forward(x, f, h0, seq_start, keep=True)
    for _ in range(3):
        state = h0.clone()
        y2, last2, kept2 = scan.forward(x, f, state, seq_start, keep=True, h_last=state)
        assert last2 is state
        for got, want in ((y2, y), (state, last), (kept2, kept)):
            assert torch.equal(got, want)
    assert scan.status() == zb.ZG_OK


def backward_in_place(scan, x, f, dy, kept, h0, d, seq_start):
    """The C call with dh0 in dh_last's memory, ``d``; (tokens, channels) or (batch, tokens, channels)."""
    import ctypes

    dt = zb.ZG_DTYPE_BF16 if x.dtype is torch.bfloat16 else zb.ZG_DTYPE_F32
    b, t, c = (1, *x.shape) if x.dim() == 2 else x.shape
    shape = zb._ScanShape(b, t, c, None if seq_start is None else seq_start.data_ptr(), d.shape[0], dt)
    view = lambda v: ctypes.byref(zb._View(v.data_ptr(), v.stride(0) if v.dim() == 3 else 0, v.stride(-2)))  # noqa: E731
    dx, df = torch.empty_like(x), torch.empty_like(x)
    assert zb.lib().zg_gated_scan_bwd(scan.handle, ctypes.byref(shape), view(x), view(f), view(dy), kept.data_ptr(),
                                      h0.data_ptr(), d.data_ptr(), view(dx), view(df), d.data_ptr(),
                                      torch.cuda.current_stream().cuda_stream) == 0
    return dx, df


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t,c", [(300, 66), (1500, 771), (5000, 64), (700, 8256)])
def test_packed_gradients_of_states_in_place(t, c, dtype):
    """dh0 in dh_last's own memory: the same bits as apart."""
    starts = packed_starts(t, t + c)
    x, f = (v[0] for v in views(1, t, c, DT[dtype], "plain", 85))
    dy = rand((t, c), 86).to(DT[dtype]).cuda()
    seq_start = torch.tensor(starts, dtype=torch.int64).cuda()
    h0, dh = (rand((len(starts) - 1, c), s, 50.0).float().cuda() for s in (87, 88))
    scan = zb.GatedScan(1, t, c)
    _, _, kept = scan.forward(x, f, h0, seq_start, keep=True)
    want = scan.backward(x, f, dy, kept, h0, dh, seq_start)
    for _ in range(3):
        d = dh.clone()
        got = (*backward_in_place(scan, x, f, dy, kept, h0, d, seq_start), d)
        for p, q in zip(got, want):
            assert torch.equal(p, q)
    assert scan.status() == zb.ZG_OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("b,t,c", [(2, 9, 70), (2, 100, 66), (1, 5000, 130), (3, 700, 4160)])
def test_rows_in_place(b, t, c, dtype):
    """States and their gradients in place, in rows of few and of many chunks."""
    x, f = views(b, t, c, DT[dtype], "plain", 89)
    dy = rand((b, t, c), 90).to(DT[dtype]).cuda()
    h0, dh = (rand((b, c), s, 50.0).float().cuda() for s in (91, 92))
    scan = zb.GatedScan(b, t, c)
    y, last, kept = scan.forward(x, f, h0, keep=True)
    want = scan.backward(x, f, dy, kept, h0, dh)
    for _ in range(3):
        state, d = h0.clone(), dh.clone()
        y2, _, kept2 = scan.forward(x, f, state, keep=True, h_last=state)
        for p, q in zip((y2, state, kept2, *backward_in_place(scan, x, f, dy, kept, h0, d, None), d), (y, last, kept, *want)):
            assert torch.equal(p, q)
    assert scan.status() == zb.ZG_OK


def test_a_new_handle_on_a_stream_that_waits_for_nothing():
    """The handle's workspace is ready when it is made, whatever the default stream is busy with."""
    b, t, c = 2, 1500, 130
    x, f = views(b, t, c, torch.bfloat16, "plain", 93)
    want = zb.GatedScan(b, t, c).forward(x, f)[0]
    side = torch.cuda.Stream()  # does not wait for the default stream
    torch.cuda.synchronize()
    for _ in range(20):
        torch.cuda._sleep(20_000_000)  # some 10 ms on the default stream
        scan = zb.GatedScan(b, t, c)
        with torch.cuda.stream(side):
            got = scan.forward(x, f)[0]
        assert scan.status(side) == zb.ZG_OK
        assert torch.equal(got, want)
    torch.cuda.synchronize()


def test_a_wait_that_ran_out_does_not_concern_the_next_scan():
    """Whether the status has been asked for or not: it is kept for the asking, and no more."""
    b, t, c = 1, 40000, 130
    x, f = views(b, t, c, torch.bfloat16, "plain", 95)
    dy = rand((b, t, c), 96).to(torch.bfloat16).cuda()
    scan = zb.GatedScan(b, t, c)
    y, _, kept = scan.forward(x, f, keep=True)
    want = (y, *scan.backward(x, f, dy, kept))
    assert scan.status() == zb.ZG_OK
    for _ in range(5):
        scan.set_wait_limit(0)
        scan.forward(x, f)
        scan.set_wait_limit(4000000)
        got = (scan.forward(x, f)[0], *scan.backward(x, f, dy, kept))
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        assert scan.status() == zb.ZG_ERR_DEVICE_TIMEOUT
        assert scan.status() == zb.ZG_OK


def remember_nan(shape, dtype, n=8):
    """Leaves NaNs in the memory that the next allocations of this size are given."""
    kept = [torch.full(shape, math.nan, dtype=dtype, device="cuda") for _ in range(n)]
    torch.cuda.synchronize()
    del kept


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t,end,c", [(5, 4, 67), (300, 290, 64), (300, 0, 68), (1100, 130, 71), (700, 513, 8256), (260, 257, 8257)])
def test_outputs_past_the_last_sequence_are_zero(t, end, c, dtype):
    """What forward and backward allocate is whole: a weight's gradient multiplies all its rows."""
    dt = DT[dtype]
    x, f = (v[0] for v in views(1, t, c, dt, "plain", 97))
    dy = rand((t, c), 98).to(dt).cuda()
    x[end:], f[end:], dy[end:] = math.nan, math.nan, math.nan
    starts = torch.tensor([0, end // 2, end], dtype=torch.int64).cuda()
    scan = zb.GatedScan(1, t, c)
    remember_nan((t, c), dt)
    y, _, kept = scan.forward(x, f, None, starts, keep=True)
    dx, df, _ = scan.backward(x, f, dy, kept, None, None, starts)
    for got in (y, dx, df):
        assert bool((got[end:] == 0).all()) and bool(torch.isfinite(got).all())
    # and the rest has the bits that it has in the caller's own memory, whose tail stays
    mine = [torch.full((t, c), 7.0, dtype=dt, device="cuda") for _ in range(3)]
    scan.forward(x, f, None, starts, out=mine[0])
    scan.backward(x, f, dy, kept, None, None, starts, out=(mine[1], mine[2]))
    for got, want in zip(mine, (y, dx, df)):
        assert torch.equal(got[:end], want[:end]) and bool((got[end:] == 7.0).all())


def test_outputs_belong_to_the_given_stream():
    """What a call allocates is of the stream that it is given, as under torch.cuda.stream: memory
    given back goes to that stream's calls, not to the current one's while the other still writes."""
    b, t, c = 2, 300, 64
    x, f = views(b, t, c, torch.bfloat16, "plain", 99)
    scan = zb.GatedScan(b, t, c)
    y, last, kept = scan.forward(x, f, keep=True)
    want = [y, last, kept, *scan.backward(x, f, x, kept), *scan.step(x[:, 0], f[:, 0], last)]
    z = rand((40, 1003), 100).to(torch.bfloat16).cuda()
    values, index = zb.topk_logits(z, 20)
    loss, lse = zb.distill_loss(z, values, index, 1.0)
    want += [values, index, loss, lse, zb.distill_grad(z, lse, values, index, 1.0), *zb.distill_loss_grad(z, values, index, 1.0)]
    torch.cuda.synchronize()
    for side in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        got = [*scan.forward(x, f, keep=True, stream=side), *scan.backward(x, f, x, kept, stream=side),
               *scan.step(x[:, 0], f[:, 0], last, stream=side), *zb.topk_logits(z, 20, stream=side),
               *zb.distill_loss(z, values, index, 1.0, stream=side),
               zb.distill_grad(z, lse, values, index, 1.0, stream=side),
               *zb.distill_loss_grad(z, values, index, 1.0, stream=side)]
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want)) and len(got) == len(want)
        sizes = [(v.numel() * v.element_size(), v.data_ptr()) for v in got]
        del got
        for size, ptr in sizes:  # none of it is handed out for the current stream
            assert torch.empty(size, dtype=torch.uint8, device="cuda").data_ptr() != ptr
    # and the default stream by its address
    got = scan.forward(x, f, stream=0)[0]
    torch.cuda.synchronize()
    assert torch.equal(got, y)
