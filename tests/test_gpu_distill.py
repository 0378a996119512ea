"""The teacher's top logits and the distillation loss with its gradient,
against a stable sort and the formulas in 64 bits."""
import math

import numpy as np
import pytest
import torch

import operators_ref as ref
from gpu_helpers import Guarded
from zero_sharded_mixed_flat_gb300 import binding as zb

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def rand(shape, seed, scale=1.0):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape) * scale)


def logits_of(n, v, dtype, seed, pad=0, offset=0, scale=2.5):
    """Row-strided logits whose first element is ``offset`` elements off the allocation's alignment."""
    flat = torch.zeros(offset + n * (v + pad), dtype=dtype)
    z = flat[offset:].view(n, v + pad)[:, :v]
    z.copy_(rand((n, v), seed, scale).to(dtype))
    return flat.cuda()[offset:].view(n, v + pad)[:, :v]


# ------------------------------------------------------------------ top-k

def top_by_sort(z, k):
    """Stable descending sort of -0 = +0 values with NaNs first."""
    key = z.double().cpu() + 0.0
    key = torch.where(torch.isnan(key), torch.full_like(key, math.nan), key)
    order = torch.sort(torch.where(torch.isnan(key), torch.full_like(key, 1e300), torch.clamp(key, -1e290, 1e290)),
                       dim=1, descending=True, stable=True).indices[:, :k]
    return order


def check_top(z, k):
    values, index = zb.topk_logits(z, k)
    want = top_by_sort(z, k)
    assert index.dtype == torch.int32 and values.dtype == z.dtype
    assert torch.equal(index.cpu().long(), want)
    bits = torch.int16 if z.dtype is torch.bfloat16 else torch.int32
    # gathered as whole numbers: a NaN's bits need not survive a gather of floats on the host
    assert torch.equal(values.view(bits).cpu(), z.contiguous().view(bits).cpu().gather(1, want))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,v,k", [(1, 1, 1), (2, 2, 2), (3, 7, 3), (2, 33, 33), (5, 256, 256), (4, 257, 256), (3, 1000, 100),
                                   (2, 4099, 17), (7, 50257, 64), (300, 2001, 8), (2, 131075, 256), (1, 262147, 1),
                                   (200, 50257, 50)])
def test_topk_sizes(n, v, k, dtype):
    check_top(logits_of(n, v, DT[dtype], n + v + k), k)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,offset", [(1, 0), (0, 1), (3, 5), (47, 2)])
def test_topk_strides_and_alignment(pad, offset, dtype):
    check_top(logits_of(5, 5003, DT[dtype], 3, pad, offset), 40)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("v", [300, 5001, 50257, 140001])
def test_topk_ties_and_orders(v, dtype):
    dt = DT[dtype]
    ramp = torch.arange(v, dtype=torch.float64)
    rows = [torch.zeros(v), ramp / v, -ramp / v, (ramp % 3), torch.full((v,), -math.inf),
            torch.where(ramp % 2 == 0, 0.0, -0.0), torch.where(ramp < 20, -math.inf, ramp * 0 - 5.0),
            torch.where(ramp == v - 1, math.inf, ramp * 0), torch.where(ramp % 97 == 5, math.nan, ramp % 11),
            torch.where(ramp % 2 == 0, math.nan, -math.inf), (ramp * 7919 % 101) - 50, ramp.flip(0) ** 2 - 1e6,
            torch.where(ramp < 100, 3.0, torch.where(ramp >= v - 100, 3.0, 1.0)), ramp * 1e-40, ramp * 1e34 - 1e38]
    z = torch.stack([r.to(torch.float64) for r in rows]).to(dt).cuda()
    z[8, 5] = -z[8, 5]  # a NaN with its sign set
    for k in (1, 37, 256):
        check_top(z, k)


def test_topk_wide_rows_of_one_value_range():
    """Many more values at the threshold than any list could hold."""
    z = (rand((6, 60001), 5).sign() * 2).to(torch.bfloat16).cuda()
    check_top(z, 200)
    z = (rand((6, 120001), 6) * 0.25).round().float().cuda()
    check_top(z, 256)


def test_topk_only_writes_its_outputs():
    n, v, k = 3, 1001, 33
    z = logits_of(n, v, torch.float32, 9)
    vals, idx = Guarded(n * k, torch.float32), Guarded(n * k, torch.int32)
    assert zb.lib().zg_topk(z.data_ptr(), zb.ZG_DTYPE_F32, n, v, v, k, vals.view.data_ptr(), idx.view.data_ptr(),
                            torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert vals.intact() and idx.intact()
    assert torch.equal(idx.view.view(n, k).cpu().long(), top_by_sort(z, k))


# ------------------------------------------------------------------ distillation

def teacher(n, v, k, dtype, seed, ragged=True):
    rng = np.random.default_rng(seed)
    index = np.stack([rng.permutation(v)[:k] if v >= k else rng.integers(0, v, k) for _ in range(n)]).astype(np.int32)
    t = (rng.standard_normal((n, k)) * 2 + 3)
    if ragged:
        for r in range(n):
            if r % 3 == 1:
                index[r, rng.integers(0, k):] = -1
            if r % 5 == 4:
                index[r] = -1
    return torch.from_numpy(t).to(dtype).cuda(), torch.from_numpy(index).cuda()


def check_distill(z, t, index, temperature, scale=64.0, weights=True):
    n, v = z.shape
    dloss = rand(n, 77).abs().float() if weights else None
    want = ref.distill(z.double().cpu(), t.double().cpu(), index.cpu(), temperature, scale,
                       None if dloss is None else dloss.double())
    loss, lse, grad, loss_err, lse_err, grad_err = want
    d = None if dloss is None else dloss.cuda()
    got_loss, got_lse = zb.distill_loss(z, t, index, temperature)
    f32 = torch.float32
    ref.check(got_loss, loss, ref.stored(loss, loss_err, f32), "loss")
    ref.check(got_lse, lse, ref.stored(lse, lse_err, f32), "lse")
    err = ref.stored(grad, grad_err, z.dtype)
    ref.check(zb.distill_grad(z, got_lse, t, index, temperature, scale, d), grad, err, "grad")
    one_loss, one = zb.distill_loss_grad(z, t, index, temperature, scale, d)
    ref.check(one_loss, loss, ref.stored(loss, loss_err, f32), "loss of both")
    ref.check(one, grad, err, "grad of both")
    again_loss, again = zb.distill_loss_grad(z, t, index, temperature, scale, d)
    assert torch.equal(one, again) and torch.equal(one_loss, again_loss)
    # in the logits' own memory
    mine = torch.empty_strided(z.shape, z.stride(), dtype=z.dtype, device="cuda").copy_(z)
    _, out = zb.distill_loss_grad(mine, t, index, temperature, scale, d, out=mine)
    assert out is mine and torch.equal(mine, one)
    mine.copy_(z)
    assert torch.equal(zb.distill_grad(mine, got_lse, t, index, temperature, scale, d, out=mine),
                       zb.distill_grad(z, got_lse, t, index, temperature, scale, d))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,v,k", [(1, 1, 1), (2, 2, 2), (3, 7, 3), (2, 31, 31), (6, 257, 256), (7, 1000, 64), (5, 4099, 100),
                                   (6, 50257, 64), (400, 1003, 5), (2, 131075, 32), (1, 262147, 256), (160, 50257, 20)])
def test_distill_sizes(n, v, k, dtype):
    t, index = teacher(n, v, k, DT[dtype], n + v)
    check_distill(logits_of(n, v, DT[dtype], n * 7 + v), t, index, 2.0)


@pytest.mark.parametrize("dtype,t_dtype", [("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("temperature", [0.5, 1.0, 1.7, 20.0])
def test_distill_types_and_temperatures(dtype, t_dtype, temperature):
    t, index = teacher(6, 3001, 40, DT[t_dtype], 3)
    check_distill(logits_of(6, 3001, DT[dtype], 4), t, index, temperature, weights=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,offset", [(1, 0), (0, 1), (3, 5), (47, 2)])
def test_distill_strides_and_alignment(pad, offset, dtype):
    t, index = teacher(5, 5003, 40, DT[dtype], 3)
    z = logits_of(5, 5003, DT[dtype], 5, pad, offset)
    check_distill(z, t, index, 2.0)
    # an output whose rows sit differently from the logits'
    want = zb.distill_loss_grad(z, t, index, 2.0)[1]
    out = logits_of(5, 5003, DT[dtype], 6, pad + 1, offset + 2)
    zb.distill_loss_grad(z, t, index, 2.0, out=out)
    assert torch.equal(out, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("v", [90, 5003, 50257])
def test_distill_repeated_and_absent_entries(v, dtype):
    z = logits_of(5, v, DT[dtype], 11)
    t, index = teacher(5, v, 60, DT[dtype], 12, ragged=False)
    index[:, 10:40] = index[:, 9:10]      # thirty times the same index
    index[:, 40] = v                      # past the vocabulary: absent
    index[:, 41] = -7
    index[:, 42] = 2 ** 31 - 1
    index[1] = index[1, 0]                # one index alone
    t[2, 5:50] = -math.inf
    check_distill(z, t, index, 2.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("v", [90, 5003, 50257])
def test_distill_empty_rows_do_not_look_at_their_logits(v, dtype):
    z = logits_of(4, v, DT[dtype], 13)
    t, index = teacher(4, v, 30, DT[dtype], 14, ragged=False)
    index[1] = -1
    z[1] = math.nan
    t[3] = -math.inf
    z[3, 5:] = math.inf
    check_distill(z, t, index, 2.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("v", [90, 5003, 50257])
def test_distill_masked_and_extreme_logits(v, dtype):
    z = logits_of(6, v, DT[dtype], 15)
    t, index = teacher(6, v, 30, DT[dtype], 16, ragged=False)
    free = torch.ones(v, dtype=torch.bool)
    free[index[0].long().cpu()] = False
    z[0, free.cuda()] = -math.inf         # only the teacher's entries are left
    z[1, :] = torch.finfo(DT[dtype]).min  # all at the type's lowest value: a uniform row
    z[2] *= 1000                          # one logit takes it all
    z[3, : v // 2] = torch.finfo(DT[dtype]).min
    z[3, index[3].long()] = 1.0
    z[4] = 0
    t[5, 3:] = torch.finfo(DT[dtype]).min / 4
    check_distill(z, t, index, 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("v", [90, 50257])
def test_distill_non_finite_rows_say_so_and_stay_alone(v, dtype):
    """A NaN or +inf in a live row makes that row's loss and gradient NaN, and no other's."""
    z = logits_of(6, v, DT[dtype], 17)
    t, index = teacher(6, v, 30, DT[dtype], 18, ragged=False)
    clean_loss, clean = zb.distill_loss_grad(z, t, index, 2.0)
    z[1, v - 1] = math.nan
    z[3, 7] = math.inf
    t[5, 2] = math.nan
    loss, grad = zb.distill_loss_grad(z, t, index, 2.0)
    only, lse = zb.distill_loss(z, t, index, 2.0)
    two = zb.distill_grad(z, lse, t, index, 2.0)
    for r in range(6):
        if r in (0, 2, 4):
            assert torch.equal(loss[r], clean_loss[r]) and torch.equal(grad[r], clean[r])
        else:
            assert bool(torch.isnan(loss[r])) and bool(torch.isnan(only[r]))
            assert bool(torch.isnan(grad[r]).any()) and bool(torch.isnan(two[r]).any())
    assert bool(torch.isnan(grad[1]).all()) and bool(torch.isnan(two[1]).all())
    # the teacher gives weight to a logit that is masked out: an infinite loss
    z = logits_of(1, v, DT[dtype], 19)
    t, index = teacher(1, v, 3, DT[dtype], 20, ragged=False)
    z[0, index[0, 0].long()] = -math.inf
    assert float(zb.distill_loss(z, t, index, 2.0)[0]) == math.inf
    assert bool(torch.isfinite(zb.distill_loss_grad(z, t, index, 2.0)[1]).all())


def test_distill_gradient_against_differences():
    v = 301
    z = logits_of(3, v, torch.float32, 21)
    t, index = teacher(3, v, 20, torch.float32, 22, ragged=False)
    w = rand(3, 23).float()
    _, grad = zb.distill_loss_grad(z, t, index, 1.5, 3.0, w.cuda())
    d, step = rand((3, v), 24), 1e-5

    def value(sign):
        zz = z.double().cpu() + sign * step * d
        return 3.0 * float((ref.distill(zz, t.double().cpu(), index.cpu(), 1.5)[0] * w.double()).sum())

    slope = (value(1) - value(-1)) / (2 * step)
    mine = (grad.double().cpu() * d)
    assert abs(slope - float(mine.sum())) <= 1e-5 * float(mine.abs().sum())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("v", [37, 5003, 50257, 131075])
def test_distill_only_writes_its_outputs(v, dtype):
    n, k, dt = 3, 20, DT[dtype]
    z = logits_of(n, v, dt, 25)
    t, index = teacher(n, v, k, dt, 26)
    grad, loss = Guarded(n * v, dt), Guarded(n, torch.float32)
    a = zb._distill(z, t, index, 2.0)
    import ctypes
    assert zb.lib().zg_distill_loss_grad(ctypes.byref(a), 1.0, None, loss.view.data_ptr(), None, grad.view.data_ptr(), v,
                                         torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert grad.intact() and loss.intact()
    # padding columns between rows keep theirs
    out = torch.full((n, v + 3), 7.0, dtype=dt, device="cuda")
    zb.distill_loss_grad(z, t, index, 2.0, out=out[:, :v])
    assert bool((out[:, v:] == 7.0).all())
    assert torch.equal(out[:, :v], grad.view.view(n, v))


def test_teacher_to_student():
    """What topk_logits selects is what distill_loss takes; a student equal to
    its teacher pays only for the mass outside the selection."""
    z = logits_of(4, 5003, torch.float32, 27)
    t, index = zb.topk_logits(z, 50)
    loss, _ = zb.distill_loss(z, t, index, 1.0)
    inside = torch.softmax(z.double(), 1).gather(1, index.long()).sum(1)
    assert torch.allclose(loss.double(), -torch.log(inside), rtol=1e-5)


def test_no_rows_is_nothing_to_do():
    z = torch.empty(0, 100, dtype=torch.bfloat16, device="cuda")
    t, index = torch.empty(0, 5, device="cuda"), torch.empty(0, 5, dtype=torch.int32, device="cuda")
    assert zb.topk_logits(z, 5)[0].shape == (0, 5)
    assert zb.distill_loss(z, t, index, 1.0)[0].shape == (0,)
    assert zb.distill_loss_grad(z, t, index, 1.0)[1].shape == (0, 100)


def test_another_stream_and_graph_replay():
    z = logits_of(20, 5003, torch.bfloat16, 29)
    t, index = teacher(20, 5003, 30, torch.bfloat16, 30)
    want = zb.distill_loss_grad(z, t, index, 2.0)
    top = zb.topk_logits(z, 30)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = zb.distill_loss_grad(z, t, index, 2.0)
        got_top = zb.topk_logits(z, 30)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip((*got, *got_top), (*want, *top)))
    s = torch.zeros_like(z)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = (*zb.distill_loss_grad(s, t, index, 2.0), *zb.topk_logits(s, 30))
    s.copy_(z)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(kept, (*want, *top)))


def test_refusals():
    z = torch.zeros(4, 100, dtype=torch.bfloat16, device="cuda")
    t, index = torch.zeros(4, 5, device="cuda"), torch.zeros(4, 5, dtype=torch.int32, device="cuda")
    with pytest.raises(zb.ZgError, match="k must be in"):
        zb.topk_logits(z, 0)
    with pytest.raises(zb.ZgError, match="k must be in"):
        zb.topk_logits(torch.zeros(1, 1000, device="cuda"), 257)
    with pytest.raises(zb.ZgError, match="more than vocab"):
        zb.topk_logits(z, 101)
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        zb.topk_logits(z.half(), 3)
    with pytest.raises(ValueError, match="contiguous"):
        zb.topk_logits(z.t(), 3)
    for bad in (0.0, -1.0, math.nan, math.inf, 1e-45):
        with pytest.raises(zb.ZgError, match="temperature"):
            zb.distill_loss(z, t, index, bad)
    with pytest.raises(zb.ZgError, match="scale"):
        zb.distill_loss_grad(z, t, index, 1.0, math.inf)
    with pytest.raises(TypeError, match="t_index must have dtype"):
        zb.distill_loss(z, t, index.long(), 1.0)
    with pytest.raises(ValueError, match="t_index must have shape"):
        zb.distill_loss(z, t, index[:, :4], 1.0)
    with pytest.raises(ValueError, match="dloss must have shape"):
        zb.distill_loss_grad(z, t, index, 1.0, 1.0, torch.zeros(3, device="cuda"))
    with pytest.raises(zb.ZgError, match="row_stride"):
        zb.distill_loss(z[:1].expand(4, 100), t, index, 1.0)
    with pytest.raises(ValueError, match="out must have shape"):
        zb.distill_loss_grad(z, t, index, 1.0, out=z[:, :50])


def check_rows_like(z, same, t, index, temperature, only_both=False):
    """The outputs for z against the formulas for ``same``: logits with the same
    probabilities (masked ones at -inf, or all moved by one number), whose smaller
    values give the tight bounds. ``only_both``: not what goes through lse, which is
    held to the formulas for z itself."""
    d = rand(z.shape[0], 78).abs().float()
    loss, lse, grad, loss_err, lse_err, grad_err = ref.distill(same, t.double().cpu(), index.cpu(), temperature, 64.0, d.double())
    err, f32 = ref.stored(grad, grad_err, z.dtype), torch.float32
    one_loss, one = zb.distill_loss_grad(z, t, index, temperature, 64.0, d.cuda())
    ref.check(one_loss, loss, ref.stored(loss, loss_err, f32), "loss of both")
    ref.check(one, grad, err, "grad of both")
    got_loss, got_lse = zb.distill_loss(z, t, index, temperature)
    ref.check(got_loss, loss, ref.stored(loss, loss_err, f32), "loss")
    if only_both:
        _, lse, grad, _, lse_err, grad_err = ref.distill(z.double().cpu(), t.double().cpu(), index.cpu(), temperature, 64.0,
                                                         d.double())
        err = ref.stored(grad, grad_err, z.dtype)
    ref.check(got_lse, lse, ref.stored(lse, lse_err, f32), "lse")
    ref.check(zb.distill_grad(z, got_lse, t, index, temperature, 64.0, d.cuda()), grad, err, "grad")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("temperature", [0.1, 0.25, 1.0, 2.0])
@pytest.mark.parametrize("v", [90, 5003, 50257])
def test_distill_finite_masks(v, temperature, dtype):
    """Logits closed by a large finite number count for nothing, whatever the number and
    however many a thread meets before its first open one."""
    dt, lowest = DT[dtype], torch.finfo(DT[dtype]).min
    t, index = teacher(6, v, 30, dt, 31, ragged=False)
    at = torch.arange(v)
    shut = torch.stack([at < v // 2, at >= v // 2, at % 16 < 8, at % 7 != 3, torch.ones(v, dtype=torch.bool), at < 0])
    shut.scatter_(1, index.long().cpu(), False)  # the teacher's entries stay open
    z = logits_of(6, v, dt, 32)
    same = torch.where(shut, -math.inf, z.double().cpu())
    for mask in (-1e4, -1e9, -1e10, -1e12, -1e15, -1e20, -1e29, lowest):
        check_rows_like(z.masked_fill(shut.cuda(), mask), same, t, index, temperature)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_distill_finite_masks_in_many_rows(dtype):
    """The same with a block to a row."""
    n, v, dt = 610, 20011, DT[dtype]
    t, index = teacher(n, v, 20, dt, 33)
    shut = torch.arange(v).expand(n, v) < (torch.arange(n) * 37 % v)[:, None]
    shut = shut.scatter(1, index.long().clamp(min=0).cpu(), False)
    z = logits_of(n, v, dt, 34)
    same = torch.where(shut, -math.inf, z.double().cpu())
    for mask in (-1e10, -1e20):
        check_rows_like(z.masked_fill(shut.cuda(), mask), same, t, index, 1.0)


@pytest.mark.parametrize("temperature", [0.5, 2.0])
@pytest.mark.parametrize("v", [90, 5003, 50257])
def test_distill_rows_far_from_zero(v, temperature):
    """A row moved by one number has the same probabilities, and so the same loss and, in
    one pass, the same gradient: neither goes through the log-sum-exp, whose last place
    grows with the move."""
    t, index = teacher(6, v, 30, torch.float32, 35, ragged=False)
    for move in (3e3, 1e5, -1e6, -1e10, 1e15, -1e30):
        z = (logits_of(6, v, torch.float32, 36) + move).contiguous()
        z[5] = move  # uniform
        same = z.double().cpu() - z.double().cpu().max(1, keepdim=True).values
        check_rows_like(z, same, t, index, temperature, only_both=True)
    z = torch.full((6, v), torch.finfo(torch.bfloat16).min, dtype=torch.bfloat16, device="cuda")
    d = torch.ones(6, device="cuda")
    want = ref.distill(torch.zeros(6, v, dtype=torch.float64), t.double().cpu(), index.cpu(), temperature)
    ref.check(zb.distill_loss_grad(z, t, index, temperature, 1.0, d)[1], want[2], ref.stored(want[2], want[5], torch.bfloat16))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,v", [(3, 90), (3, 50257), (200, 20011)])
def test_distill_gradient_of_rows_far_from_zero_in_place(n, v, dtype):
    """Where lse does not do, the row is read twice, and its own memory is written over after that."""
    dt = DT[dtype]
    t, index = teacher(n, v, 20, dt, 37)
    z = logits_of(n, v, dt, 38)
    z[::2] = -1e10
    loss, lse = zb.distill_loss(z, t, index, 1.0)
    want = zb.distill_grad(z, lse, t, index, 1.0)
    mine = z.clone()
    assert zb.distill_grad(mine, lse, t, index, 1.0, out=mine) is mine
    assert torch.equal(mine, want) and bool(torch.isfinite(want).all())
