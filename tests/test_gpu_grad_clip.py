"""The common norm of many gradients and their clipping, against the formulas in 64 bits."""
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
EPS = 1e-6


def grads_of(sizes, dtype, seed, scale=1.0, offset=0):
    rng = np.random.default_rng(seed)
    out = []
    for i, n in enumerate(sizes):
        dt = DT[("bf16", "f32")[i % 2]] if dtype == "mixed" else DT[dtype]
        flat = torch.empty(n + offset, dtype=dt, device="cuda")
        flat[offset:].copy_(torch.from_numpy(rng.standard_normal(n) * scale))
        out.append(flat[offset:])
    return out


def bound(want, rel, dtype):
    # the coefficient has the norm's error, and takes two roundings with its product
    return ref.stored(want, want.abs() * (rel + 4 * ref.ULP), dtype)


def check(grads, outs, stats, host, scale, max_norm, eps=EPS):
    norm, coef, want, rel = ref.clip(host, scale, max_norm, eps)
    got = stats.double().cpu()
    assert abs(float(got[0]) - float(norm)) <= (rel + ref.ULP) * float(norm) + ref.TINY
    assert abs(float(got[1]) - float(coef)) <= (rel + 2 * ref.ULP) * float(coef)
    for o, w in zip(outs, want):
        ref.check(o.reshape(-1), w.reshape(-1), bound(w.reshape(-1), rel, o.dtype), "clipped")


SIZES = [[1], [7, 1, 3], [16384], [16385, 16383], [100000, 3, 0, 77, 40000], [5] * 300, [1 << 20, 13, 333333]]


@pytest.mark.parametrize("dtype", ["bf16", "f32", "mixed"])
@pytest.mark.parametrize("offset", [0, 1, 3])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
def test_clip(sizes, offset, dtype):
    grads = grads_of(sizes, dtype, 1, offset=offset)
    host = [g.cpu() for g in grads]
    norm = float(ref.clip(host, 0.25, 1.0, EPS)[0])
    for flat_dtype in DT.values():
        for max_norm in (0.5 * norm, 2.0 * norm):
            flat = torch.full((sum(sizes) + 9,), 7.0, dtype=flat_dtype, device="cuda")
            plan = zb.GradClip(grads, out=flat)
            stats = plan.clip(max_norm, EPS, 0.25)
            check(grads, flat[:sum(sizes)].split(sizes), stats, host, 0.25, max_norm)
            assert bool((flat[sum(sizes):] == 7.0).all())
            assert torch.equal(plan.norm(0.25)[:1], stats[:1]) and float(plan.norm(0.25)[1]) == 1.0
    assert all(torch.equal(g.cpu(), h) for g, h in zip(grads, host))
    # where they are, and into a list of others
    others = [torch.empty(n, device="cuda") for n in sizes]
    check(grads, others, zb.GradClip(grads, out=others).clip(0.5 * norm, EPS, 0.25), host, 0.25, 0.5 * norm)
    stats = zb.GradClip(grads).clip(0.5 * norm, EPS, 0.25)
    check(grads, grads, stats, host, 0.25, 0.5 * norm)


def test_shapes_stay_and_outputs_are_written_alone():
    grads = [g.view(4, -1) for g in grads_of([40, 4000], "mixed", 2)]
    out = Guarded(4040, torch.bfloat16)
    plan = zb.GradClip(grads, out=out.view)
    plan.clip(0.1)
    torch.cuda.synchronize()
    assert out.intact()
    check(grads, out.view.split([40, 4000]), plan.clip(0.1), [g.cpu() for g in grads], 1.0, 0.1)


def test_the_list_reads_what_is_there_at_the_call():
    grads = grads_of([1000, 50], "f32", 3)
    plan = zb.GradClip(grads)
    first = float(plan.norm()[0])
    grads[0].mul_(3)
    assert abs(float(plan.norm()[0]) - float(torch.cat(grads).double().norm())) <= 1e-5 * first


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_non_finite_gradients_pass_unclipped(dtype):
    for bad in (math.inf, -math.inf, math.nan):
        grads = grads_of([3000, 20, 70000], dtype, 4)
        grads[2][69999] = bad
        host = [g.cpu() for g in grads]
        flat = torch.empty(73020, dtype=DT[dtype], device="cuda")
        stats = zb.GradClip(grads, out=flat).clip(0.5, EPS, 0.5)
        assert not math.isfinite(float(stats[0])) and float(stats[1]) == 1.0
        for got, h in zip(flat.split([3000, 20, 70000]), host):
            assert torch.equal(torch.nan_to_num(got.cpu(), 123.0), torch.nan_to_num(h * 0.5, 123.0))
    # finite values whose squares are not
    grads = grads_of([100], dtype, 5, 1e30)
    assert float(zb.GradClip(grads).norm()[0]) == math.inf


@pytest.mark.parametrize("dtype", ["bf16", "f32", "mixed"])
@pytest.mark.parametrize("size", [1e20, 1e30, 1e35, 1e-19, 1e-20, 1e-25, 1e-30])
def test_finite_gradients_of_any_size_are_clipped(size, dtype):
    """Squares that overflow binary32, or vanish in it, of all elements and of one."""
    sizes = [3000, 20, 70000]
    every = grads_of(sizes, dtype, 8, size, offset=1)
    one = grads_of(sizes, dtype, 9, 1e-3 if size > 1 else 0.0, offset=1)
    one[2][40001] = -size
    for grads in (every, one):
        host = [g.cpu() for g in grads]
        for scale in (0.25, 1.0):
            norm = float(ref.clip(host, scale, 1.0, 0.0)[0])
            for max_norm in (norm / 2, 2 * norm):
                flat = torch.empty(sum(sizes), dtype=torch.float32, device="cuda")
                stats = zb.GradClip(grads, out=flat).clip(max_norm, 0.0, scale)
                check(grads, flat.split(sizes), stats, host, scale, max_norm, 0.0)
            if size < 1:
                assert abs(float(zb.GradClip(grads).norm(scale)[0]) - norm) <= (ref.DEEP + ref.ULP) * norm


def test_one_exploded_element_of_a_long_list():
    """As many parts as take the sums' own launch."""
    g = grads_of([34_000_000, 7], "bf16", 10, 1e-3)
    g[0][33_999_999] = 1e30
    host, flat = [t.cpu() for t in g], torch.empty(34_000_007, dtype=torch.bfloat16, device="cuda")
    check(g, flat.split([34_000_000, 7]), zb.GradClip(g, out=flat).clip(1.0), host, 1.0, 1.0)
    assert float(flat.float().abs().max()) == 1.0


def test_a_norm_beyond_binary32():
    g = torch.full((100,), 3e38, device="cuda")
    h = g.double()
    stats = zb.GradClip([g]).clip(1e3)  # norm 3e39
    assert float(stats[0]) == math.inf
    coef = 1e3 / float(h.norm())
    assert abs(float(stats[1]) - coef) <= 4 * ref.ULP * coef
    assert float(((g - h * coef).abs() / (h * coef)).max()) <= 8 * ref.ULP
    g[0], g[1] = 0.0, math.inf  # an element that is not finite
    assert float(zb.GradClip([g]).clip(1e3)[1]) == 1.0


def test_zero_gradients_and_no_limit():
    grads = [torch.zeros(100, device="cuda"), torch.zeros(0, device="cuda")]
    stats = zb.GradClip(grads).clip(1.0)
    assert stats.tolist() == [0.0, 1.0] and bool((grads[0] == 0).all())
    grads = grads_of([100, 7], "f32", 6)
    host = [g.clone() for g in grads]
    assert float(zb.GradClip(grads).clip(math.inf)[1]) == 1.0
    assert all(torch.equal(a, b) for a, b in zip(grads, host))
    empty = zb.GradClip([torch.zeros(0, device="cuda")])
    assert empty.norm().tolist() == [0.0, 1.0] and empty.clip(1.0).tolist() == [0.0, 1.0]


def test_same_bits_streams_and_graphs():
    grads = grads_of([300000, 17, 768, 50257], "mixed", 7)
    outs = [torch.empty(351042, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    plans = [zb.GradClip(grads, out=o) for o in outs]
    stats = plans[0].clip(1.0)
    want = outs[0].clone()
    torch.cuda.synchronize()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    outs[0].zero_()
    torch.cuda.synchronize()
    assert torch.equal(plans[0].clip(1.0, stream=side), stats)
    side.synchronize()
    assert torch.equal(outs[0], want)
    graphs, kept = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for g, p in zip(graphs, plans[1:]):
        with torch.cuda.graph(g):
            kept.append((p.clip(1.0), p.norm()))
    for _ in range(3):
        for g, st in zip(graphs, (side, other)):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for (s, n), o in zip(kept, outs[1:]):
        assert torch.equal(s, stats) and torch.equal(n[:1], stats[:1]) and torch.equal(o, want)


def test_refusals():
    g = [torch.zeros(8, device="cuda"), torch.zeros(8, dtype=torch.bfloat16, device="cuda")]
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        zb.GradClip([g[0].double()])
    with pytest.raises(TypeError, match="must be a CUDA tensor"):
        zb.GradClip([g[0].cpu()])
    with pytest.raises(ValueError, match="contiguous"):
        zb.GradClip([torch.zeros(4, 4, device="cuda").t()])
    with pytest.raises(ValueError, match="no tensors"):
        zb.GradClip([])
    with pytest.raises(ValueError, match="holds 15 elements"):
        zb.GradClip(g, out=torch.zeros(15, device="cuda"))
    with pytest.raises(ValueError, match="out has 1 tensors"):
        zb.GradClip(g, out=[g[0]])
    with pytest.raises(ValueError, match="out\\[1\\] holds"):
        zb.GradClip(g, out=[torch.zeros(8, device="cuda"), torch.zeros(7, device="cuda")])
    with pytest.raises(zb.ZgError, match="outputs of .* overlap"):
        zb.GradClip([g[0], g[0]])  # the same tensor twice would be clipped twice
    with pytest.raises(zb.ZgError, match="overlaps the output"):
        both = torch.zeros(16, device="cuda")
        zb.GradClip([both[:8], both[8:]], out=[both[8:], torch.zeros(8, device="cuda")])
    rows = (zb._Grad * 1)(zb._Grad(g[0].data_ptr(), g[0].data_ptr(), 4, zb.ZG_DTYPE_F32, zb.ZG_DTYPE_BF16))
    handle = ctypes.c_void_p()
    assert zb.lib().zg_grads_init(rows, 1, ctypes.byref(handle)) == zb.ZG_ERR_INVALID_ARG and handle.value is None
    assert b"keeps its dtype" in zb.lib().zg_last_error()
    plan = zb.GradClip(g)
    for bad in (0.0, -1.0, math.nan):
        with pytest.raises(zb.ZgError, match="max_norm"):
            plan.clip(bad)
    for bad in (0.0, math.inf, math.nan):
        with pytest.raises(zb.ZgError, match="scale"):
            plan.clip(1.0, scale=bad)
    with pytest.raises(zb.ZgError, match="eps"):
        plan.clip(1.0, -1.0)
    stats, work = torch.zeros(2, device="cuda"), torch.zeros(64, dtype=torch.uint8, device="cuda")
    assert zb.lib().zg_grads_norm(plan.handle, 1.0, stats.data_ptr(), work.data_ptr(), 8, None) == zb.ZG_ERR_INVALID_ARG
    # the same gradient twice is counted twice where it is not written over
    twice = torch.ones(4, device="cuda")
    assert abs(float(zb.GradClip([twice, twice], out=torch.zeros(8, device="cuda")).norm()[0]) - math.sqrt(8)) < 1e-6
