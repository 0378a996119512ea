"""The token embedding and its gradient, against the formulas in 64 bits."""
import math

import numpy as np
import pytest
import torch

import block_ref as ref
from gpu_helpers import Guarded
from zero_sharded_mixed_flat_gb300 import binding as zb

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def rand(shape, seed, dtype, scale=1.0):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape) * scale).to(dtype)


def strided(t, pad, offset):
    """The same values in rows ``pad`` apart, ``offset`` elements off an allocation."""
    flat = torch.full((offset + t.shape[0] * (t.shape[1] + pad),), 7.0, dtype=t.dtype, device="cuda")
    view = flat[offset:].view(t.shape[0], t.shape[1] + pad)[:, :t.shape[1]]
    view.copy_(t)
    return view


def ids(n, vocab, seed, kind="zipf"):
    rng = np.random.default_rng(seed)
    if kind == "one":
        t = np.full(n, vocab // 2)
    elif kind == "two":
        t = np.where(np.arange(n) % 3 == 0, 0, vocab - 1)
    elif kind == "even":
        t = rng.integers(0, vocab, n)
    else:
        t = np.minimum(np.exp(rng.random(n) * math.log(vocab + 1)).astype(np.int64) - 1, vocab - 1).clip(0)
    t = torch.from_numpy(t.astype(np.int64))
    if kind == "zipf" and n > 8:
        t[n - n // 8:] = -1
        t[1], t[3] = vocab, -(1 << 31)
    return t


SIZES = [(1, 1, 1), (1, 300, 768), (3, 2, 7), (7, 50257, 8), (33, 1000, 64), (100, 50257, 771), (257, 5, 130), (1000, 1, 31),
         (2048, 997, 256), (5000, 70001, 24), (4097, 3, 1024), (300, 40, 4099)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,vocab,width", SIZES)
def test_lookup(n, vocab, width, dtype):
    table = rand((vocab, width), 1, DT[dtype])
    tokens = ids(n, vocab, 2)
    want, err = ref.embed(table, tokens, 27.7)
    for wide in (torch.int64, torch.int32):
        got = zb.embed(table.cuda(), tokens.to(wide).cuda(), 27.7)
        assert got.dtype == DT[dtype]
        ref.check(got, want, ref.stored(want, err, DT[dtype]), "rows")
    for pad, offset in ((1, 0), (8, 8), (5, 3)):
        out = torch.full((n, width + pad), 7.0, dtype=DT[dtype], device="cuda")
        zb.embed(strided(table, pad, offset), tokens.cuda(), 27.7, out=out[:, :width])
        ref.check(out[:, :width], want, ref.stored(want, err, DT[dtype]), "rows, strided")
        assert bool((out[:, width:] == 7.0).all())


def test_lookup_of_any_shape_and_scale_one_is_a_copy():
    table = rand((500, 96), 3, torch.bfloat16).cuda()
    tokens = ids(60, 500, 4, "even").view(3, 4, 5).cuda()
    out = zb.embed(table, tokens)
    assert out.shape == (3, 4, 5, 96) and torch.equal(out, table[tokens])
    assert zb.embed(table, tokens[:0]).shape == (0, 4, 5, 96)
    assert zb.embed(table, tokens[0, 0, 0]).shape == (96,)
    special = table.clone()
    special[tokens[0, 0, 0]] = math.inf
    assert bool((zb.embed(special, tokens)[0, 0, 0] == math.inf).all())


@pytest.mark.parametrize("drow_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["zipf", "one", "two", "even"])
@pytest.mark.parametrize("n,vocab,width", SIZES)
def test_gradient(n, vocab, width, kind, dtype, drow_dtype):
    d = rand((n, width), 5, DT[drow_dtype], 1e-3)
    tokens = ids(n, vocab, 6, kind)
    want, err = ref.embed_grad(d, tokens, vocab, 27.7)
    got = zb.embed_grad(d.cuda(), tokens.cuda(), vocab, 27.7, dtype=DT[dtype])
    assert got.dtype == DT[dtype]
    ref.check(got, want, ref.stored(want, err, DT[dtype]), "gradient")
    again = zb.embed_grad(d.cuda(), tokens.to(torch.int32).cuda(), vocab, 27.7, dtype=DT[dtype])
    assert torch.equal(got, again)


@pytest.mark.parametrize("kind", ["zipf", "one", "two", "even"])
@pytest.mark.parametrize("n,vocab,width", [(65536, 300000, 16), (65537, 511, 9), (150001, 40000, 8), (70000, 1, 16),
                                           (300000, 1 << 20, 1), (9000, 1 << 24, 2)])
def test_gradient_of_many_tokens(n, vocab, width, kind):
    """Several tiles to a sorting block; more tokens than the filling blocks look through; tables of up to four
    digits; runs of one token over thousands of tiles."""
    d, tokens = rand((n, width), 21, torch.bfloat16), ids(n, vocab, 22, kind)
    want, err = ref.embed_grad(d, tokens, vocab, 1.0)
    got = zb.embed_grad(d.cuda(), tokens.cuda(), vocab, dtype=torch.float32)
    ref.check(got, want, ref.stored(want, err, torch.float32), "gradient")
    mine = torch.ones(vocab, width, device="cuda")
    zb.embed_grad(d.cuda(), tokens.cuda(), vocab, add=mine, out=mine)
    ref.check(mine, want + 1, ref.stored(want + 1, err + ref.ULP * (want + 1).abs(), torch.float32), "in place")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,vocab,width", [(7, 50257, 8), (100, 997, 771), (3000, 300, 64)])
def test_gradient_added_to_another(n, vocab, width, dtype):
    d, other = rand((n, width), 7, DT[dtype], 1e-3), rand((vocab, width), 8, DT[dtype], 1e-3)
    tokens = ids(n, vocab, 9)
    want, err = ref.embed_grad(d, tokens, vocab, 3.0, other)
    bound = ref.stored(want, err, DT[dtype])
    got = zb.embed_grad(d.cuda(), tokens.cuda(), vocab, 3.0, add=other.cuda())
    ref.check(got, want, bound, "gradient")
    for pad, offset in ((0, 0), (1, 0), (8, 8), (3, 5)):
        mine, rows = strided(other, pad, offset), strided(d, pad, offset)
        assert zb.embed_grad(rows, tokens.cuda(), vocab, 3.0, add=mine, out=mine) is mine
        ref.check(mine, want, bound, "in place")
        hit = torch.zeros(vocab, dtype=torch.bool)
        hit[tokens[(tokens >= 0) & (tokens < vocab)]] = True
        assert torch.equal(mine.cpu()[~hit], other[~hit])
        whole = mine.as_strided((vocab, width + pad), (width + pad, 1))
        if pad:  # the padding between rows stays as it was
            assert bool((whole[:-1, width:] == 7.0).all())


def test_gradient_writes_its_outputs_alone():
    n, vocab, width = 700, 333, 70
    d, tokens = rand((n, width), 10, torch.bfloat16).cuda(), ids(n, vocab, 11).cuda()
    out = Guarded(vocab * width, torch.bfloat16)
    size = zb.lib().zg_embed_grad_workspace(n, vocab, width)
    work = Guarded(size, torch.uint8)
    work.view.fill_(0xFF)  # what the workspace holds does not matter
    assert zb.lib().zg_embed_grad(d.data_ptr(), 0, width, tokens.data_ptr(), 8, n, vocab, width, 1.0, None, 0,
                                  out.view.data_ptr(), 0, width, work.view.data_ptr(), size,
                                  torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert out.intact() and work.intact()
    assert torch.equal(out.view.view(vocab, width), zb.embed_grad(d, tokens, vocab))


def test_gradient_of_no_tokens_and_of_absent_ones():
    d = torch.ones(4, 8, device="cuda")
    other = rand((5, 8), 12, torch.float32).cuda()
    none = torch.full((4,), -1, device="cuda")
    assert bool((zb.embed_grad(d, none, 5) == 0).all())
    assert torch.equal(zb.embed_grad(d, none, 5, add=other), other)
    assert bool((zb.embed_grad(d[:0], none[:0], 5) == 0).all())
    assert torch.equal(zb.embed_grad(d[:0], none[:0], 5, add=other), other)
    d[:] = math.nan  # padding rows may hold anything
    assert bool((zb.embed_grad(d, none, 5) == 0).all())


def test_non_finite_rows_stay_with_their_token():
    d = rand((6, 40), 13, torch.float32).cuda()
    tokens = torch.tensor([3, 1, 3, 0, 1, 4], device="cuda")
    clean = zb.embed_grad(d, tokens, 6)
    d[2, 5] = math.nan
    d[4, 7] = math.inf
    got = zb.embed_grad(d, tokens, 6)
    assert bool(torch.isnan(got[3, 5])) and float(got[1, 7]) == math.inf
    clean[3, 5], clean[1, 7] = got[3, 5], got[1, 7]
    assert torch.equal(got.nan_to_num(0.0), clean.nan_to_num(0.0))


def test_gradient_against_differences():
    table, tokens = rand((11, 6), 14, torch.float32).cuda(), ids(30, 11, 15).cuda()
    d, move = rand((30, 6), 16, torch.float32).cuda(), rand((11, 6), 17, torch.float64)
    grad = zb.embed_grad(d, tokens, 11, 5.0).double().cpu()
    value = lambda s: float((ref.embed(table.double().cpu() + s * move, tokens.cpu(), 5.0)[0] * d.double().cpu()).sum())  # noqa: E731
    slope = (value(1.0) - value(-1.0)) / 2  # linear in the table
    assert abs(slope - float((grad * move).sum())) <= 64 * ref.ULP * float((grad * move).abs().sum())


def test_another_stream_and_graph_replay():
    table, tokens = rand((997, 128), 18, torch.bfloat16).cuda(), ids(3000, 997, 19).cuda()
    d = rand((3000, 128), 20, torch.bfloat16).cuda()
    want = zb.embed(table, tokens, 2.0), zb.embed_grad(d, tokens, 997, 2.0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = zb.embed(table, tokens, 2.0, stream=side), zb.embed_grad(d, tokens, 997, 2.0, stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    s = torch.zeros_like(tokens)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    kept = []
    for g in graphs:
        with torch.cuda.graph(g):
            kept.append((zb.embed(table, s, 2.0), zb.embed_grad(d, s, 997, 2.0)))
    s.copy_(tokens)
    torch.cuda.synchronize()
    # both at once, each on a stream of its own
    other = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(side):
            graphs[0].replay()
        with torch.cuda.stream(other):
            graphs[1].replay()
    torch.cuda.synchronize()
    for k in kept:
        assert all(torch.equal(p, q) for p, q in zip(k, want))


def test_refusals():
    table, tokens = torch.zeros(10, 8, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    d = torch.zeros(4, 8, device="cuda")
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        zb.embed(table.half(), tokens)
    with pytest.raises(TypeError, match="int32 or int64"):
        zb.embed(table, tokens.short())
    with pytest.raises(ValueError, match="tokens must be contiguous"):
        zb.embed(table, torch.zeros(8, dtype=torch.int64, device="cuda")[::2])
    with pytest.raises(TypeError, match="tokens must be a CUDA tensor"):
        zb.embed(table, tokens.cpu())
    with pytest.raises(ValueError, match="out must have shape"):
        zb.embed(table, tokens, out=torch.zeros(4, 7, device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        zb.embed(table.t(), tokens)
    with pytest.raises(zb.ZgError, match="scale"):
        zb.embed(table, tokens, math.nan)
    with pytest.raises(zb.ZgError, match="table_stride"):
        zb.embed(table[:1].expand(10, 8), tokens)
    with pytest.raises(zb.ZgError, match="out_stride"):
        zb.embed(table, tokens, out=table[:1].expand(4, 8))
    with pytest.raises(ValueError, match="tokens must have shape"):
        zb.embed_grad(d, tokens[:3], 10)
    with pytest.raises(ValueError, match="add must have shape"):
        zb.embed_grad(d, tokens, 10, add=table[:5])
    with pytest.raises(TypeError, match="add must have dtype"):
        zb.embed_grad(d, tokens, 10, add=table, out=table.bfloat16())
    for n, vocab, width in ((4, 0, 8), (4, 1 << 31, 8), (-1, 5, 8), (1 << 31, 5, 8), (4, 5, 0), (4, 5, (1 << 20) + 1)):
        assert zb.lib().zg_embed_grad_workspace(n, vocab, width) == -1
    with pytest.raises(zb.ZgError, match="vocab must be in"):
        zb.embed_grad(d, tokens, 0)
    L, st = zb.lib(), torch.cuda.current_stream().cuda_stream
    assert L.zg_embed_grad(d.data_ptr(), 1, 8, tokens.data_ptr(), 8, 4, 10, 8, 1.0, None, 0, table.data_ptr(), 1, 8, None, 0,
                           st) == zb.ZG_ERR_INVALID_ARG and b"work has 0 bytes" in L.zg_last_error()
    assert L.zg_embed(table.data_ptr(), 1, 10, 8, 8, tokens.data_ptr(), 2, 4, 1.0, d.data_ptr(), 8, st) == zb.ZG_ERR_INVALID_ARG
