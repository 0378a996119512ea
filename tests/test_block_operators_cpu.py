"""The operators around a block without a GPU: their refusals come before any CUDA
call, the structs match the header, and the 64-bit formulas that the GPU tests
compare with agree with torch's own gradients."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import block_ref as ref
from zero_sharded_mixed_flat_gb300 import binding as zb
from zero_sharded_mixed_flat_gb300 import build as zbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BAD, OK = zb.ZG_ERR_INVALID_ARG, zb.ZG_OK


@pytest.fixture(scope="module")
def lib():
    zbuild.build()
    return zb.lib()


def test_embedding_refusals(lib):
    look = {"table": None, "dtype": 0, "vocab": 5, "width": 8, "table_stride": 8, "tokens": None, "token_bytes": 8, "n": 0,
            "scale": 1.0, "out": None, "out_stride": 8, "stream": None}
    assert lib.zg_embed(*look.values()) == OK
    for kw in ({"dtype": 2}, {"vocab": 0}, {"vocab": 1 << 31}, {"width": 0}, {"width": (1 << 20) + 1}, {"table_stride": 7},
               {"token_bytes": 2}, {"n": -1}, {"n": 1 << 31}, {"scale": float("nan")}, {"out_stride": 7}, {"n": 3}):
        assert lib.zg_embed(*{**look, **kw}.values()) == BAD, kw
    assert b"tokens is NULL" in lib.zg_last_error()
    grad = {"drows": None, "dtype": 0, "drow_stride": 8, "tokens": None, "token_bytes": 4, "n": 0, "vocab": 5, "width": 8,
            "scale": 1.0, "add": None, "add_stride": 0, "dtable": None, "table_dtype": 1, "dtable_stride": 8, "work": None,
            "work_bytes": 0, "stream": None}
    assert lib.zg_embed_grad(*grad.values()) == BAD and b"dtable is NULL" in lib.zg_last_error()
    for kw in ({"dtype": -1}, {"table_dtype": 3}, {"drow_stride": 7}, {"dtable_stride": 7}, {"token_bytes": 0}, {"n": 2},
               {"scale": float("inf")}, {"vocab": 1 << 31}):
        assert lib.zg_embed_grad(*{**grad, **kw}.values()) == BAD, kw
    for sizes in ((-1, 5, 8), (4, 0, 8), (4, 5, 0), (1 << 31, 5, 8)):
        assert lib.zg_embed_grad_workspace(*sizes) == -1
    assert lib.zg_embed_grad_workspace(4, 5, 8) >= 0


def test_block_refusals(lib):
    def block(**kw):
        b = zb._Block(0, 8, 1, 0, None, None, 8, 8, None, None, None, 1.0, 1e-6)
        for k, v in kw.items():
            setattr(b, k, v)
        return ctypes.byref(b)

    call = lambda **kw: lib.zg_block_norm(block(**kw), None, 0, None, 0, None, None)  # noqa: E731
    assert call() == OK
    assert lib.zg_block_norm(None, None, 0, None, 0, None, None) == BAD
    for kw in ({"dtype": 5}, {"rows": -1}, {"width": 0}, {"width": zb.ZG_BLOCK_MAX_WIDTH + 1}, {"groups": 0},
               {"rows": 6, "groups": 4}, {"rows": 2, "groups": 4}, {"res_scale": float("nan")}, {"eps": -1.0},
               {"eps": float("inf")}, {"rows": 2}, {"rows": 2, "gate": 16}):
        assert call(**kw) == BAD, kw
    back = lambda **kw: lib.zg_block_norm_grad(block(**kw), None, *[None, 0] * 4, None, None, None, None, 0, None)  # noqa: E731
    assert back() == OK
    for kw in ({"dtype": 5}, {"rows": 2}, {"eps": -1.0}, {"width": 0}):
        assert back(**kw) == BAD, kw
    assert lib.zg_block_norm_workspace(6, 8, 4) == -1 and lib.zg_block_norm_workspace(6, 0, 1) == -1
    assert lib.zg_block_norm_workspace(0, 8, 1) == 0 and lib.zg_block_norm_workspace(6, 8, 3) > 0


def test_policy_refusals(lib):
    def args(**kw):
        a = zb._Policy(None, 0, 10, 10, 0, 8, None, None, None, None, 0.2, 0.2, 0.0, 1.0)
        for k, v in kw.items():
            setattr(a, k, v)
        return ctypes.byref(a)

    assert lib.zg_policy_loss(args(), None, None, None, None) == OK
    assert lib.zg_policy_loss(None, None, None, None, None) == BAD
    nan, inf = float("nan"), float("inf")
    for kw in ({"dtype": 7}, {"rows": -3}, {"vocab": 0}, {"vocab": 1 << 31, "row_stride": 1 << 31}, {"row_stride": 9},
               {"token_bytes": 2}, {"temperature": 0.0}, {"temperature": 4.2e-39}, {"temperature": nan}, {"clip_low": -0.1},
               {"clip_low": 1.1}, {"clip_high": -0.1}, {"clip_high": inf}, {"kl": nan}, {"rows": 1}):
        assert lib.zg_policy_loss(args(**kw), None, None, None, None) == BAD, kw
    assert b"logits is NULL" in lib.zg_last_error()
    assert lib.zg_policy_grad(args(), None, inf, None, None, 10, None) == BAD
    assert lib.zg_policy_grad(args(), None, 1.0, None, None, 9, None) == BAD
    assert lib.zg_policy_loss_grad(args(), 1.0, None, None, None, None, 9, None) == BAD
    assert lib.zg_token_logp(None, 0, 0, 10, 10, None, 8, 1.0, None, None, None) == OK
    for bad in ((None, 3, 0, 10, 10, None, 8, 1.0), (None, 0, 0, 10, 9, None, 8, 1.0), (None, 0, 0, 10, 10, None, 1, 1.0),
                (None, 0, 0, 10, 10, None, 8, -1.0), (None, 0, 1, 10, 10, None, 8, 1.0)):
        assert lib.zg_token_logp(*bad, None, None, None) == BAD


def test_gradient_list_refusals(lib):
    out = ctypes.c_void_p()
    assert lib.zg_grads_init(None, 1, ctypes.byref(out)) == BAD and lib.zg_grads_init(None, 0, None) == BAD
    for row in ((None, None, -1, 0, 0), (None, None, 1 << 40, 0, 0), (None, None, 4, 0, 0), (None, None, 4, 2, 0),
                (None, None, 4, 0, 9)):
        rows = (zb._Grad * 1)(zb._Grad(*row))
        assert lib.zg_grads_init(rows, 1, ctypes.byref(out)) == BAD and out.value is None, row
    assert lib.zg_grads_workspace(None) == -1
    assert lib.zg_grads_norm(None, 1.0, None, None, 0, None) == BAD
    assert lib.zg_grads_clip(None, 1.0, 0.0, 1.0, None, None, 0, None) == BAD
    lib.zg_grads_destroy(None)


def test_host_tensors_never_reach_the_library():
    z, t, f = torch.zeros(2, 8), torch.zeros(2, dtype=torch.int64), torch.zeros(2)
    for call in (lambda: zb.embed(z, t), lambda: zb.embed_grad(z, t, 5), lambda: zb.block_norm(z, f),
                 lambda: zb.block_norm_grad(z, f), lambda: zb.token_logp(z, t), lambda: zb.policy_loss(z, t, f, f),
                 lambda: zb.policy_grad(z, f, t, f, f), lambda: zb.policy_loss_grad(z, t, f, f), lambda: zb.GradClip([z])):
        with pytest.raises(TypeError, match="must be a CUDA tensor"):
            call()
    for call in (lambda: zb.embed(3, t), lambda: zb.block_norm(None), lambda: zb.token_logp([1.0], t), lambda: zb.GradClip([1])):
        with pytest.raises(TypeError, match="must be a tensor"):
            call()


def test_struct_layouts_and_constants_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    structs = {"zg_block": zb._Block, "zg_policy_args": zb._Policy, "zg_grad": zb._Grad}
    names = ["ZG_EMBED_MAX_WIDTH", "ZG_BLOCK_MAX_WIDTH"]
    lines = ['#include <stddef.h>', '#include <stdio.h>', '#include "zg.h"', "int main(void) {"]
    for name, cls in structs.items():
        lines.append(f'printf("{name} size %zu\\n", sizeof({name}));')
        lines += [f'printf("{name} {f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    lines += [f'printf("{n} value %d\\n", {n});' for n in names] + ["return 0;", "}"]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines) + "\n")
    subprocess.run([cc, "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = {tuple(line.split()[:2]): int(line.split()[2])
           for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines()}
    for name, cls in structs.items():
        assert got[(name, "size")] == ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            assert got[(name, f)] == getattr(cls, f).offset, (name, f)
    for n in names:
        assert got[(n, "value")] == getattr(zb, n)


def test_reference_block_against_autograd():
    torch.manual_seed(0)
    n, d, groups = 6, 5, 3
    x, o = (torch.randn(n, d, dtype=torch.float64, requires_grad=True) for _ in range(2))
    w1, w2 = (torch.randn(d, dtype=torch.float64, requires_grad=True) for _ in range(2))
    gate = torch.randn(groups, d, dtype=torch.float64, requires_grad=True)
    b = o * torch.rsqrt((o * o).mean(1, keepdim=True) + 1e-6) * w1
    xn = 0.9 * x + gate.repeat_interleave(2, 0) * b
    nn = xn * torch.rsqrt((xn * xn).mean(1, keepdim=True) + 1e-6) * w2
    dn, dy = (torch.randn(n, d, dtype=torch.float64) for _ in range(2))
    ((nn * dn).sum() + (xn * dy).sum()).backward()
    with torch.no_grad():
        f = ref.block(x, o, w1, gate, w2, 0.9)
        g, _ = ref.block_grad(x, dn, dy, o, w1, gate, w2, 0.9)
    for got, want in ((f["x"], xn), (f["n"], nn), *zip(g, (x.grad, o.grad, w2.grad, w1.grad, gate.grad))):
        assert torch.allclose(got, want, rtol=1e-11, atol=1e-13)


def test_reference_policy_against_autograd():
    torch.manual_seed(1)
    z = torch.randn(5, 9, dtype=torch.float64, requires_grad=True)
    tokens = torch.tensor([3, 8, -1, 0, 9])
    adv, w = torch.randn(5), torch.rand(5)
    logp = torch.log_softmax(z / 1.7, 1).gather(1, tokens.clamp(0, 8)[:, None])[:, 0]
    old, refl = (logp.detach() + torch.tensor([0.1, -0.4, 0, 0.5, 0])).float(), (logp.detach() + 0.3).float()
    ratio, d = torch.exp(logp - old), refl - logp
    loss = -torch.minimum(ratio * adv, ratio.clamp(0.8, 1.28) * adv) + 0.1 * (torch.exp(d) - 1 - d)
    there = (tokens >= 0) & (tokens < 9)
    ((loss * w)[there].sum() * 8).backward()
    with torch.no_grad():
        (got, lp, lse, grad), _ = ref.policy(z, tokens, 1.7, old, adv, refl, (0.2, 0.28), 0.1, 8.0, w)
    assert torch.allclose(got, loss * there, rtol=1e-11) and torch.allclose(lp, logp * there, rtol=1e-11)
    assert torch.allclose(lse, torch.logsumexp(z / 1.7, 1) * there, rtol=1e-11)
    assert torch.allclose(grad, z.grad, rtol=1e-11, atol=1e-13)


def test_reference_embedding_against_autograd():
    table = torch.randn(7, 4, dtype=torch.float64, requires_grad=True)
    tokens = torch.tensor([3, 3, -1, 0, 7, 6, 3])
    rows, _ = ref.embed(table, tokens, 2.5)
    d = torch.randn(7, 4, dtype=torch.float64)
    (rows * d).sum().backward()
    assert torch.allclose(ref.embed_grad(d, tokens, 7, 2.5)[0], table.grad, rtol=1e-12, atol=0)
