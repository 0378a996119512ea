"""The training operators without a GPU: their refusals come before any CUDA
call, the structs match the header, and the 64-bit formulas that the GPU tests
compare with agree with torch's own gradients."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import operators_ref as ref
from zero_sharded_mixed_flat_gb300 import binding as zb
from zero_sharded_mixed_flat_gb300 import build as zbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    zbuild.build()
    return zb.lib()


def test_null_and_range_refusals(lib):
    bad, ok = zb.ZG_ERR_INVALID_ARG, zb.ZG_OK
    out = ctypes.c_void_p()
    assert lib.zg_scan_init(1, 1, 1, None) == bad
    for shape in ((0, 1, 1), (1, 0, 1), (1, 1, 0), (1 << 30, 1 << 30, 1 << 10)):
        assert lib.zg_scan_init(*shape, ctypes.byref(out)) == bad and out.value is None
    assert lib.zg_gated_scan(None, None, None, None, None, None, None, None, None) == bad
    assert lib.zg_gated_scan_bwd(*[None] * 12) == bad
    assert lib.zg_scan_status(None, None, None) == bad
    assert lib.zg_scan_set_wait_limit(None, 1) == bad
    lib.zg_scan_destroy(None)
    topk = lambda dt=0, rows=1, vocab=10, stride=10, k=1: lib.zg_topk(None, dt, rows, vocab, stride, k, None, None, None)  # noqa: E731
    for kw in ({"dt": 2}, {"rows": -1}, {"vocab": 0}, {"vocab": 1 << 31, "stride": 1 << 31}, {"stride": 9}, {"k": 0},
               {"k": zb.ZG_TOPK_MAX + 1}, {"k": 11}, {"rows": 1 << 60}, {}):
        assert topk(**kw) == bad, kw
    assert topk(rows=0) == ok
    assert lib.zg_distill_loss(None, None, None, None) == bad
    for field, value in (("dtype", 7), ("t_dtype", -1), ("k", 0), ("temperature", 0.0), ("temperature", float("nan")),
                         ("row_stride", 5), ("vocab", 0), ("rows", -3)):
        a = zb._Distill(None, 0, 10, 10, 0, None, None, 0, 3, 1.0)
        assert lib.zg_distill_loss(ctypes.byref(a), None, None, None) == ok
        setattr(a, field, value)
        assert lib.zg_distill_loss(ctypes.byref(a), None, None, None) == bad, field
    a = zb._Distill(None, 0, 10, 10, 0, None, None, 0, 3, 1.0)
    assert lib.zg_distill_grad(ctypes.byref(a), None, float("inf"), None, None, 10, None) == bad
    assert lib.zg_distill_grad(ctypes.byref(a), None, 1.0, None, None, 9, None) == bad
    a.rows = 1
    assert lib.zg_distill_loss_grad(ctypes.byref(a), 1.0, None, None, None, None, 10, None) == bad
    assert b"logits is NULL" in lib.zg_last_error()


def test_host_tensors_never_reach_the_library():
    z, t, index = torch.zeros(2, 8), torch.zeros(2, 3), torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(TypeError, match="logits must be a CUDA tensor"):
        zb.topk_logits(z, 2)
    with pytest.raises(TypeError, match="logits must be a CUDA tensor"):
        zb.distill_loss(z, t, index, 1.0)
    scan = zb.GatedScan.__new__(zb.GatedScan)  # no handle is reached: the checks come first
    scan.handle = None
    with pytest.raises(TypeError, match="x must be a CUDA tensor"):
        scan.forward(torch.zeros(2, 3, 4), torch.zeros(2, 3, 4))
    with pytest.raises(TypeError, match="x must be a tensor"):
        scan.forward(3, 4)


def test_struct_layouts_and_constants_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    structs = {"zg_view": zb._View, "zg_scan_shape": zb._ScanShape, "zg_distill_args": zb._Distill}
    names = ["ZG_DTYPE_BF16", "ZG_DTYPE_F32", "ZG_SCAN_CHUNK", "ZG_TOPK_MAX"]
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


def test_reference_scan_against_autograd():
    torch.manual_seed(1)
    x, f, h0 = (torch.randn(*s, dtype=torch.float64, requires_grad=True) for s in ((1, 12, 3), (1, 12, 3), (3, 3)))
    bounds = [(0, 0, 5), (0, 5, 5), (0, 5, 12)]
    dy, dh = torch.randn(1, 12, 3, dtype=torch.float64), torch.randn(3, 3, dtype=torch.float64)
    ys, lasts = [], []
    for s, (_, lo, hi) in enumerate(bounds):
        h = h0[s]
        for t in range(lo, hi):
            a = torch.sigmoid(f[0, t])
            h = a * h + (1 - a) * x[0, t]
            ys.append(h)
        lasts.append(h)
    y, last = torch.stack(ys)[None], torch.stack(lasts)
    ((y * dy).sum() + (last * dh).sum()).backward()
    with torch.no_grad():
        h, wl, *_ = ref.scan(x, f, h0, bounds)
        dx, df, dh0, *_ = ref.scan_grad(x, f, h0, dy, dh, bounds)
    for got, want in ((h, y), (wl, last), (dx, x.grad), (df, f.grad), (dh0, h0.grad)):
        assert torch.allclose(got, want, rtol=1e-11, atol=1e-13)


def test_reference_distillation_against_autograd():
    torch.manual_seed(2)
    z = torch.randn(4, 11, dtype=torch.float64, requires_grad=True)
    t = torch.randn(4, 5, dtype=torch.float64)
    index = torch.stack([torch.randperm(11)[:5] for _ in range(4)]).int()
    index[1, 2], index[2], index[3, 4] = -1, -1, index[3, 0]
    w = torch.rand(4, dtype=torch.float64)
    loss = torch.zeros(4, dtype=torch.float64)
    for r in (0, 1, 3):
        there = index[r] >= 0
        p = torch.softmax(t[r][there] / 1.7, 0)
        loss[r] = 1.7 ** 2 * (p * (torch.log(p) - torch.log_softmax(z[r] / 1.7, 0)[index[r][there].long()])).sum()
    (loss * w * 8).sum().backward()
    with torch.no_grad():
        got, _, grad, *_ = ref.distill(z, t, index, 1.7, 8.0, w)
    assert torch.allclose(got, loss, rtol=1e-11, atol=1e-13) and torch.allclose(grad, z.grad, rtol=1e-11, atol=1e-13)


def test_two_threads_on_one_handle_pass_their_own_arguments(monkeypatch):
    """A call's arguments are whole when the library reads them, whatever another thread
    does with the same handle meanwhile (the interpreter's lock is free during the call)."""
    import threading

    both, seen = threading.Barrier(2, timeout=60), {}

    class Library:  # in place of the C calls: looks at its arguments when both threads are in them
        @staticmethod
        def zg_gated_scan(handle, shape, x, f, h0, y, h_last, states, stream):
            both.wait()
            seen[threading.get_ident()] = (shape._obj.tokens, x._obj.ptr, f._obj.ptr, y._obj.ptr, y._obj.token_stride)
            both.wait()
            return zb.ZG_OK

        @staticmethod
        def zg_scan_destroy(handle):
            pass

    monkeypatch.setattr(zb, "_lib", Library)
    monkeypatch.setattr(zb, "_like", lambda t, ref, what: t)
    monkeypatch.setattr(zb, "_side", lambda t, *args: None if t is None else t.data_ptr())
    monkeypatch.setattr(zb, "_stream_of", lambda *args: 0)
    scan = zb.GatedScan.__new__(zb.GatedScan)
    scan.handle = None
    want, outs = {}, []

    def call(tokens):
        x, f, y = (torch.zeros(1, tokens, 8, dtype=torch.bfloat16) for _ in range(3))
        outs.append((x, f, y))
        want[threading.get_ident()] = (tokens, x.data_ptr(), f.data_ptr(), y.data_ptr(), 8)
        scan.forward(x, f, out=y)

    threads = [threading.Thread(target=call, args=(n,)) for n in (30, 50)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(want) == 2 and seen == want


def test_temperatures_whose_exponents_overflow_are_refused(lib):
    """z / T is taken as z * (log2(e) / T): the factor has to be finite."""
    a = zb._Distill(None, 0, 10, 10, 0, None, None, 0, 3, 1.0)
    for bad, fine in ((3e-39, 4.5e-39), (4.2e-39, 1e-30)):
        a.temperature = bad
        assert lib.zg_distill_loss(ctypes.byref(a), None, None, None) == zb.ZG_ERR_INVALID_ARG, bad
        assert b"temperature" in lib.zg_last_error()
        a.temperature = fine
        assert lib.zg_distill_loss(ctypes.byref(a), None, None, None) == zb.ZG_OK, fine
