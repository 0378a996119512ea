"""Thin Python binding over libzg.so (declared in include/zg.h).

Argument marshalling only: torch tensors supply device pointers, torch
streams supply the cudaStream_t, and every step of the computation runs in
the library's CUDA kernels. Each ``zg_*`` function here calls the C function
of the same name and raises ``ZgError`` on a non-zero status.

There is no fallback: if ``libzg.so`` has not been built (``python -m
zero_sharded_mixed_flat_gb300.build``) or CUDA is unavailable, the first call
fails loudly.
"""
from __future__ import annotations

import ctypes
import os
import threading
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libzg.so")

ZG_OK = 0
ZG_ERR_INVALID_ARG = -1
ZG_ERR_MISALIGNED = -2
ZG_ERR_NOT_BOUND = -3
ZG_ERR_CUDA = -4
ZG_ERR_DEVICE_TIMEOUT = -5
ZG_ERR_STALE_NORM = -6
ZG_ERR_NO_MEMORY = -7
ZG_ERR_STATE_PARTIAL = -8
ZG_VARIANT_LDG = 0
ZG_VARIANT_TMA = 1
ZG_VARIANT_STAGED = 2
ZG_VARIANT_SINGLE = 3
ZG_MAX_RANKS = 16
ZG_BUCKET_FIRST = 1
ZG_BUCKET_LAST = 2
ZG_DTYPE_BF16 = 0
ZG_DTYPE_F32 = 1
ZG_SCAN_CHUNK = 128
ZG_TOPK_MAX = 256
ZG_EMBED_MAX_WIDTH = 1 << 20
ZG_BLOCK_MAX_WIDTH = 16384


class ZgError(RuntimeError):
    def __init__(self, code: int, where: str, detail: str):
        super().__init__(f"{where}: {detail} (status {code})")
        self.code = code


class _Hp(ctypes.Structure):
    _fields_ = [
        ("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
        ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double),
        ("max_grad_norm", ctypes.c_double), ("norm_eps", ctypes.c_double), ("grad_average", ctypes.c_int),
    ]


class _Info(ctypes.Structure):
    _fields_ = [
        ("sumsq", ctypes.c_double), ("norm", ctypes.c_double), ("clip_coef", ctypes.c_float),
        ("found_inf", ctypes.c_int), ("step_t", ctypes.c_int64), ("status", ctypes.c_int),
    ]


_P, _I64 = ctypes.c_void_p, ctypes.c_int64


class _View(ctypes.Structure):
    _fields_ = [("ptr", _P), ("batch_stride", _I64), ("token_stride", _I64)]


class _ScanShape(ctypes.Structure):
    _fields_ = [("batch", _I64), ("tokens", _I64), ("channels", _I64), ("seq_start", _P), ("n_seq", _I64),
                ("dtype", ctypes.c_int), ("clear_rest", ctypes.c_int)]


class _Distill(ctypes.Structure):
    _fields_ = [("logits", _P), ("rows", _I64), ("vocab", _I64), ("row_stride", _I64), ("dtype", ctypes.c_int),
                ("t_logits", _P), ("t_index", _P), ("t_dtype", ctypes.c_int), ("k", ctypes.c_int),
                ("temperature", ctypes.c_float)]


class _Block(ctypes.Structure):
    _fields_ = [("rows", _I64), ("width", _I64), ("groups", _I64), ("dtype", ctypes.c_int), ("x", _P), ("o", _P),
                ("x_stride", _I64), ("o_stride", _I64), ("w_post", _P), ("gate", _P), ("w_pre", _P),
                ("res_scale", ctypes.c_float), ("eps", ctypes.c_float)]


class _Policy(ctypes.Structure):
    _fields_ = [("logits", _P), ("rows", _I64), ("vocab", _I64), ("row_stride", _I64), ("dtype", ctypes.c_int),
                ("token_bytes", ctypes.c_int), ("tokens", _P), ("old_logp", _P), ("advantage", _P), ("ref_logp", _P),
                ("clip_low", ctypes.c_float), ("clip_high", ctypes.c_float), ("kl", ctypes.c_float),
                ("temperature", ctypes.c_float)]


class _Grad(ctypes.Structure):
    _fields_ = [("grad", _P), ("out", _P), ("n", _I64), ("dtype", ctypes.c_int), ("out_dtype", ctypes.c_int)]


@dataclass(frozen=True)
class Hparams:
    lr: float = 1e-3
    beta1: float = 0.9
    beta2: float = 0.999
    eps: float = 1e-8
    weight_decay: float = 0.01
    max_grad_norm: float = 1.0
    norm_eps: float = 1e-6
    grad_average: int = 1


@dataclass
class StepInfo:
    sumsq: float
    norm: float
    clip_coef: float
    found_inf: bool
    step_t: int
    status: int


_lib = None


def lib() -> ctypes.CDLL:
    """Load libzg.so from the package directory (no search path, no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with `python -m zero_sharded_mixed_flat_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        sig = {
            "zg_init": (ctypes.c_int, [_I64, ctypes.c_int, ctypes.POINTER(_Hp), ctypes.POINTER(_P)]),
            "zg_shard_len": (_I64, [_P]),
            "zg_bind": (ctypes.c_int, [_P, _P, _P, _P, _P]),
            "zg_bind_grad_stage": (ctypes.c_int, [_P, _P]),
            "zg_bind_params_mxfp8": (ctypes.c_int, [_P, _P, _P]),
            "zg_step": (ctypes.c_int, [_P, _P, ctypes.c_float, _P]),
            "zg_grad_norm": (ctypes.c_int, [_P, _P, ctypes.c_float, _P]),
            "zg_shard_step": (ctypes.c_int, [_P, _P, ctypes.c_float, _P]),
            "zg_grad_norm_bucket": (ctypes.c_int, [_P, _P, _I64, _I64, ctypes.c_float, ctypes.c_int, _P]),
            "zg_quant_mxfp8": (ctypes.c_int, [_P, _I64, _P, _P, _P]),
            "zg_step_mxfp8": (ctypes.c_int, [_P, _P, _P, ctypes.c_float, _P]),
            "zg_grad_norm_mxfp8": (ctypes.c_int, [_P, _P, _P, ctypes.c_float, _P]),
            "zg_shard_step_mxfp8": (ctypes.c_int, [_P, _P, _P, ctypes.c_float, _P]),
            "zg_quant_norm_mxfp8": (ctypes.c_int, [_P, _P, _P, _P, ctypes.c_float, _P]),
            "zg_get_info": (ctypes.c_int, [_P, _P, ctypes.POINTER(_Info)]),
            "zg_set_step": (ctypes.c_int, [_P, _I64, _P]),
            "zg_set_variant": (ctypes.c_int, [_P, ctypes.c_int]),
            "zg_set_wait_limit": (ctypes.c_int, [_P, _I64]),
            "zg_probe_copy": (ctypes.c_int, [_P, _P, _I64, _P]),
            "zg_gather_params": (ctypes.c_int, [_P, _P, _I64, _I64, _P, _P]),
            "zg_gather_params_mxfp8": (ctypes.c_int, [_P, _P, _P, _I64, _I64, _P, _P]),
            "zg_gather_params_dma": (ctypes.c_int, [_P, _P, _I64, _I64, _P, _P]),
            "zg_grad_norm_noalloc": (ctypes.c_int, [_P, ctypes.c_int, _I64, ctypes.c_float, ctypes.c_int, _P, _P]),
            "zg_destroy": (None, [_P]),
            "zg_scan_init": (ctypes.c_int, [_I64, _I64, _I64, ctypes.POINTER(_P)]),
            "zg_scan_destroy": (None, [_P]),
            "zg_gated_scan": (ctypes.c_int, [_P] * 9),
            "zg_gated_scan_bwd": (ctypes.c_int, [_P] * 12),
            "zg_scan_status": (ctypes.c_int, [_P, _P, ctypes.POINTER(ctypes.c_int)]),
            "zg_scan_set_wait_limit": (ctypes.c_int, [_P, _I64]),
            "zg_topk": (ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _I64, ctypes.c_int, _P, _P, _P]),
            "zg_distill_loss": (ctypes.c_int, [_P, _P, _P, _P]),
            "zg_distill_grad": (ctypes.c_int, [_P, _P, ctypes.c_float, _P, _P, _I64, _P]),
            "zg_distill_loss_grad": (ctypes.c_int, [_P, ctypes.c_float, _P, _P, _P, _P, _I64, _P]),
            "zg_embed": (ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _I64, _P, ctypes.c_int, _I64, ctypes.c_float, _P, _I64,
                                        _P]),
            "zg_embed_grad_workspace": (_I64, [_I64, _I64, _I64]),
            "zg_embed_grad": (ctypes.c_int, [_P, ctypes.c_int, _I64, _P, ctypes.c_int, _I64, _I64, _I64, ctypes.c_float, _P,
                                             _I64, _P, ctypes.c_int, _I64, _P, _I64, _P]),
            "zg_block_norm": (ctypes.c_int, [_P, _P, _I64, _P, _I64, _P, _P]),
            "zg_block_norm_workspace": (_I64, [_I64, _I64, _I64]),
            "zg_block_norm_grad": (ctypes.c_int, [_P, _P, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _P, _I64, _P]),
            "zg_token_logp": (ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _I64, _P, ctypes.c_int, ctypes.c_float, _P, _P,
                                             _P]),
            "zg_policy_loss": (ctypes.c_int, [_P, _P, _P, _P, _P]),
            "zg_policy_grad": (ctypes.c_int, [_P, _P, ctypes.c_float, _P, _P, _I64, _P]),
            "zg_policy_loss_grad": (ctypes.c_int, [_P, ctypes.c_float, _P, _P, _P, _P, _I64, _P]),
            "zg_grads_init": (ctypes.c_int, [_P, _I64, ctypes.POINTER(_P)]),
            "zg_grads_destroy": (None, [_P]),
            "zg_grads_workspace": (_I64, [_P]),
            "zg_grads_norm": (ctypes.c_int, [_P, ctypes.c_float, _P, _P, _I64, _P]),
            "zg_grads_clip": (ctypes.c_int, [_P, ctypes.c_float, ctypes.c_float, ctypes.c_float, _P, _P, _I64, _P]),
            "zg_strerror": (ctypes.c_char_p, [ctypes.c_int]),
            "zg_last_error": (ctypes.c_char_p, []),
            "zg_version": (ctypes.c_int, []),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype, fn.argtypes = res, args
        _lib = L
    return _lib


def _check(rc: int, where: str) -> None:
    if rc != ZG_OK:
        L = lib()
        detail = (L.zg_last_error() or b"").decode() or L.zg_strerror(rc).decode()
        raise ZgError(rc, where, detail)


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dev_ptr(t: torch.Tensor, dtype: torch.dtype, min_numel: int, what: str, host_ok: bool = False) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a tensor")
    if not t.is_cuda and not (host_ok and t.is_pinned()):
        raise TypeError(f"{what} must be a CUDA tensor" + (" or pinned host memory" if host_ok else ""))
    if t.dtype != dtype:
        raise TypeError(f"{what} must have dtype {dtype} (got {t.dtype})")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if t.numel() < min_numel:
        raise ValueError(f"{what} holds {t.numel()} elements, needs at least {min_numel}")
    return t.data_ptr()


def _ptr_array(ptrs) -> ctypes.Array:
    return (ctypes.c_void_p * len(ptrs))(*ptrs)


class Ctx:
    """Owns one zg_ctx handle; remembers N and P for the marshalling checks."""

    def __init__(self, handle: int, n: int, p: int):
        self.handle, self.n, self.p = handle, n, p

    def __del__(self):
        if getattr(self, "handle", None) and _lib is not None:
            _lib.zg_destroy(self.handle)
            self.handle = None


# ----------------------------------------------------------------- the C ABI

def zg_init(n: int, p: int, hp: Hparams = Hparams()) -> Ctx:
    out = ctypes.c_void_p()
    h = _Hp(hp.lr, hp.beta1, hp.beta2, hp.eps, hp.weight_decay, hp.max_grad_norm, hp.norm_eps, int(hp.grad_average))
    _check(lib().zg_init(n, p, ctypes.byref(h), ctypes.byref(out)), "zg_init")
    return Ctx(out.value, n, p)


def zg_shard_len(ctx: Ctx) -> int:
    return int(lib().zg_shard_len(ctx.handle))


def zg_bind(ctx: Ctx, w: torch.Tensor, m: torch.Tensor, v: torch.Tensor, params: torch.Tensor) -> None:
    """w, m, v may be CUDA tensors or pinned host tensors (optimizer state
    offloaded to host memory, read and written by the kernels in place)."""
    ptrs = [_dev_ptr(w, torch.float32, ctx.n, "w", True), _dev_ptr(m, torch.float32, ctx.n, "m", True),
            _dev_ptr(v, torch.float32, ctx.n, "v", True), _dev_ptr(params, torch.bfloat16, ctx.n, "params")]
    _check(lib().zg_bind(ctx.handle, *ptrs), "zg_bind")
    ctx._state = (w, m, v, params)  # keep the memory alive while bound


def zg_bind_grad_stage(ctx: Ctx, stage: torch.Tensor) -> None:
    _check(lib().zg_bind_grad_stage(ctx.handle, _dev_ptr(stage, torch.float32, ctx.n, "stage")), "zg_bind_grad_stage")
    ctx._stage = stage


def zg_bind_params_mxfp8(ctx: Ctx, codes: torch.Tensor | None, scales: torch.Tensor | None) -> None:
    """Write the parameters as MXFP8 codes + scales instead of bf16 (None, None: back to bf16)."""
    if codes is None and scales is None:
        _check(lib().zg_bind_params_mxfp8(ctx.handle, None, None), "zg_bind_params_mxfp8")
        ctx._mx_params = None
        return
    c = _dev_ptr(codes, torch.uint8, ctx.n, "codes")
    s = _dev_ptr(scales, torch.uint8, (ctx.n + 31) // 32, "scales")
    _check(lib().zg_bind_params_mxfp8(ctx.handle, c, s), "zg_bind_params_mxfp8")
    ctx._mx_params = (codes, scales)


def _grads(ctx: Ctx, grads) -> ctypes.Array:
    if len(grads) != ctx.p:
        raise ValueError(f"expected {ctx.p} gradient buffers, got {len(grads)}")
    return _ptr_array([_dev_ptr(g, torch.bfloat16, ctx.n, f"grads[{r}]") for r, g in enumerate(grads)])


def _mx(ctx: Ctx, codes, scales):
    if len(codes) != ctx.p or len(scales) != ctx.p:
        raise ValueError(f"expected {ctx.p} code and scale buffers")
    nb = (ctx.n + 31) // 32
    c = _ptr_array([_dev_ptr(x, torch.uint8, ctx.n, f"codes[{r}]") for r, x in enumerate(codes)])
    s = _ptr_array([_dev_ptr(x, torch.uint8, nb, f"scales[{r}]") for r, x in enumerate(scales)])
    return c, s


def zg_step(ctx: Ctx, grads, loss_scale: float, stream=None) -> None:
    _check(lib().zg_step(ctx.handle, _grads(ctx, grads), loss_scale, _stream(stream)), "zg_step")


def zg_grad_norm(ctx: Ctx, grads, loss_scale: float, stream=None) -> None:
    _check(lib().zg_grad_norm(ctx.handle, _grads(ctx, grads), loss_scale, _stream(stream)), "zg_grad_norm")


def zg_grad_norm_bucket(ctx: Ctx, grads, lo: int, hi: int, loss_scale: float, flags: int, stream=None) -> None:
    _check(lib().zg_grad_norm_bucket(ctx.handle, _grads(ctx, grads), lo, hi, loss_scale, flags, _stream(stream)),
           "zg_grad_norm_bucket")


def zg_shard_step(ctx: Ctx, grads, loss_scale: float, stream=None) -> None:
    _check(lib().zg_shard_step(ctx.handle, _grads(ctx, grads), loss_scale, _stream(stream)), "zg_shard_step")


def _shard_ptrs(ctx: Ctx, shards, dtype: torch.dtype, block: int, what: str) -> ctypes.Array:
    """P shard pointers, one unit per ``block`` parameters (1 for values and
    codes, 32 for MX scales): from P tensors (rank r's part), or from one
    tensor holding all P shards end to end (rank r's part starts at unit
    r * S / block; ranks that own nothing get a pointer that is never read)."""
    s = zg_shard_len(ctx)
    if isinstance(shards, torch.Tensor):
        base = _dev_ptr(shards, dtype, -(-ctx.n // block), what)
        return _ptr_array([base + r * (s // block) * shards.element_size() for r in range(ctx.p)])
    if len(shards) != ctx.p:
        raise ValueError(f"expected {ctx.p} {what} shards, got {len(shards)}")
    need = [-(-max(0, min(s, ctx.n - r * s)) // block) for r in range(ctx.p)]
    return _ptr_array([_dev_ptr(x, dtype, need[r], f"{what}[{r}]") for r, x in enumerate(shards)])


def zg_gather_params(ctx: Ctx, shards, lo: int, hi: int, out: torch.Tensor, stream=None) -> None:
    """Stage three: parameters [lo, hi) gathered from the P bf16 shards into
    out[0, hi - lo). ``shards``: P tensors, or the whole parameter vector."""
    sp = _shard_ptrs(ctx, shards, torch.bfloat16, 1, "shards")
    o = _dev_ptr(out, torch.bfloat16, max(hi - lo, 0), "out")
    _check(lib().zg_gather_params(ctx.handle, sp, lo, hi, o, _stream(stream)), "zg_gather_params")


def zg_gather_params_dma(ctx: Ctx, shards, lo: int, hi: int, out: torch.Tensor, stream=None) -> None:
    """zg_gather_params on the copy engines (one device-to-device copy per shard crossed)."""
    sp = _shard_ptrs(ctx, shards, torch.bfloat16, 1, "shards")
    o = _dev_ptr(out, torch.bfloat16, max(hi - lo, 0), "out")
    _check(lib().zg_gather_params_dma(ctx.handle, sp, lo, hi, o, _stream(stream)), "zg_gather_params_dma")


def zg_gather_params_mxfp8(ctx: Ctx, codes, scales, lo: int, hi: int, out: torch.Tensor, stream=None) -> None:
    """The gather from MXFP8 parameter shards, decoded to bf16. ``codes`` and
    ``scales``: P tensors each, or the whole code and scale vectors."""
    cp = _shard_ptrs(ctx, codes, torch.uint8, 1, "codes")
    sp = _shard_ptrs(ctx, scales, torch.uint8, 32, "scales")
    o = _dev_ptr(out, torch.bfloat16, max(hi - lo, 0), "out")
    _check(lib().zg_gather_params_mxfp8(ctx.handle, cp, sp, lo, hi, o, _stream(stream)), "zg_gather_params_mxfp8")


def zg_quant_mxfp8(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, n: int | None = None,
                   stream=None) -> None:
    n = x.numel() if n is None else n
    ptrs = (_dev_ptr(x, torch.bfloat16, n, "in"), _dev_ptr(codes, torch.uint8, n, "codes"),
            _dev_ptr(scales, torch.uint8, (n + 31) // 32, "scales"))
    _check(lib().zg_quant_mxfp8(ptrs[0], n, ptrs[1], ptrs[2], _stream(stream)), "zg_quant_mxfp8")


def zg_step_mxfp8(ctx: Ctx, codes, scales, loss_scale: float, stream=None) -> None:
    c, s = _mx(ctx, codes, scales)
    _check(lib().zg_step_mxfp8(ctx.handle, c, s, loss_scale, _stream(stream)), "zg_step_mxfp8")


def zg_grad_norm_mxfp8(ctx: Ctx, codes, scales, loss_scale: float, stream=None) -> None:
    c, s = _mx(ctx, codes, scales)
    _check(lib().zg_grad_norm_mxfp8(ctx.handle, c, s, loss_scale, _stream(stream)), "zg_grad_norm_mxfp8")


def zg_quant_norm_mxfp8(ctx: Ctx, grads, codes, scales, loss_scale: float, stream=None) -> None:
    """Encode the P bf16 gradients into ``codes``/``scales`` and take the norm
    pass from the encoded values, in one launch."""
    g = _grads(ctx, grads)
    c, s = _mx(ctx, codes, scales)
    _check(lib().zg_quant_norm_mxfp8(ctx.handle, g, c, s, loss_scale, _stream(stream)), "zg_quant_norm_mxfp8")


def zg_shard_step_mxfp8(ctx: Ctx, codes, scales, loss_scale: float, stream=None) -> None:
    c, s = _mx(ctx, codes, scales)
    _check(lib().zg_shard_step_mxfp8(ctx.handle, c, s, loss_scale, _stream(stream)), "zg_shard_step_mxfp8")


def zg_get_info(ctx: Ctx, stream=None) -> StepInfo:
    i = _Info()
    _check(lib().zg_get_info(ctx.handle, _stream(stream), ctypes.byref(i)), "zg_get_info")
    return StepInfo(i.sumsq, i.norm, i.clip_coef, bool(i.found_inf), int(i.step_t), int(i.status))


def zg_set_step(ctx: Ctx, t: int, stream=None) -> None:
    """Resume at applied-step count t, in stream order (does not wait)."""
    _check(lib().zg_set_step(ctx.handle, t, _stream(stream)), "zg_set_step")


def zg_set_variant(ctx: Ctx, variant: int) -> None:
    _check(lib().zg_set_variant(ctx.handle, variant), "zg_set_variant")


def zg_set_wait_limit(ctx: Ctx, polls: int) -> None:
    _check(lib().zg_set_wait_limit(ctx.handle, polls), "zg_set_wait_limit")


def zg_probe_copy(src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
    """Copy src's bytes into dst with the library's streaming copy kernel
    (both CUDA tensors, contiguous; any dtype, byte count a multiple of 16)."""
    nbytes = src.numel() * src.element_size() if isinstance(src, torch.Tensor) else 0
    s = _dev_ptr(src, src.dtype if isinstance(src, torch.Tensor) else None, 0, "src")
    d = _dev_ptr(dst, dst.dtype if isinstance(dst, torch.Tensor) else None, 0, "dst")
    if dst.numel() * dst.element_size() < nbytes:
        raise ValueError("dst smaller than src")
    _check(lib().zg_probe_copy(s, d, nbytes, _stream(stream)), "zg_probe_copy")


def zg_grad_norm_noalloc(grads, n: int, loss_scale: float, out: torch.Tensor, grad_average: int = 1,
                         stream=None) -> None:
    """The norm pass without any device allocation: writes sum of squares and
    norm into ``out`` (a CUDA float64 tensor of at least two elements)."""
    ptrs = _ptr_array([_dev_ptr(g, torch.bfloat16, n, f"grads[{r}]") for r, g in enumerate(grads)])
    o = _dev_ptr(out, torch.float64, 2, "out")
    _check(lib().zg_grad_norm_noalloc(ptrs, len(grads), n, loss_scale, grad_average, o, _stream(stream)),
           "zg_grad_norm_noalloc")


def zg_version() -> int:
    return int(lib().zg_version())


# ----------------------------------------------------------------- convenience

class ShardedAdamW:
    """A context plus torch-allocated state: fp32 w, m, v and bf16 params,
    each N long, bound to the context. With ``offload`` the fp32 state lives
    in pinned host memory and the kernels read and write it there."""

    def __init__(self, n: int, p: int, hp: Hparams = Hparams(), w0: torch.Tensor | None = None,
                 device: str | torch.device = "cuda", offload: bool = False):
        self.ctx = zg_init(n, p, hp)
        self.n, self.p, self.hp = n, p, hp

        def state(init=None):
            if offload:
                t = torch.zeros(n, dtype=torch.float32, pin_memory=True)
            else:
                t = torch.zeros(n, dtype=torch.float32, device=device)
            if init is not None:
                t.copy_(init.to(torch.float32).reshape(-1))
            return t

        self.w = state(w0)
        self.m = state()
        self.v = state()
        self.params = self.w.to(device=device, dtype=torch.bfloat16)
        zg_bind(self.ctx, self.w, self.m, self.v, self.params)

    def use_mx_params(self) -> None:
        """Store the parameters as MXFP8 (allocates codes and scales with torch)."""
        dev = self.params.device
        self.pcodes = torch.zeros(self.n, dtype=torch.uint8, device=dev)
        self.pscales = torch.zeros((self.n + 31) // 32, dtype=torch.uint8, device=dev)
        zg_bind_params_mxfp8(self.ctx, self.pcodes, self.pscales)

    def use_staged(self) -> None:
        """Switch to the staged variant (allocates the fp32 stage with torch)."""
        self.stage = torch.empty(self.n, dtype=torch.float32, device=self.w.device)
        zg_bind_grad_stage(self.ctx, self.stage)
        zg_set_variant(self.ctx, ZG_VARIANT_STAGED)

    @property
    def shard_len(self) -> int:
        return zg_shard_len(self.ctx)

    def step(self, grads, loss_scale: float, stream=None) -> None:
        zg_step(self.ctx, grads, loss_scale, stream)

    def step_mxfp8(self, codes, scales, loss_scale: float, stream=None) -> None:
        zg_step_mxfp8(self.ctx, codes, scales, loss_scale, stream)

    def info(self, stream=None) -> StepInfo:
        return zg_get_info(self.ctx, stream)

    def gather(self, lo: int, hi: int, out: torch.Tensor | None = None, stream=None,
               dma: bool = False) -> torch.Tensor:
        """Stage three: parameters [lo, hi) gathered from the P rank shards of
        the parameter vector (from the MX shards, decoded, when MX parameters
        are bound) into ``out`` (allocated when None); ``dma`` moves bf16
        shards with the copy engines instead of a kernel."""
        if out is None:
            out = torch.empty(max(hi - lo, 0), dtype=torch.bfloat16, device=self.params.device)
        if getattr(self, "pcodes", None) is not None:
            zg_gather_params_mxfp8(self.ctx, self.pcodes, self.pscales, lo, hi, out, stream)
        elif dma:
            zg_gather_params_dma(self.ctx, self.params, lo, hi, out, stream)
        else:
            zg_gather_params(self.ctx, self.params, lo, hi, out, stream)
        return out


# ----------------------------------------------------------------- training operators
#
# Each runs on ``stream``, or on the current one, and allocates its outputs there, as under
# ``torch.cuda.stream``: inputs, and outputs used elsewhere, are the caller's to order and to
# keep. None is recorded by autograd: of tensors that require gradients the values are taken.

_DTYPES = {torch.bfloat16: ZG_DTYPE_BF16, torch.float32: ZG_DTYPE_F32}


def _dtype(t: torch.Tensor, what: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a tensor")
    if t.dtype not in _DTYPES:
        raise TypeError(f"{what} must be bfloat16 or float32 (got {t.dtype})")
    return _DTYPES[t.dtype]


def _like(t: torch.Tensor, ref: torch.Tensor, what: str) -> torch.Tensor:
    """A CUDA tensor of ref's device, dtype and shape whose last dimension is contiguous (an empty one's
    strides lead nowhere, and may be any)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a tensor")
    if not t.is_cuda:
        raise TypeError(f"{what} must be a CUDA tensor")
    if t is not ref:
        if t.get_device() != ref.get_device():
            raise ValueError(f"{what} is on {t.device}, not on {ref.device}")
        if t.dtype != ref.dtype:
            raise TypeError(f"{what} must have dtype {ref.dtype} (got {t.dtype})")
        if t.shape != ref.shape:
            raise ValueError(f"{what} must have shape {tuple(ref.shape)} (got {tuple(t.shape)})")
    if t.stride(-1) != 1 and t.shape[-1] != 1 and t.numel():
        raise ValueError(f"the last dimension of {what} must be contiguous")
    return t


def _side(t: torch.Tensor | None, dtype: torch.dtype, shape: tuple, ref: torch.Tensor, what: str) -> int | None:
    """The address of an optional contiguous CUDA tensor of exactly ``shape``."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a tensor")
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {shape} (got {tuple(t.shape)})")
    if t.is_cuda and t.get_device() != ref.get_device():
        raise ValueError(f"{what} is on {t.device}, not on {ref.device}")
    return _dev_ptr(t, dtype, 0, what)


def _stream_of(ref: torch.Tensor) -> int:
    """The address of ref's device's current stream."""
    return torch._C._cuda_getCurrentRawStream(ref.get_device())


def _on(stream, ref, call, *args):
    """``call(*args)`` with ``stream`` (a stream or its address) as the current one, so that
    what it allocates is that stream's too: memory of the current stream's could be given
    out again there while the other still writes."""
    if not isinstance(stream, torch.cuda.Stream):
        device = ref.device if isinstance(ref, torch.Tensor) and ref.is_cuda else None
        address = _stream(stream)
        stream = torch.cuda.ExternalStream(address, device) if address > 1 else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return call(*args)


class _Blocks(threading.local):
    """A thread's argument blocks: filled anew by every call, kept only to spare their
    construction. A thread has its own, since a call's are read by the library while other
    threads may run, on the same handle too."""

    def __init__(self):
        self.shape = _ScanShape()
        self.views = [_View() for _ in range(5)]
        self.refs = [ctypes.byref(self.shape), *[ctypes.byref(v) for v in self.views]]


_blocks = _Blocks()


def _fill(v: _View, t: torch.Tensor) -> None:
    v.ptr = t.data_ptr()
    if t.dim() == 3:
        v.batch_stride, v.token_stride, _ = t.stride()
    else:
        v.batch_stride, v.token_stride = 0, t.stride(0)


class GatedScan:
    """The gated linear recurrence h_t = sigmoid(f_t) h_{t-1} + sigmoid(-f_t) x_t
    over time, channel by channel, with its backward pass, on a handle for up
    to ``batch`` rows of up to ``tokens`` tokens by ``channels`` channels.

    x and f are (batch, tokens, channels), or (tokens, channels) for one row,
    bfloat16 or float32, the channels contiguous (parts of a wider projection
    are fine). ``seq_start``: for one row that holds several sequences end to
    end, the int64 CUDA tensor of their starts and the last one's end. States
    are float32 (sequences, channels). One handle serves one stream at a time, and any
    thread.
    """

    def __init__(self, batch: int, tokens: int, channels: int):
        out = ctypes.c_void_p()
        self.handle = None
        _check(lib().zg_scan_init(batch, tokens, channels, ctypes.byref(out)), "zg_scan_init")
        self.handle = out.value

    def __del__(self):
        if getattr(self, "handle", None) and _lib is not None:
            _lib.zg_scan_destroy(self.handle)
            self.handle = None

    @staticmethod
    def _describe(blocks, x, f, seq_start, clear_rest) -> int:
        """Fill the shape and the views of x and f; returns the number of sequences."""
        dtype = _dtype(x, "x")
        _like(x, x, "x")
        _like(f, x, "f")
        s, views, dims = blocks.shape, blocks.views, x.dim()
        s.dtype, s.clear_rest = dtype, clear_rest
        if dims == 3:
            s.batch, s.tokens, s.channels = x.shape
        elif dims == 2:
            s.batch = 1
            s.tokens, s.channels = x.shape
        else:
            raise ValueError(f"x must be (batch, tokens, channels) or (tokens, channels) (got {tuple(x.shape)})")
        _fill(views[0], x)
        _fill(views[1], f)
        if seq_start is None:
            s.seq_start, s.n_seq = None, 0
            return s.batch
        if not isinstance(seq_start, torch.Tensor) or seq_start.dim() != 1 or seq_start.numel() < 2:
            raise ValueError("seq_start must hold the starts of the sequences and the end of the last")
        s.n_seq = seq_start.numel() - 1
        s.seq_start = _side(seq_start, torch.int64, (s.n_seq + 1,), x, "seq_start")
        return s.n_seq

    def forward(self, x, f, h0=None, seq_start=None, keep: bool = False, out=None, h_last=None, stream=None):
        """y, the state after each sequence, and with ``keep`` the states that
        ``backward`` starts from (else None). ``out`` and ``h_last`` are
        allocated when None; h_last may be h0 itself. Rows of y past the last
        packed sequence are zero, or in an ``out`` of yours left as they are."""
        if stream is not None:
            return _on(stream, x, self.forward, x, f, h0, seq_start, keep, out, h_last)
        b = _blocks
        n = self._describe(b, x, f, seq_start, out is None)
        s, side = b.shape, (n, b.shape.channels)
        y = torch.empty_like(x, memory_format=torch.contiguous_format) if out is None else _like(out, x, "out")
        _fill(b.views[2], y)
        p0 = _side(h0, torch.float32, side, x, "h0")
        last = torch.empty(side, dtype=torch.float32, device=x.device) if h_last is None else h_last
        p1 = last.data_ptr() if h_last is None else _side(last, torch.float32, side, x, "h_last")
        kept = None
        if keep:
            kept = torch.empty((s.batch, -(-s.tokens // ZG_SCAN_CHUNK), s.channels), dtype=torch.float32, device=x.device)
        r = b.refs
        _check(_lib.zg_gated_scan(self.handle, r[0], r[1], r[2], p0, r[3], p1, kept.data_ptr() if keep else None,
                                  _stream_of(x)), "zg_gated_scan")
        return y, last, kept

    def backward(self, x, f, dy, kept, h0=None, dh_last=None, seq_start=None, out=None, stream=None):
        """The gradients (dx, df, dh0) from dy and dh_last (None: zero), for the
        x, f and h0 of the forward call that gave ``kept``. ``out``: (dx, df)
        to write into, for instance the parts of one projection's gradient.
        Rows of dx and df past the last packed sequence are zero, or in an
        ``out`` of yours left as they are."""
        if stream is not None:
            return _on(stream, x, self.backward, x, f, dy, kept, h0, dh_last, seq_start, out)
        b = _blocks
        n = self._describe(b, x, f, seq_start, out is None)
        s, side = b.shape, (n, b.shape.channels)
        _fill(b.views[2], _like(dy, x, "dy"))
        if kept is None:
            raise ValueError("kept is None: call forward with keep=True")
        if out is None:
            dx, df = (torch.empty_like(x, memory_format=torch.contiguous_format) for _ in range(2))
        else:
            dx, df = _like(out[0], x, "dx"), _like(out[1], x, "df")
        _fill(b.views[3], dx)
        _fill(b.views[4], df)
        dh0 = torch.empty(side, dtype=torch.float32, device=x.device)
        pk = _side(kept, torch.float32, (s.batch, -(-s.tokens // ZG_SCAN_CHUNK), s.channels), x, "kept")
        r = b.refs
        _check(_lib.zg_gated_scan_bwd(self.handle, r[0], r[1], r[2], r[3], pk, _side(h0, torch.float32, side, x, "h0"),
                                      _side(dh_last, torch.float32, side, x, "dh_last"), r[4], r[5], dh0.data_ptr(),
                                      _stream_of(x)), "zg_gated_scan_bwd")
        return dx, df, dh0

    def step(self, x, f, state, out_state=None, out=None, stream=None):
        """One token for each of x's rows (batch, channels): y and the new
        state, written to ``out_state`` (``state`` itself to update it in place)."""
        if stream is not None:
            return _on(stream, x, self.step, x, f, state, out_state, out)
        if not isinstance(x, torch.Tensor) or x.dim() != 2:
            raise ValueError("x must be (batch, channels)")
        b = _blocks
        self._describe(b, x, f, None, False)
        y = torch.empty_like(x, memory_format=torch.contiguous_format) if out is None else _like(out, x, "out")
        _fill(b.views[2], y)
        # each row is a sequence of one token: what was the token stride leads from row to row
        s, side = b.shape, tuple(x.shape)
        s.batch, s.tokens = s.tokens, 1
        for v in b.views[:3]:
            v.batch_stride = v.token_stride
        p0 = _side(state, torch.float32, side, x, "state")
        last = torch.empty(side, dtype=torch.float32, device=x.device) if out_state is None else out_state
        p1 = last.data_ptr() if out_state is None else _side(last, torch.float32, side, x, "out_state")
        r = b.refs
        _check(_lib.zg_gated_scan(self.handle, r[0], r[1], r[2], p0, r[3], p1, None, _stream_of(x)),
               "zg_gated_scan")
        return y, last

    def set_wait_limit(self, polls: int) -> None:
        """Bound, in polls, on a block's wait for the tokens before its own."""
        _check(lib().zg_scan_set_wait_limit(self.handle, polls), "zg_scan_set_wait_limit")

    def status(self, stream=None) -> int:
        """ZG_OK, or ZG_ERR_DEVICE_TIMEOUT when a bounded wait of a scan since the last call ran out, so
        that its outputs are not valid; later scans are not concerned. Waits for the stream;
        ``forward`` and ``backward`` do not look."""
        st = ctypes.c_int()
        _check(lib().zg_scan_status(self.handle, _stream(stream), ctypes.byref(st)), "zg_scan_status")
        return st.value


def _rows(t, what: str) -> torch.Tensor:
    _dtype(t, what)
    if t.dim() != 2:
        raise ValueError(f"{what} must be (rows, vocab) (got {tuple(t.shape)})")
    return _like(t, t, what)


def _row_stride(t: torch.Tensor) -> int:
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


def topk_logits(logits, k: int, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """The k largest of each row of ``logits`` (rows, vocab), largest first,
    ties to the lowest index: values (rows, k) and int32 indices."""
    if stream is not None:
        return _on(stream, logits, topk_logits, logits, k)
    _rows(logits, "logits")
    n, v = logits.shape
    values = torch.empty((n, k), dtype=logits.dtype, device=logits.device)
    index = torch.empty((n, k), dtype=torch.int32, device=logits.device)
    _check(lib().zg_topk(logits.data_ptr(), _DTYPES[logits.dtype], n, v, _row_stride(logits), k, values.data_ptr(),
                         index.data_ptr(), _stream_of(logits)), "zg_topk")
    return values, index


def _distill(logits, t_logits, t_index, temperature: float) -> _Distill:
    _rows(logits, "logits")
    tdt = _dtype(t_logits, "t_logits")
    n, v = logits.shape
    if t_logits.dim() != 2:
        raise ValueError(f"t_logits must be (rows, k) (got {tuple(t_logits.shape)})")
    k = t_logits.shape[1]
    return _Distill(logits.data_ptr(), n, v, _row_stride(logits), _DTYPES[logits.dtype],
                    _side(t_logits, t_logits.dtype, (n, k), logits, "t_logits"),
                    _side(t_index, torch.int32, (n, k), logits, "t_index"), tdt, k, temperature)


def distill_loss(logits, t_logits, t_index, temperature: float, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """The distillation loss of each row of student ``logits`` (rows, vocab)
    against the teacher's entries ``t_logits`` and ``t_index`` (rows, k; index
    -1 for none), and each row's log-sum-exp of logits / temperature."""
    if stream is not None:
        return _on(stream, logits, distill_loss, logits, t_logits, t_index, temperature)
    a = _distill(logits, t_logits, t_index, temperature)
    loss = torch.empty(a.rows, dtype=torch.float32, device=logits.device)
    lse = torch.empty(a.rows, dtype=torch.float32, device=logits.device)
    _check(lib().zg_distill_loss(ctypes.byref(a), loss.data_ptr(), lse.data_ptr(), _stream_of(logits)),
           "zg_distill_loss")
    return loss, lse


def _gradient_of(logits, out) -> torch.Tensor:
    return torch.empty_like(logits, memory_format=torch.contiguous_format) if out is None else _like(out, logits, "out")


def distill_grad(logits, lse, t_logits, t_index, temperature: float, scale: float = 1.0, dloss=None, out=None,
                 stream=None) -> torch.Tensor:
    """The gradient of sum(scale * dloss * loss) by the logits, from the lse of
    ``distill_loss`` (dloss None: ones). ``out`` may be the logits themselves."""
    if stream is not None:
        return _on(stream, logits, distill_grad, logits, lse, t_logits, t_index, temperature, scale, dloss, out)
    a = _distill(logits, t_logits, t_index, temperature)
    out = _gradient_of(logits, out)
    _check(lib().zg_distill_grad(ctypes.byref(a), _side(lse, torch.float32, (a.rows,), logits, "lse"), scale,
                                 _side(dloss, torch.float32, (a.rows,), logits, "dloss"), out.data_ptr(),
                                 _row_stride(out), _stream_of(logits)), "zg_distill_grad")
    return out


def distill_loss_grad(logits, t_logits, t_index, temperature: float, scale: float = 1.0, dloss=None, out=None,
                      stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """The loss of each row and the gradient of sum(scale * dloss * loss) by the
    logits, in one pass over them. ``out`` may be the logits themselves."""
    if stream is not None:
        return _on(stream, logits, distill_loss_grad, logits, t_logits, t_index, temperature, scale, dloss, out)
    a = _distill(logits, t_logits, t_index, temperature)
    out = _gradient_of(logits, out)
    loss = torch.empty(a.rows, dtype=torch.float32, device=logits.device)
    _check(lib().zg_distill_loss_grad(ctypes.byref(a), scale, _side(dloss, torch.float32, (a.rows,), logits, "dloss"),
                                      loss.data_ptr(), None, out.data_ptr(), _row_stride(out),
                                      _stream_of(logits)), "zg_distill_loss_grad")
    return loss, out


# ----------------------------------------------------------------- around a block

_TOKEN_BYTES = {torch.int32: 4, torch.int64: 8}


def _tokens(t, ref: torch.Tensor, shape=None) -> int:
    """The size in bytes of a contiguous CUDA tensor of token ids (of ``shape``, if given)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("tokens must be a tensor")
    if t.dtype not in _TOKEN_BYTES:
        raise TypeError(f"tokens must be int32 or int64 (got {t.dtype})")
    if not t.is_cuda:
        raise TypeError("tokens must be a CUDA tensor")
    if t.get_device() != ref.get_device():
        raise ValueError(f"tokens is on {t.device}, not on {ref.device}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"tokens must have shape {tuple(shape)} (got {tuple(t.shape)})")
    if not t.is_contiguous():
        raise ValueError("tokens must be contiguous")
    return _TOKEN_BYTES[t.dtype]


def _stride_of_rows(t: torch.Tensor, what: str) -> int:
    """The distance of the rows (the last dimension) of a tensor that are evenly spaced."""
    if t.dim() == 2:
        return _row_stride(t)
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous, or (rows, width)")
    return t.shape[-1]


def _workspace(size: int, ref: torch.Tensor) -> torch.Tensor | None:
    return torch.empty(size, dtype=torch.uint8, device=ref.device) if size else None


def embed(table, tokens, scale: float = 1.0, out=None, stream=None) -> torch.Tensor:
    """Rows of ``table`` (vocab, width) times ``scale``, for int32 or int64 ``tokens`` of any shape:
    (*tokens.shape, width). A token outside [0, vocab) gives a row of zeros."""
    if stream is not None:
        return _on(stream, table, embed, table, tokens, scale, out)
    dtype = _dtype(table, "table")
    shape = table.shape
    if len(shape) != 2:
        raise ValueError(f"table must be (vocab, width) (got {tuple(shape)})")
    _like(table, table, "table")
    size = _tokens(tokens, table)
    vocab, width = shape
    if out is None:
        out = torch.empty((*tokens.shape, width), dtype=table.dtype, device=table.device)
        stride = width
    else:
        _beside(out, table, (*tokens.shape, width), "out")
        stride = _stride_of_rows(out, "out")
    _check(lib().zg_embed(table.data_ptr(), dtype, vocab, width, _row_stride(table), tokens.data_ptr(), size,
                          tokens.numel(), scale, out.data_ptr(), stride, _stream_of(table)), "zg_embed")
    return out


def _beside(t, ref: torch.Tensor, shape, what: str, dtype=None) -> torch.Tensor:
    """A CUDA tensor of ref's device, of ``dtype`` (or ref's) and ``shape``, its last dimension contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a tensor")
    if not t.is_cuda:
        raise TypeError(f"{what} must be a CUDA tensor")
    if t.get_device() != ref.get_device():
        raise ValueError(f"{what} is on {t.device}, not on {ref.device}")
    if t.dtype != (dtype or ref.dtype):
        raise TypeError(f"{what} must have dtype {dtype or ref.dtype} (got {t.dtype})")
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    if t.stride(-1) != 1 and t.shape[-1] != 1:
        raise ValueError(f"the last dimension of {what} must be contiguous")
    return t


def embed_grad(drows, tokens, vocab: int, scale: float = 1.0, add=None, out=None, dtype=None, stream=None) -> torch.Tensor:
    """The gradient by the table (vocab, width) from that of ``embed``'s rows, plus ``add`` (the table's gradient
    from elsewhere). Allocated in ``dtype`` (add's, else drows' own) when ``out`` is None; ``out`` may be
    ``add`` itself, of which then only rows with a token are touched. The same bits for the same inputs."""
    if stream is not None:
        return _on(stream, drows, embed_grad, drows, tokens, vocab, scale, add, out, dtype)
    rows_dtype = _dtype(drows, "drows")
    if drows.dim() < 1:
        raise ValueError("drows must be (*tokens.shape, width)")
    width = drows.shape[-1]
    _like(drows, drows, "drows")
    size = _tokens(tokens, drows, drows.shape[:-1])
    if out is None:
        out = torch.empty((vocab, width), dtype=dtype or (drows if add is None else add).dtype, device=drows.device)
    _beside(out, drows, (vocab, width), "out", dtype or out.dtype)
    if add is not None:
        _beside(add, drows, (vocab, width), "add", out.dtype)
    L, n = lib(), tokens.numel()
    work_bytes = L.zg_embed_grad_workspace(n, vocab, width)
    _check(min(work_bytes, 0), "zg_embed_grad_workspace")
    work = _workspace(work_bytes, drows)
    _check(L.zg_embed_grad(drows.data_ptr(), rows_dtype, _stride_of_rows(drows, "drows"), tokens.data_ptr(), size, n,
                           vocab, width, scale, None if add is None else add.data_ptr(),
                           0 if add is None else _row_stride(add), out.data_ptr(), _dtype(out, "out"), _row_stride(out),
                           None if work is None else work.data_ptr(), work_bytes, _stream_of(drows)), "zg_embed_grad")
    return out


def _weight_ptr(w, x: torch.Tensor, shape, what: str) -> int | None:
    if w is None:
        return None
    if not (isinstance(w, torch.Tensor) and w.dtype == x.dtype and w.shape == shape and w.get_device() == x.get_device()):
        _beside(w, x, shape, what)
    if not w.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return w.data_ptr()


def _block(x, w_pre, o, w_post, gate, res_scale: float, eps: float) -> _Block:
    dtype = _dtype(x, "x")
    shape = x.shape
    if not shape:
        raise ValueError("x must have rows")
    if not x.is_cuda:
        raise TypeError("x must be a CUDA tensor")
    p_x, x_stride = _rows_like(x, x, "x")
    width = shape[-1]
    vector = (width,)
    groups, p_gate, p_o, o_stride = 1, None, None, 0
    if gate is not None:
        if isinstance(gate, torch.Tensor) and gate.dim() == 2:
            groups = gate.shape[0]
            p_gate = _weight_ptr(gate, x, (groups, width), "gate")
        else:
            p_gate = _weight_ptr(gate, x, vector, "gate")
    if o is not None:
        p_o, o_stride = _rows_like(o, x, "o")
    rows = shape[0] if len(shape) == 2 else x.numel() // width if width else 0
    return _Block(rows, width, groups, dtype, p_x, p_o, x_stride, o_stride,
                  _weight_ptr(w_post, x, vector, "w_post"), p_gate, _weight_ptr(w_pre, x, vector, "w_pre"), res_scale, eps)


def _rows_like(t, x: torch.Tensor, what: str) -> tuple:
    """Address and row stride of an optional tensor like x."""
    if t is None:
        return None, 0
    shape = x.shape
    if not (isinstance(t, torch.Tensor) and t.dtype == x.dtype and t.shape == shape and t.get_device() == x.get_device()):
        _like(t, x, what)  # says what differs
    strides = t.stride()
    if len(strides) == 2 and strides[1] == 1 and shape[0] > 1:
        return t.data_ptr(), strides[0]
    _like(t, x, what)
    return t.data_ptr(), _stride_of_rows(t, what)


def _new_rows(x: torch.Tensor) -> torch.Tensor:
    return torch.empty_like(x, memory_format=torch.contiguous_format)


def block_norm(x, w_pre=None, o=None, w_post=None, gate=None, res_scale: float = 1.0, eps: float = 1e-6,
               keep: bool = False, out=None, n_out=None, stream=None):
    """x_new = res_scale * x + gate * b, with b = w_post * o / rms(o) (o itself without w_post), and
    n = w_pre * x_new / rms(x_new): the residual stream after a block and the next one's input. x, o are
    (..., width); w_post and w_pre (width,); gate (width,), or (groups, width) for as many equal runs of rows.
    Returns x_new (``out``, which may be x; without o only if asked for), n (``n_out``, which may be o; None
    without w_pre) and, with ``keep``, what ``block_norm_grad`` takes (else None)."""
    if stream is not None:
        return _on(stream, x, block_norm, x, w_pre, o, w_post, gate, res_scale, eps, keep, out, n_out)
    b = _block(x, w_pre, o, w_post, gate, res_scale, eps)
    if out is not None:
        p_out, out_stride = _rows_like(out, x, "out")
    elif o is not None:
        out = _new_rows(x)
        p_out, out_stride = out.data_ptr(), b.width
    else:
        p_out, out_stride = None, 0
    if n_out is not None:
        p_n, n_stride = _rows_like(n_out, x, "n_out")
    elif w_pre is not None:
        n_out = _new_rows(x)
        p_n, n_stride = n_out.data_ptr(), b.width
    else:
        p_n, n_stride = None, 0
    kept = torch.empty((2, b.rows), dtype=torch.float32, device=x.device) if keep else None
    _check(lib().zg_block_norm(ctypes.byref(b), p_out, out_stride, p_n, n_stride, kept.data_ptr() if keep else None,
                               _stream_of(x)), "zg_block_norm")
    return out, n_out, kept


def block_norm_grad(x, kept, dn=None, dx_new=None, w_pre=None, o=None, w_post=None, gate=None, res_scale: float = 1.0,
                    eps: float = 1e-6, out=None, stream=None):
    """The gradients (dx, do, dw_pre, dw_post, dgate) from those of n and of x_new (None: zero), for the x and o of
    the ``block_norm`` call that gave ``kept``; None for what that call did not have. ``out``: (dx, do) to
    write into; they may be dx_new and dn themselves."""
    if stream is not None:
        return _on(stream, x, block_norm_grad, x, kept, dn, dx_new, w_pre, o, w_post, gate, res_scale, eps, out)
    if kept is None:
        raise ValueError("kept is None: call block_norm with keep=True")
    b = _block(x, w_pre, o, w_post, gate, res_scale, eps)
    if out is not None:
        dx, do = out
        (p_dx, dx_stride), (p_do, do_stride) = _rows_like(dx, x, "dx"), _rows_like(do, x, "do")
    else:
        dx, do = _new_rows(x), None if o is None else _new_rows(x)
        p_dx, dx_stride, p_do, do_stride = dx.data_ptr(), b.width, None if o is None else do.data_ptr(), b.width
    dw_pre, dw_post, dgate = (None if w is None else torch.empty_like(w) for w in (w_pre, w_post, gate))
    L = lib()
    work_bytes = L.zg_block_norm_workspace(b.rows, b.width, b.groups)
    _check(min(work_bytes, 0), "zg_block_norm_workspace")
    work = _workspace(work_bytes, x)
    _check(L.zg_block_norm_grad(ctypes.byref(b), _side(kept, torch.float32, (2, b.rows), x, "kept"),
                                *_rows_like(dn, x, "dn"), *_rows_like(dx_new, x, "dx_new"), p_dx, dx_stride, p_do, do_stride,
                                None if dw_pre is None else dw_pre.data_ptr(),
                                None if dw_post is None else dw_post.data_ptr(),
                                None if dgate is None else dgate.data_ptr(),
                                None if work is None else work.data_ptr(), work_bytes, _stream_of(x)), "zg_block_norm_grad")
    return dx, do, dw_pre, dw_post, dgate


# ----------------------------------------------------------------- policies

def token_logp(logits, tokens, temperature: float = 1.0, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """The log-probability of each row's token (rows,) under softmax(logits / temperature), and each row's
    log-sum-exp of logits / temperature. Zeros for a token outside [0, vocab)."""
    if stream is not None:
        return _on(stream, logits, token_logp, logits, tokens, temperature)
    _rows(logits, "logits")
    n, v = logits.shape
    size = _tokens(tokens, logits, (n,))
    logp, lse = (torch.empty(n, dtype=torch.float32, device=logits.device) for _ in range(2))
    _check(lib().zg_token_logp(logits.data_ptr(), _DTYPES[logits.dtype], n, v, _row_stride(logits), tokens.data_ptr(), size,
                               temperature, logp.data_ptr(), lse.data_ptr(), _stream_of(logits)), "zg_token_logp")
    return logp, lse


def _policy(logits, tokens, old_logp, advantage, ref_logp, clip, kl: float, temperature: float) -> _Policy:
    _rows(logits, "logits")
    n, v = logits.shape
    size = _tokens(tokens, logits, (n,))
    low, high = clip
    return _Policy(logits.data_ptr(), n, v, _row_stride(logits), _DTYPES[logits.dtype], size, tokens.data_ptr(),
                   *(_side(t, torch.float32, (n,), logits, what) for t, what in
                     ((old_logp, "old_logp"), (advantage, "advantage"), (ref_logp, "ref_logp"))),
                   low, high, kl, temperature)


def policy_loss(logits, tokens, old_logp, advantage, ref_logp=None, clip=(0.2, 0.2), kl: float = 0.0,
                temperature: float = 1.0, stream=None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """The clipped policy loss of each row's token, -min(r A, clamp(r, 1 - clip[0], 1 + clip[1]) A) with
    r = exp(logp - old_logp), plus kl (exp(d) - 1 - d) with d = ref_logp - logp where there is a reference; the
    rows' logp; and what ``policy_grad`` takes. Zeros for a token outside [0, vocab)."""
    if stream is not None:
        return _on(stream, logits, policy_loss, logits, tokens, old_logp, advantage, ref_logp, clip, kl, temperature)
    a = _policy(logits, tokens, old_logp, advantage, ref_logp, clip, kl, temperature)
    loss, logp = (torch.empty(a.rows, dtype=torch.float32, device=logits.device) for _ in range(2))
    kept = torch.empty((a.rows, 3), dtype=torch.float32, device=logits.device)
    _check(lib().zg_policy_loss(ctypes.byref(a), loss.data_ptr(), logp.data_ptr(), kept.data_ptr(), _stream_of(logits)),
           "zg_policy_loss")
    return loss, logp, kept


def policy_grad(logits, kept, tokens, old_logp, advantage, ref_logp=None, clip=(0.2, 0.2), kl: float = 0.0,
                temperature: float = 1.0, scale: float = 1.0, dloss=None, out=None, stream=None) -> torch.Tensor:
    """The gradient of sum(scale * dloss * loss) by the logits, from what ``policy_loss`` kept for the same
    arguments (dloss None: ones). ``out`` may be the logits themselves."""
    if stream is not None:
        return _on(stream, logits, policy_grad, logits, kept, tokens, old_logp, advantage, ref_logp, clip, kl, temperature,
                   scale, dloss, out)
    a = _policy(logits, tokens, old_logp, advantage, ref_logp, clip, kl, temperature)
    out = _gradient_of(logits, out)
    _check(lib().zg_policy_grad(ctypes.byref(a), _side(kept, torch.float32, (a.rows, 3), logits, "kept"), scale,
                                _side(dloss, torch.float32, (a.rows,), logits, "dloss"), out.data_ptr(), _row_stride(out),
                                _stream_of(logits)), "zg_policy_grad")
    return out


def policy_loss_grad(logits, tokens, old_logp, advantage, ref_logp=None, clip=(0.2, 0.2), kl: float = 0.0,
                     temperature: float = 1.0, scale: float = 1.0, dloss=None, out=None,
                     stream=None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """The loss and logp of each row and the gradient of sum(scale * dloss * loss) by the logits, in one pass over
    them. ``out`` may be the logits themselves."""
    if stream is not None:
        return _on(stream, logits, policy_loss_grad, logits, tokens, old_logp, advantage, ref_logp, clip, kl, temperature,
                   scale, dloss, out)
    a = _policy(logits, tokens, old_logp, advantage, ref_logp, clip, kl, temperature)
    out = _gradient_of(logits, out)
    loss, logp = (torch.empty(a.rows, dtype=torch.float32, device=logits.device) for _ in range(2))
    _check(lib().zg_policy_loss_grad(ctypes.byref(a), scale, _side(dloss, torch.float32, (a.rows,), logits, "dloss"),
                                     loss.data_ptr(), logp.data_ptr(), out.data_ptr(), _row_stride(out),
                                     _stream_of(logits)), "zg_policy_loss_grad")
    return loss, logp, out


# ----------------------------------------------------------------- many gradients

class GradClip:
    """The common norm of many gradients, and their clipping: for contiguous bf16 or float32 tensors, whose
    memory this object keeps (make another when they get new memory). ``out``: None to clip them
    where they are; a flat tensor, bf16 or float32, that receives them end to end in their order (the flat
    gradient of ``ShardedAdamW.step``, say; elements past them are left as they were); or a list of tensors of
    their sizes. Calls may run on any stream; two that write at once must be ordered by the caller. A graph that
    captured a call needs this object as long as it is replayed. The norm is of this list: over several ranks
    the clipping by the reduced gradient's norm is ``ShardedAdamW.step``'s own (``max_grad_norm``)."""

    def __init__(self, tensors, out=None):
        self.handle = None
        tensors = list(tensors)
        for i, t in enumerate(tensors):
            _dtype(t, f"tensors[{i}]")
            _dev_ptr(t, t.dtype, 0, f"tensors[{i}]")
            if t.get_device() != tensors[0].get_device():
                raise ValueError(f"tensors[{i}] is on {t.device}, not on {tensors[0].device}")
        if not tensors:
            raise ValueError("there are no tensors")
        if out is None:
            outs = tensors
        elif isinstance(out, torch.Tensor):
            _dtype(out, "out")
            _dev_ptr(out, out.dtype, sum(t.numel() for t in tensors), "out")
            outs, at = [], 0
            flat = out.view(-1)
            for t in tensors:
                outs.append(flat[at:at + t.numel()])
                at += t.numel()
        else:
            outs = list(out)
            if len(outs) != len(tensors):
                raise ValueError(f"out has {len(outs)} tensors for {len(tensors)}")
        for i, (t, o) in enumerate(zip(tensors, outs)):
            _dtype(o, f"out[{i}]")
            _dev_ptr(o, o.dtype, 0, f"out[{i}]")
            if o.numel() != t.numel():
                raise ValueError(f"out[{i}] holds {o.numel()} elements, not {t.numel()}")
            if o.get_device() != tensors[0].get_device():
                raise ValueError(f"out[{i}] is on {o.device}, not on {tensors[0].device}")
        rows = (_Grad * len(tensors))(*(_Grad(t.data_ptr(), o.data_ptr(), t.numel(), _DTYPES[t.dtype], _DTYPES[o.dtype])
                                        for t, o in zip(tensors, outs)))
        self.tensors, self.out, self._outs = tensors, out, outs  # the memory stays while the list has its addresses
        handle = ctypes.c_void_p()
        with torch.cuda.device(tensors[0].device):
            _check(lib().zg_grads_init(rows, len(tensors), ctypes.byref(handle)), "zg_grads_init")
        self.handle = handle.value
        self._work_bytes = _lib.zg_grads_workspace(self.handle)

    def __del__(self):
        if getattr(self, "handle", None) and _lib is not None:
            _lib.zg_grads_destroy(self.handle)
            self.handle = None

    def norm(self, scale: float = 1.0, stream=None) -> torch.Tensor:
        """A float32 CUDA tensor of two: the norm of ``scale`` times all gradients (infinite where their squares
        overflow binary32, which ``clip`` bears), and 1."""
        ref = self.tensors[0]
        if stream is not None:
            return _on(stream, ref, self.norm, scale)
        stats = torch.empty(2, dtype=torch.float32, device=ref.device)
        work = _workspace(self._work_bytes, ref)
        _check(_lib.zg_grads_norm(self.handle, scale, stats.data_ptr(), work.data_ptr(), self._work_bytes,
                                  _stream_of(ref)), "zg_grads_norm")
        return stats

    def clip(self, max_norm: float, eps: float = 1e-6, scale: float = 1.0, stream=None) -> torch.Tensor:
        """Write scale * min(1, max_norm / (norm + eps)) times the gradients (scale times them where an element is
        not finite): a float32 CUDA tensor of the norm, of ``scale`` times them, and the coefficient."""
        ref = self.tensors[0]
        if stream is not None:
            return _on(stream, ref, self.clip, max_norm, eps, scale)
        stats = torch.empty(2, dtype=torch.float32, device=ref.device)
        work = _workspace(self._work_bytes, ref)
        _check(_lib.zg_grads_clip(self.handle, max_norm, eps, scale, stats.data_ptr(), work.data_ptr(), self._work_bytes,
                                  _stream_of(ref)), "zg_grads_clip")
        return stats
