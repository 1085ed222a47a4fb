"""Training operators: layer norm, GELU, activations kept in 8 bits and the
weight gradient taken from them (libgq_train.so, ``include/gq_train.h``).

They stand before the gradient compressor: what a transformer block computes
and keeps between its forward and backward passes, whose gradients then go
through ``ddp.global_qsgd_hook``.  An activation is kept as one byte a value
and one power of two per 32 columns (``Act8``), rounded to nearest, or, given
a seed, at random without bias, with the compressor's own Philox uniforms.
The weight gradient is linear in the kept activation, so random rounding
leaves its expectation exact.

Two layers:

- ``gqt_*``: the C entry points on CUDA (HIP) tensors, argument marshalling
  only.  Matrices are [rows, d] with unit column stride (a row stride of at
  least d, or 0); outputs are new contiguous tensors.  They launch on
  ``stream`` (default: torch's current stream) and never synchronize.  There
  is no fallback: without the built library or a GPU they raise.
- ``layer_norm``, ``gelu``, ``linear`` and ``Mlp8``: the same operators under
  autograd, and a transformer's MLP block that keeps everything it needs for
  its backward pass in 8 bits.
"""
from __future__ import annotations

import contextlib
import ctypes
import itertools
import os

import torch

from . import GQ_IN_BF16, GQ_IN_F32, STATUS, GQError

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgq_train.so")

GQT_ROUND_NEAREST = 0
GQT_ROUND_RANDOM = 1
GQT_GELU_ERF = 0
GQT_GELU_TANH = 1


class _CAct8(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("exps", ctypes.c_void_p),
                ("rounding", ctypes.c_int32), ("seed", ctypes.c_uint64)]


_i32, _i64, _f32, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p
_act8 = ctypes.POINTER(_CAct8)
SIGNATURES = {
    "gqt_act8_groups": (_i64, [_i64]),
    "gqt_act8_code_pitch": (_i64, [_i64]),
    "gqt_act8_save": (_i32, [_vp, _i32, _i64, _i64, _i64, _act8, _vp]),
    "gqt_act8_restore": (_i32, [_act8, _i64, _i64, _i32, _vp, _vp]),
    "gqt_layer_norm": (_i32, [_vp, _i32, _i64, _i64, _i64, _vp, _vp, _i32, _f32, _vp, _vp, _vp,
                              _act8, _act8, _vp]),
    "gqt_layer_norm_backward_workspace_bytes": (_i64, [_i64, _i64]),
    "gqt_layer_norm_backward": (_i32, [_vp, _i32, _i64, _i64, _i64, _vp, _i64, _act8, _vp, _vp,
                                       _vp, _i32, _vp, _vp, _vp, _vp, _i64, _vp]),
    "gqt_gelu": (_i32, [_vp, _i32, _i64, _i64, _i64, _i32, _vp, _act8, _act8, _vp]),
    "gqt_gelu_backward": (_i32, [_vp, _i32, _i64, _i64, _i64, _vp, _i64, _act8, _i32, _vp, _vp]),
    "gqt_weight_grad_workspace_bytes": (_i64, [_i64, _i64, _i64, _i32]),
    "gqt_weight_grad": (_i32, [_vp, _i32, _i64, _i64, _i64, _act8, _i64, _vp, _vp, _i32, _vp,
                               _i64, _vp]),
    "gqt_last_error": (ctypes.c_char_p, []),
}

_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libgq_train.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _check(status: int):
    if status != 0:
        raise GQError(status, lib().gqt_last_error().decode())


# ---------------------------------------------------------------------------
# arguments

_DTYPES = {torch.float32: GQ_IN_F32, torch.bfloat16: GQ_IN_BF16}


def _dtype(t, name: str) -> int:
    dt = _DTYPES.get(t)
    if dt is None:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t}")
    return dt


def _matrix(x, name: str, shape=None, dtype=None, device=None):
    """(dtype code, row stride) of a [rows, d] device tensor with unit column
    stride; its shape, dtype and device, where given, have to be these."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if x.dim() != 2 or x.shape[1] < 1:
        raise ValueError(f"{name} must be [rows, d] with d >= 1, got {list(x.shape)}")
    dt = _dtype(x.dtype, name)
    if shape is not None and tuple(x.shape) != tuple(shape):
        raise ValueError(f"{name} is {list(x.shape)}, expected {list(shape)}")
    if dtype is not None and x.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {x.dtype}")
    if device is not None and x.device != device:
        raise ValueError(f"{name} is on {x.device}, expected {device}")
    rows, d = x.shape
    s0, s1 = x.stride()
    if d > 1 and s1 != 1:
        raise ValueError(f"{name} must have unit column stride, has {s1}")
    if rows <= 1:
        return dt, d
    if s0 != 0 and s0 < d:
        raise ValueError(f"{name} has overlapping rows")
    return dt, s0


def _vector(v, name: str, n: int, device, dtype=None):
    """A contiguous 1-d device tensor of n elements (or None)."""
    if v is None:
        return None
    if not isinstance(v, torch.Tensor) or v.device != device:
        raise ValueError(f"{name} must be a tensor on {device}")
    if v.dim() != 1 or v.shape[0] != n or not v.is_contiguous():
        raise ValueError(f"{name} must be contiguous [{n}], got {list(v.shape)}")
    if dtype is not None and v.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {v.dtype}")
    return v


def _weights(w, b, d: int, device):
    """The dtype code of w and b (None: fp32), both checked."""
    _vector(w, "weight", d, device)
    _vector(b, "bias", d, device, None if w is None else w.dtype)
    given = w if w is not None else b
    return GQ_IN_F32 if given is None else _dtype(given.dtype, "weight")


def _ptr(t):
    return None if t is None else t.data_ptr()


class _Elsewhere:
    """Runs a call on another stream or device than the current one: its new
    tensors and workspaces belong to that stream, and the given ones are not
    reused before the work there is done."""

    def __init__(self, device, stream, tensors):
        if stream is None:
            stream = torch.cuda.current_stream(device)
        elif not hasattr(stream, "cuda_stream"):
            stream = (torch.cuda.ExternalStream(int(stream), device=device) if int(stream)
                      else torch.cuda.default_stream(device))
        elif stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors are on {device}")
        self.stream, self.tensors = stream, tensors

    def __enter__(self):
        self.ctx = torch.cuda.stream(self.stream)
        self.ctx.__enter__()
        return self

    def __exit__(self, *exc):
        self.ctx.__exit__(*exc)
        for t in self.tensors:
            for part in (t.codes, t.exps) if isinstance(t, Act8) else (t,):
                # a host tensor, refused inside, has no stream to be kept for
                if isinstance(part, torch.Tensor) and part.is_cuda:
                    part.record_stream(self.stream)


def _elsewhere(device, stream) -> bool:
    return stream is not None or device.index != torch.cuda.current_device()


def _current(device) -> int:
    """The current stream's handle; the accessor that builds no stream object
    takes 0.1 us of a call's 7, torch.cuda.current_stream 2.5."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _like(x):
    """A new contiguous tensor of x's shape, dtype and device."""
    return torch.empty_like(x, memory_format=torch.contiguous_format)


# ---------------------------------------------------------------------------
# the 8-bit copy

def gqt_act8_groups(d: int) -> int:
    return int(lib().gqt_act8_groups(d))


def gqt_act8_code_pitch(d: int) -> int:
    return int(lib().gqt_act8_code_pitch(d))


class Act8:
    """The 8-bit copy of a [rows, d] matrix: ``codes`` int8 [rows, 32 G] and
    ``exps`` uint8 [rows, G], G = ceil(d / 32); code q of a group with
    exponent byte e stands for q 2^(e - 127)."""

    __slots__ = ("codes", "exps", "d")

    def __init__(self, codes: torch.Tensor, exps: torch.Tensor, d: int):
        self.codes, self.exps, self.d = codes, exps, int(d)

    @classmethod
    def empty(cls, rows: int, d: int, device) -> "Act8":
        groups = (int(d) + 31) // 32
        return cls(torch.empty((rows, 32 * groups), dtype=torch.int8, device=device),
                   torch.empty((rows, groups), dtype=torch.uint8, device=device), d)

    @property
    def shape(self):
        return self.codes.shape[0], self.d

    def __repr__(self):
        return f"Act8({self.shape[0]} x {self.d}, {self.codes.device})"


def _kept(a, name: str, rows: int, d: int, device, seed=None):
    """The C view of a copy of a [rows, d] matrix (None for None)."""
    if a is None:
        return None
    if not isinstance(a, Act8):
        raise TypeError(f"{name} must be an Act8, got {type(a).__name__}")
    groups = (d + 31) // 32
    if a.d != d or a.codes.shape != (rows, 32 * groups) or a.exps.shape != (rows, groups):
        raise ValueError(f"{name} is the copy of {list(a.shape)}, expected {[rows, d]}")
    if a.codes.dtype != torch.int8 or a.exps.dtype != torch.uint8:
        raise TypeError(f"{name} must hold int8 codes and uint8 exps")
    if a.codes.device != device or a.exps.device != device:
        raise ValueError(f"{name} is on {a.codes.device}, expected {device}")
    if not a.codes.is_contiguous() or not a.exps.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if seed is None:
        return _CAct8(a.codes.data_ptr(), a.exps.data_ptr(), GQT_ROUND_NEAREST, 0)
    return _CAct8(a.codes.data_ptr(), a.exps.data_ptr(), GQT_ROUND_RANDOM,
                  int(seed) & 0xFFFFFFFFFFFFFFFF)


def gqt_act8_save(x: torch.Tensor, *, seed=None, out: Act8 | None = None, stream=None) -> Act8:
    """The 8-bit copy of x [rows, d]: to nearest, or with a 64-bit `seed` at
    random without bias."""
    dt, ldx = _matrix(x, "x")
    if _elsewhere(x.device, stream):
        with _Elsewhere(x.device, stream, (x, out)):
            return gqt_act8_save(x, seed=seed, out=out)
    rows, d = x.shape
    if out is None:
        out = Act8.empty(rows, d, x.device)
    _check(lib().gqt_act8_save(x.data_ptr(), dt, rows, d, ldx,
                               _kept(out, "out", rows, d, x.device, seed), _current(x.device)))
    return out


def gqt_act8_restore(a: Act8, dtype=torch.bfloat16, *, stream=None) -> torch.Tensor:
    """The values a copy stands for, [rows, d] (exact in either dtype)."""
    dt = _dtype(dtype, "dtype")
    if not isinstance(a, Act8) or not a.codes.is_cuda:
        raise ValueError("a must be an Act8 on a device")
    device = a.codes.device
    if _elsewhere(device, stream):
        with _Elsewhere(device, stream, (a,)):
            return gqt_act8_restore(a, dtype)
    rows, d = a.shape
    out = torch.empty((rows, d), dtype=dtype, device=device)
    _check(lib().gqt_act8_restore(_kept(a, "a", rows, d, device), rows, d, dt, out.data_ptr(),
                                  _current(device)))
    return out


# ---------------------------------------------------------------------------
# layer norm

def gqt_layer_norm(x: torch.Tensor, weight=None, bias=None, eps: float = 1e-5, *,
                   stats: bool = True, save_x: Act8 | None = None, seed_x=None,
                   save_y: Act8 | None = None, seed_y=None, stream=None):
    """Layer norm of each row: (y, mean, rstd), the last two fp32 [rows]
    (None without `stats`).  save_x / save_y receive the 8-bit copies of x
    and y in the same pass."""
    dt, ldx = _matrix(x, "x")
    device = x.device
    if _elsewhere(device, stream):
        with _Elsewhere(device, stream, (x, weight, bias, save_x, save_y)):
            return gqt_layer_norm(x, weight, bias, eps, stats=stats, save_x=save_x, seed_x=seed_x,
                                  save_y=save_y, seed_y=seed_y)
    rows, d = x.shape
    wdt = _weights(weight, bias, d, device)
    y = _like(x)
    mean = rstd = None
    if stats:
        mean = torch.empty(rows, dtype=torch.float32, device=device)
        rstd = torch.empty(rows, dtype=torch.float32, device=device)
    _check(lib().gqt_layer_norm(x.data_ptr(), dt, rows, d, ldx, _ptr(weight), _ptr(bias), wdt,
                                eps, y.data_ptr(), _ptr(mean), _ptr(rstd),
                                _kept(save_x, "save_x", rows, d, device, seed_x),
                                _kept(save_y, "save_y", rows, d, device, seed_y), _current(device)))
    return y, mean, rstd


def gqt_layer_norm_backward(dy: torch.Tensor, x, mean: torch.Tensor, rstd: torch.Tensor,
                            weight=None, *, weight_grad: bool = True, bias_grad: bool = True,
                            stream=None):
    """(dx, dw, db) of gqt_layer_norm from dy and x, x given as itself or as
    its 8-bit copy.  dw and db have the weight's dtype (fp32 without one);
    either is None where it is not wanted."""
    dt, lddy = _matrix(dy, "dy")
    device = dy.device
    if _elsewhere(device, stream):
        with _Elsewhere(device, stream, (dy, x, mean, rstd, weight)):
            return gqt_layer_norm_backward(dy, x, mean, rstd, weight, weight_grad=weight_grad,
                                           bias_grad=bias_grad)
    rows, d = dy.shape
    wdt = _weights(weight, None, d, device)
    for t, name in ((mean, "mean"), (rstd, "rstd")):
        if t is None:
            raise ValueError(f"{name} is required")
        _vector(t, name, rows, device, torch.float32)
    x8 = xp = None
    ldx = 0
    if isinstance(x, Act8):
        x8 = _kept(x, "x", rows, d, device)
    else:
        _, ldx = _matrix(x, "x", dy.shape, dy.dtype, device)
        xp = x.data_ptr() or None
    dx = _like(dy)
    wt = torch.float32 if weight is None else weight.dtype
    dw = torch.empty(d, dtype=wt, device=device) if weight_grad else None
    db = torch.empty(d, dtype=wt, device=device) if bias_grad else None
    ws, nws = None, 0
    if rows == 0 and xp is None and x8 is None:
        x8 = _CAct8()  # an empty x has no address
    if weight_grad or bias_grad:
        nws = lib().gqt_layer_norm_backward_workspace_bytes(rows, d)
        ws = torch.empty(max(nws, 16), dtype=torch.uint8, device=device)
    _check(lib().gqt_layer_norm_backward(dy.data_ptr(), dt, rows, d, lddy, xp, ldx, x8,
                                         mean.data_ptr(), rstd.data_ptr(), _ptr(weight), wdt,
                                         dx.data_ptr(), _ptr(dw), _ptr(db), _ptr(ws), nws,
                                         _current(device)))
    return dx, dw, db


# ---------------------------------------------------------------------------
# GELU

def _form(approximate) -> int:
    if approximate == "none":
        return GQT_GELU_ERF
    if approximate == "tanh":
        return GQT_GELU_TANH
    raise ValueError(f"approximate must be 'none' or 'tanh', got {approximate!r}")


def gqt_gelu(h: torch.Tensor, approximate: str = "none", *, save_h: Act8 | None = None,
             seed_h=None, save_y: Act8 | None = None, seed_y=None, stream=None) -> torch.Tensor:
    """GELU of h [rows, d]; save_h / save_y receive the 8-bit copies of h and
    of the result in the same pass."""
    dt, ldh = _matrix(h, "h")
    form, device = _form(approximate), h.device
    if _elsewhere(device, stream):
        with _Elsewhere(device, stream, (h, save_h, save_y)):
            return gqt_gelu(h, approximate, save_h=save_h, seed_h=seed_h, save_y=save_y,
                            seed_y=seed_y)
    rows, d = h.shape
    y = _like(h)
    _check(lib().gqt_gelu(h.data_ptr(), dt, rows, d, ldh, form, y.data_ptr(),
                          _kept(save_h, "save_h", rows, d, device, seed_h),
                          _kept(save_y, "save_y", rows, d, device, seed_y), _current(device)))
    return y


def gqt_gelu_backward(dy: torch.Tensor, h, approximate: str = "none", *,
                      stream=None) -> torch.Tensor:
    """dh = dy y'(h), h given as itself or as its 8-bit copy."""
    dt, lddy = _matrix(dy, "dy")
    form, device = _form(approximate), dy.device
    if _elsewhere(device, stream):
        with _Elsewhere(device, stream, (dy, h)):
            return gqt_gelu_backward(dy, h, approximate)
    rows, d = dy.shape
    h8 = hp = None
    ldh = 0
    if isinstance(h, Act8):
        h8 = _kept(h, "h", rows, d, device)
    else:
        _, ldh = _matrix(h, "h", dy.shape, dy.dtype, device)
        hp = h.data_ptr() or None
        if hp is None:
            h8 = _CAct8()  # an empty h has no address
    dh = _like(dy)
    _check(lib().gqt_gelu_backward(dy.data_ptr(), dt, rows, d, lddy, hp, ldh, h8, form,
                                   dh.data_ptr(), _current(device)))
    return dh


# ---------------------------------------------------------------------------
# the weight gradient

def gqt_weight_grad_workspace_bytes(m: int, n: int, k: int, dtype=torch.bfloat16) -> int:
    return int(lib().gqt_weight_grad_workspace_bytes(m, n, k, _dtype(dtype, "dtype")))


def gqt_weight_grad(dy: torch.Tensor, x: Act8, *, dtype=torch.float32, bias: bool = True,
                    workspace=None, stream=None):
    """(dw, db) of y = x w^T + b from dy [m, n] and the 8-bit copy of x
    [m, k]: dw = dy^T x [n, k] and db = the sum of dy's rows [n] (None
    without `bias`), in `dtype`."""
    dt, lddy = _matrix(dy, "dy")
    wdt, device = _dtype(dtype, "dtype"), dy.device
    if _elsewhere(device, stream):
        with _Elsewhere(device, stream, (dy, x, workspace)):
            return gqt_weight_grad(dy, x, dtype=dtype, bias=bias, workspace=workspace)
    m, n = dy.shape
    if not isinstance(x, Act8):
        raise TypeError(f"x must be an Act8, got {type(x).__name__}")
    k = x.d
    x8 = _kept(x, "x", m, k, device)
    dw = torch.empty((n, k), dtype=dtype, device=device)
    db = torch.empty(n, dtype=dtype, device=device) if bias else None
    need = lib().gqt_weight_grad_workspace_bytes(m, n, k, dt)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=device) if need > 0 else None
    elif (not isinstance(workspace, torch.Tensor) or workspace.device != device
          or not workspace.is_contiguous()
          or workspace.numel() * workspace.element_size() < need):
        raise ValueError(f"workspace must be contiguous, on {device}, of {need} bytes")
    _check(lib().gqt_weight_grad(dy.data_ptr(), dt, m, n, lddy, x8, k, dw.data_ptr(), _ptr(db),
                                 wdt, _ptr(workspace), max(need, 0), _current(device)))
    return dw, db


# ---------------------------------------------------------------------------
# under autograd

def _mix_seed(seed: int, k: int) -> int:
    """The 64-bit Philox key of the k-th copy of a step: the hook's mixing, so
    that no two copies share a random stream."""
    from .ddp import _mix64
    return _mix64(_mix64(seed & 0xFFFFFFFFFFFFFFFF) ^ k)


def _copy_seeds(seed):
    """Those of an MLP block's four copies in a pass."""
    return [None] * 4 if seed is None else [_mix_seed(seed, k) for k in range(4)]


def _rows(t: torch.Tensor, d: int) -> torch.Tensor:
    """t as [rows, d] with unit column stride (a copy where its strides do
    not allow it, such as a gradient expanded from a scalar)."""
    t = t.reshape(-1, d)
    if (d > 1 and t.stride(1) != 1) or (t.shape[0] > 1 and 0 < t.stride(0) < d):
        t = t.contiguous()
    return t


def _new_copy(t: torch.Tensor) -> Act8:
    return Act8.empty(t.shape[0], t.shape[1], t.device)


def _parts(a):
    """What a copy holds, for save_for_backward."""
    return (None, None) if a is None else (a.codes, a.exps)


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, bits, seed):
        x2 = _rows(x, x.shape[-1])
        kept = _new_copy(x2) if bits == 8 and any(ctx.needs_input_grad) else None
        y, mean, rstd = gqt_layer_norm(x2, weight, bias, eps, save_x=kept, seed_x=seed)
        ctx.bits, ctx.d = bits, x2.shape[1]
        ctx.bias_dtype = None if bias is None else bias.dtype
        ctx.save_for_backward(mean, rstd, weight, *(_parts(kept) if bits == 8 else (x2,)))
        return y.view(x.shape)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        mean, rstd, weight, *kept = ctx.saved_tensors
        x = Act8(*kept, ctx.d) if ctx.bits == 8 else kept[0]
        dx, dw, db = gqt_layer_norm_backward(
            _rows(dy, ctx.d), x, mean, rstd, weight, weight_grad=ctx.needs_input_grad[1],
            bias_grad=ctx.needs_input_grad[2])
        if db is not None:
            db = db.to(ctx.bias_dtype)  # a bias without a weight: the sums are fp32
        return dx.view(dy.shape), dw, db, None, None, None


def _bits(bits):
    """`bits`, checked; None where there is no backward pass to keep for."""
    if bits not in (None, 8):
        raise ValueError(f"bits must be None or 8, got {bits!r}")
    return bits if torch.is_grad_enabled() else None


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, *, bits=None, seed=None):
    """Layer norm over the last dimension, differentiable.  bits=8 keeps x for
    the backward pass in 8 bits (rounded at random where a seed is given).
    weight and bias have one dtype, fp32 or bf16."""
    return _LayerNorm.apply(x, weight, bias, eps, _bits(bits), seed)


class _Gelu(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, approximate, bits, seed):
        h2 = _rows(h, h.shape[-1])
        kept = _new_copy(h2) if bits == 8 and ctx.needs_input_grad[0] else None
        y = gqt_gelu(h2, approximate, save_h=kept, seed_h=seed)
        ctx.bits, ctx.d, ctx.approximate = bits, h2.shape[1], approximate
        ctx.save_for_backward(*(_parts(kept) if bits == 8 else (h2,)))
        return y.view(h.shape)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        kept = ctx.saved_tensors
        h = Act8(*kept, ctx.d) if ctx.bits == 8 else kept[0]
        dh = gqt_gelu_backward(_rows(dy, ctx.d), h, ctx.approximate)
        return dh.view(dy.shape), None, None, None


def gelu(h, approximate: str = "none", *, bits=None, seed=None):
    """GELU, differentiable; bits=8 keeps h for the backward pass in 8 bits."""
    return _Gelu.apply(h, approximate, _bits(bits), seed)


def _product_dtype(x):
    """What autocast casts a product's operands to; None outside autocast."""
    if not torch.is_autocast_enabled(x.device.type):
        return None
    dtype = torch.get_autocast_dtype(x.device.type)
    _dtype(dtype, "the dtype of autocast")
    return dtype


def _no_autocast(t):
    """Autocast off where it is on.  Inside a Function it would cast the
    weights without a graph and keep the casts, so that a later product with
    the same weights would have no gradient for them; and in a backward pass
    it would round what the forward pass did not."""
    kind = t.device.type
    return torch.autocast(kind, enabled=False) if torch.is_autocast_enabled(kind) else _AS_IT_IS


_AS_IT_IS = contextlib.nullcontext()


def _cast(t, dtype):
    return t if t is None or dtype is None or t.dtype == dtype else t.to(dtype)


def _dtypes_of(weight, bias):
    """Those of a product's parameters, which their gradients have too."""
    _dtype(weight.dtype, "weight")
    if bias is None:
        return weight.dtype, weight.dtype
    _dtype(bias.dtype, "bias")
    return weight.dtype, bias.dtype


def _parameter_grads(dy, x, dtypes, bias):
    """(dw, db) in their parameters' dtypes, of which autocast takes two: both
    are computed in the wider."""
    if dtypes[0] == dtypes[1]:
        return gqt_weight_grad(dy, x, dtype=dtypes[0], bias=bias)
    dw, db = gqt_weight_grad(dy, x, dtype=torch.promote_types(*dtypes), bias=bias)
    return _cast(dw, dtypes[0]), _cast(db, dtypes[1])


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, seed, grad):
        dtype = _product_dtype(x)
        need = ctx.needs_input_grad
        ctx.x_dtype, ctx.dtypes = x.dtype, _dtypes_of(weight, bias)
        with _AS_IT_IS if dtype is None else _no_autocast(x):
            x, weight, bias = _cast(x, dtype), _cast(weight, dtype), _cast(bias, dtype)
            x2 = _rows(x, x.shape[-1])
            if grad and (need[1] or need[2]):
                kept = gqt_act8_save(x2, seed=seed)
            else:
                _matrix(x2, "x")  # refuses what the copy would
                kept = None
            ctx.d = x2.shape[1]
            ctx.save_for_backward(weight if need[0] else None, *_parts(kept))
            return torch.nn.functional.linear(x, weight, bias)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        weight, codes, exps = ctx.saved_tensors
        dx = dw = db = None
        with _no_autocast(dy):
            if ctx.needs_input_grad[0]:
                dx = _cast(dy @ weight, ctx.x_dtype)
            if ctx.needs_input_grad[1] or ctx.needs_input_grad[2]:
                dw, db = _parameter_grads(_rows(dy, dy.shape[-1]), Act8(codes, exps, ctx.d),
                                          ctx.dtypes, ctx.needs_input_grad[2])
        return dx, dw, db, None, None


def linear(x, weight, bias=None, *, seed=None):
    """x w^T + bias (the library's product), differentiable, with x kept for
    the weight's gradient, where there is one, in 8 bits.  Under autocast the
    product and the copy are those of the cast x, and the gradients have the
    dtypes of x, weight and bias; autocast has to be to bf16."""
    return _Linear.apply(x, weight, bias, seed, torch.is_grad_enabled())


class _Mlp8(torch.autograd.Function):
    """norm -> up -> GELU -> down.  The norm and GELU leave the 8-bit copies
    of their input (for their own backward) and of their output (for the
    weight gradient of the product that reads it) in one pass each, as far as
    a gradient reads them."""

    @staticmethod
    def forward(ctx, x, nw, nb, w1, b1, w2, b2, eps, approximate, seed):
        dtype = _product_dtype(x)
        x2 = _rows(x, x.shape[-1])
        rows, d = x2.shape
        ff = w1.shape[0]
        seeds = _copy_seeds(seed)
        need = ctx.needs_input_grad
        x8 = _new_copy(x2) if any(need[:3]) else None
        a8 = _new_copy(x2) if need[3] or need[4] else None
        h8 = Act8.empty(rows, ff, x.device) if any(need[:5]) else None
        g8 = Act8.empty(rows, ff, x.device) if need[5] or need[6] else None
        ctx.d, ctx.ff, ctx.approximate, ctx.x_dtype = d, ff, approximate, x.dtype
        ctx.dtypes1, ctx.dtypes2 = _dtypes_of(w1, b1), _dtypes_of(w2, b2)
        with _AS_IT_IS if dtype is None else _no_autocast(x):
            w1, b1, w2, b2 = (_cast(t, dtype) for t in (w1, b1, w2, b2))
            cast = dtype is not None and dtype != x.dtype
            a, mean, rstd = gqt_layer_norm(x2, nw, nb, eps, save_x=x8, seed_x=seeds[0],
                                           save_y=None if cast else a8, seed_y=seeds[1])
            if cast:  # the copy is of what the product reads
                a = a.to(dtype)
                if a8 is not None:
                    gqt_act8_save(a, seed=seeds[1], out=a8)
            h = torch.nn.functional.linear(a, w1, b1)
            g = gqt_gelu(h, approximate, save_h=h8, seed_h=seeds[2], save_y=g8, seed_y=seeds[3])
            y = torch.nn.functional.linear(g, w2, b2)
        ctx.save_for_backward(mean, rstd, nw, w1 if any(need[:3]) else None,
                              w2 if any(need[:5]) else None, *_parts(x8), *_parts(a8),
                              *_parts(h8), *_parts(g8))
        return y.view(*x.shape[:-1], w2.shape[0])

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        mean, rstd, nw, w1, w2, *kept = ctx.saved_tensors
        d, ff = ctx.d, ctx.ff
        x8, a8, h8, g8 = (Act8(kept[2 * i], kept[2 * i + 1], (d, d, ff, ff)[i]) for i in range(4))
        need = ctx.needs_input_grad
        dy2 = _rows(dy, dy.shape[-1])
        dx = dnw = dnb = dw1 = db1 = dw2 = db2 = None
        with _no_autocast(dy):
            if need[5] or need[6]:
                dw2, db2 = _parameter_grads(dy2, g8, ctx.dtypes2, need[6])
            if any(need[:5]):
                dh = gqt_gelu_backward(dy2 @ w2, h8, ctx.approximate)
                if need[3] or need[4]:
                    dw1, db1 = _parameter_grads(dh, a8, ctx.dtypes1, need[4])
                if any(need[:3]):
                    dx, dnw, dnb = gqt_layer_norm_backward(
                        _cast(dh @ w1, ctx.x_dtype), x8, mean, rstd, nw, weight_grad=need[1],
                        bias_grad=need[2])
                    dx = dx.view(*dy.shape[:-1], d)
        return dx, dnw, dnb, dw1, db1, dw2, db2, None, None, None


def _is_plain(module, kind) -> bool:
    """Whether calling the module does what a `kind` does and no more: no
    other class (an adapter, a parametrization), forward or hook."""
    return (type(module) is kind and "forward" not in module.__dict__
            and not (module._forward_hooks or module._forward_pre_hooks
                     or module._backward_hooks or module._backward_pre_hooks
                     or torch.nn.modules.module._has_any_global_hook()))


_modules = itertools.count()  # numbers the blocks whose seed was not given


def _rank() -> int:
    dist = torch.distributed
    return dist.get_rank() if dist.is_available() and dist.is_initialized() else 0


class Mlp8(torch.nn.Module):
    """A transformer's MLP block, x + down(gelu(up(norm(x)))), that keeps
    its activations for the backward pass in 8 bits: x, norm(x), up(...) and
    gelu(...) take 33 bytes per 32 values, where bf16 copies take 64.

    random=True rounds them at random without bias, with a stream of its own
    for every copy of every forward pass (seeded by the block's seed, the
    number of the pass, and the four copies in it); otherwise to nearest.
    Without `seed` each block has its own, from torch's seed and the order of
    the blocks' first passes, and each rank of the default process group draws
    other numbers, so that rounding errors are independent; a copy of a block
    that has run shares its streams.  A `seed` is taken as it is: give each
    block, and each rank, another.  The number of passes (and a seed that was
    not given) is in the state dict, so that a resumed run goes on with new
    numbers.  The seeds are the host's: a captured graph draws the same
    numbers at every replay.

    norm, up and down run together as one operator.  One that was replaced or
    has hooks is called as it is instead, and keeps what it keeps; the others
    keep the same copies as before."""

    def __init__(self, d: int, hidden: int, *, eps: float = 1e-5, approximate: str = "tanh",
                 random: bool = True, seed: int | None = None, device=None,
                 dtype=torch.bfloat16):
        super().__init__()
        _form(approximate)
        kw = {"device": device, "dtype": dtype}
        self.norm = torch.nn.LayerNorm(d, eps=eps, **kw)
        self.up = torch.nn.Linear(d, hidden, **kw)
        self.down = torch.nn.Linear(hidden, d, **kw)
        self.approximate, self.random, self.seed, self.passes = approximate, random, seed, 0
        self._drawn = None  # the seed of a block that was given none

    def _pass_seed(self) -> int:
        if self.seed is not None:
            return _mix_seed(self.seed, self.passes)
        return _mix_seed(_mix_seed(self._draw(), _rank()), self.passes)

    def _draw(self) -> int:
        # not when the block is made: copies of one block would share it
        if self._drawn is None:
            self._drawn = _mix_seed(torch.initial_seed(), next(_modules))
        return self._drawn

    def get_extra_state(self) -> torch.Tensor:
        """The number of passes; whether the block drew its seed; that seed."""
        drew = self.random and self.seed is None
        drawn = self._draw() if drew else 0
        return torch.tensor([self.passes, drew, drawn - (drawn >> 63 << 64)], device="cpu")

    def set_extra_state(self, state: torch.Tensor):
        self.passes, drew, drawn = (int(v) for v in state.tolist())
        if drew:
            self._drawn = drawn & 0xFFFFFFFFFFFFFFFF

    def _load_from_state_dict(self, state_dict, prefix, *args):
        # a state without them leaves them as they are
        state_dict.setdefault(prefix + "_extra_state", self.get_extra_state())
        super()._load_from_state_dict(state_dict, prefix, *args)

    def forward(self, x):
        norm, up, down = self.norm, self.up, self.down
        own_norm = _is_plain(norm, torch.nn.LayerNorm)
        own_up, own_down = _is_plain(up, torch.nn.Linear), _is_plain(down, torch.nn.Linear)
        seed, bits = None, None
        if torch.is_grad_enabled():
            bits = 8
            if self.random:
                seed = self._pass_seed()
            self.passes += 1
            if own_norm and own_up and own_down:
                return x + _Mlp8.apply(x, norm.weight, norm.bias, up.weight, up.bias, down.weight,
                                       down.bias, norm.eps, self.approximate, seed)
        seeds = _copy_seeds(seed)
        a = (layer_norm(x, norm.weight, norm.bias, norm.eps, bits=bits, seed=seeds[0]) if own_norm
             else norm(x))
        h = linear(a, up.weight, up.bias, seed=seeds[1]) if bits and own_up else up(a)
        g = gelu(h, self.approximate, bits=bits, seed=seeds[2])
        return x + (linear(g, down.weight, down.bias, seed=seeds[3]) if bits and own_down
                    else down(g))
