"""Products of linear layers in 8-bit floating point with a scale for each
block of 128 (libgq_step.so, ``include/gq_step.h``).

A matrix is kept as e4m3 numbers, one byte a value, and a power of two for
each block: 128 columns of a row for activations and gradients (``Fp8``), a
square of 128 x 128 for weights (``Fp8Weight``, which serve the forward
product and, transposed, the one for the gradient of its input).  The matrix
cores apply the powers of two, so that y = x w^T + b runs at their 8-bit rate.
Rounding is to nearest or, given a seed, at random without bias; the gradient
of the input is linear in the copy of the gradient of the output, whose
rounding at random leaves its expectation as it is (not so the sums' own
roundings: see ``gqs_fp8_product``).

``gqs_*`` are the C entry points on CUDA (HIP) tensors, with the conventions
of ``train``'s: [rows, d] with unit column stride, new contiguous outputs,
torch's current stream unless another is given, no synchronization, no
fallback.  ``train.linear(..., fp8=True)`` and ``train.Mlp8(..., fp8=True)``
are the same under autograd.
"""
from __future__ import annotations

import functools

import torch

from ._step import check, lib
from .train import _current, _dtype, _Elsewhere, _elsewhere, _matrix, _ptr, _vector

GQS_ROUND_NEAREST = 0
GQS_ROUND_RANDOM = 1

_E4M3 = torch.float8_e4m3fn


def gqs_fp8_blocks(d: int) -> int:
    return int(lib().gqs_fp8_blocks(d))


def gqs_fp8_pitch(d: int) -> int:
    return int(lib().gqs_fp8_pitch(d))


def gqs_fp8_exp_pitch(rows: int) -> int:
    return int(lib().gqs_fp8_exp_pitch(rows))


class Fp8:
    """The row copy of a [rows, d] matrix: ``codes`` float8_e4m3fn [rows,
    128 G] and ``exps`` uint8 [G, 16 ceil(rows / 16)], G = ceil(d / 128); a
    code c of a block with exponent byte e stands for c 2^(e - 127)."""

    __slots__ = ("codes", "exps", "d")

    def __init__(self, codes: torch.Tensor, exps: torch.Tensor, d: int):
        self.codes, self.exps, self.d = codes, exps, int(d)

    @classmethod
    def empty(cls, rows: int, d: int, device) -> "Fp8":
        blocks = (int(d) + 127) // 128
        return cls(torch.empty((rows, 128 * blocks), dtype=_E4M3, device=device),
                   torch.empty((blocks, (rows + 15) // 16 * 16), dtype=torch.uint8, device=device),
                   d)

    @property
    def shape(self):
        return self.codes.shape[0], self.d

    def _tensors(self):
        return self.codes, self.exps

    def __repr__(self):
        return f"Fp8({self.shape[0]} x {self.d}, {self.codes.device})"


class Fp8Weight:
    """The copy of a weight [n, k]: ``codes`` float8_e4m3fn [n, 128 Gk],
    ``exps`` uint8 [Gn, Gk] for the squares of 128 x 128, and ``codes_t``
    [k, 128 Gn], the codes transposed.  Either may be None where only the
    product of the other is wanted (without codes, n has to be given)."""

    __slots__ = ("codes", "exps", "n", "k", "codes_t")

    def __init__(self, codes, exps: torch.Tensor, k: int, codes_t=None, n: int | None = None):
        self.codes, self.exps, self.k, self.codes_t = codes, exps, int(k), codes_t
        self.n = int(codes.shape[0] if n is None else n)

    @classmethod
    def empty(cls, n: int, k: int, device, transposed: bool = True) -> "Fp8Weight":
        gn, gk = (int(n) + 127) // 128, (int(k) + 127) // 128
        return cls(torch.empty((n, 128 * gk), dtype=_E4M3, device=device),
                   torch.empty((gn, gk), dtype=torch.uint8, device=device), k,
                   torch.empty((k, 128 * gn), dtype=_E4M3, device=device) if transposed else None)

    @property
    def shape(self):
        return self.n, self.k

    def _tensors(self):
        return self.codes, self.exps, self.codes_t

    def __repr__(self):
        return f"Fp8Weight({self.n} x {self.k}, {self.exps.device})"


def _blocks(d: int) -> int:
    return (d + 127) // 128


def _part(t, name: str, shape, dtype, device):
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise ValueError(f"{name} must be a tensor on {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {list(shape)}, got {list(t.shape)}")
    return t.data_ptr()


def _row_copy(a, name: str, rows: int, d: int, device):
    """The addresses of a row copy's codes and exps."""
    if not isinstance(a, Fp8):
        raise TypeError(f"{name} must be an Fp8, got {type(a).__name__}")
    if a.d != d:
        raise ValueError(f"{name} is the copy of {list(a.shape)}, expected {[rows, d]}")
    return (_part(a.codes, f"{name}.codes", (rows, 128 * _blocks(d)), _E4M3, device),
            _part(a.exps, f"{name}.exps", (_blocks(d), (rows + 15) // 16 * 16), torch.uint8,
                  device))


def _weight_copy(w, device, transposed: bool):
    """(codes, exps, cols, depth) of the product that reads a weight's copy."""
    if not isinstance(w, Fp8Weight):
        raise TypeError(f"w must be an Fp8Weight, got {type(w).__name__}")
    n, k = w.shape
    if n < 1 or k < 1:
        raise ValueError(f"w must be [n, k] with n, k >= 1, got {[n, k]}")
    exps = _part(w.exps, "w.exps", (_blocks(n), _blocks(k)), torch.uint8, device)
    if (w.codes_t if transposed else w.codes) is None:
        raise ValueError(f"w has no {'transposed ' if transposed else ''}codes")
    if transposed:
        return _part(w.codes_t, "w.codes_t", (k, 128 * _blocks(n)), _E4M3, device), exps, k, n
    return _part(w.codes, "w.codes", (n, 128 * _blocks(k)), _E4M3, device), exps, n, k


def _rounding(seed):
    return (GQS_ROUND_NEAREST, 0) if seed is None else (GQS_ROUND_RANDOM,
                                                         int(seed) & 0xFFFFFFFFFFFFFFFF)


def _tensors_of(*given):
    """The tensors of what a call was given, for its stream to hold."""
    held = []
    for t in given:
        held.extend(t._tensors() if isinstance(t, (Fp8, Fp8Weight)) else (t,))
    return held


def gqs_fp8_rows(x: torch.Tensor, *, seed=None, out: Fp8 | None = None, stream=None) -> Fp8:
    """The row copy of x [rows, d]: to nearest, or with a 64-bit `seed` at
    random without bias."""
    dt, ldx = _matrix(x, "x")
    device = x.device
    if _elsewhere(device, stream):
        with _Elsewhere(device, stream, _tensors_of(x, out)):
            return gqs_fp8_rows(x, seed=seed, out=out)
    rows, d = x.shape
    if out is None:
        out = Fp8.empty(rows, d, device)
    codes, exps = _row_copy(out, "out", rows, d, device)
    check(lib().gqs_fp8_rows(x.data_ptr(), dt, rows, d, ldx, *_rounding(seed), codes, exps,
                             _current(device)))
    return out


def gqs_fp8_weight(w: torch.Tensor, *, transposed: bool = True, out: Fp8Weight | None = None,
                   stream=None) -> Fp8Weight:
    """The copy of a weight [n, k], to nearest; with its transposed codes
    unless they are not wanted (with `out`, which needs codes: if it has
    them)."""
    dt, ldw = _matrix(w, "w")
    device = w.device
    if _elsewhere(device, stream):
        with _Elsewhere(device, stream, _tensors_of(w, out)):
            return gqs_fp8_weight(w, transposed=transposed, out=out)
    n, k = w.shape
    if n < 1:
        raise ValueError("w must be [n, k] with n >= 1")
    if out is None:
        out = Fp8Weight.empty(n, k, device, transposed)
    elif not isinstance(out, Fp8Weight) or out.shape != (n, k):
        raise ValueError(f"out must be the Fp8Weight of {[n, k]}")
    codes, exps, _, _ = _weight_copy(out, device, False)
    codes_t = None if out.codes_t is None else _weight_copy(out, device, True)[0]
    check(lib().gqs_fp8_weight(w.data_ptr(), dt, n, k, ldw, codes, codes_t, exps,
                               _current(device)))
    return out


def gqs_fp8_restore(a, dtype=torch.bfloat16, *, stream=None) -> torch.Tensor:
    """The values an Fp8 or Fp8Weight (with its codes) stands for, exact in
    either dtype."""
    dt = _dtype(dtype, "dtype")
    if not isinstance(a, (Fp8, Fp8Weight)) or not a.exps.is_cuda:
        raise ValueError("a must be an Fp8 or Fp8Weight on a device")
    device = a.exps.device
    if _elsewhere(device, stream):
        with _Elsewhere(device, stream, _tensors_of(a)):
            return gqs_fp8_restore(a, dtype)
    rows, d = a.shape
    squares = isinstance(a, Fp8Weight)
    if squares:
        codes, exps, _, _ = _weight_copy(a, device, False)
    else:
        codes, exps = _row_copy(a, "a", rows, d, device)
    out = torch.empty((rows, d), dtype=dtype, device=device)
    check(lib().gqs_fp8_restore(codes, exps, rows, d, squares, dt, out.data_ptr(),
                                _current(device)))
    return out


@functools.lru_cache(maxsize=1024)
def _need(entry: str, m: int, cols: int, depth: int, dt: int) -> int:
    """A workspace's bytes, which depend on nothing else."""
    return int(getattr(lib(), entry)(m, cols, depth, dt))


def _workspace(workspace, need: int, device):
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=device) if need > 0 else None
    if (not isinstance(workspace, torch.Tensor) or workspace.device != device
            or not workspace.is_contiguous()
            or workspace.numel() * workspace.element_size() < need):
        raise ValueError(f"workspace must be contiguous, on {device}, of {need} bytes")
    return workspace


def _bias(bias, cols: int, device) -> int:
    _vector(bias, "bias", cols, device)
    return 0 if bias is None else _dtype(bias.dtype, "bias")


def gqs_fp8_product_workspace_bytes(m: int, cols: int, depth: int, dtype=torch.bfloat16) -> int:
    return int(lib().gqs_fp8_product_workspace_bytes(m, cols, depth, _dtype(dtype, "dtype")))


def gqs_fp8_product(x: Fp8, w: Fp8Weight, bias=None, *, transposed: bool = False,
                    dtype=torch.bfloat16, workspace=None, stream=None) -> torch.Tensor:
    """x w^T + bias, or with `transposed` x w + bias, from the copies; the
    result and its sums in `dtype` and fp32 (fp32 results, and bf16 ones of
    few rows, are exact products summed in fp32; for bf16 ones of many rows
    the matrix cores add the products of 8-bit values in groups of eight, each
    of which can lose up to 7 2^-13 of its largest)."""
    dt = _dtype(dtype, "dtype")
    if not isinstance(x, Fp8) or not isinstance(x.codes, torch.Tensor) or not x.codes.is_cuda:
        raise ValueError("x must be an Fp8 on a device")
    device = x.codes.device
    if _elsewhere(device, stream):
        with _Elsewhere(device, stream, _tensors_of(x, w, bias, workspace)):
            return gqs_fp8_product(x, w, bias, transposed=transposed, dtype=dtype,
                                   workspace=workspace)
    codes, exps, cols, depth = _weight_copy(w, device, transposed)
    m = x.codes.shape[0]
    x_codes, x_exps = _row_copy(x, "x", m, depth, device)
    bdt = _bias(bias, cols, device)
    y = torch.empty((m, cols), dtype=dtype, device=device)
    need = _need("gqs_fp8_product_workspace_bytes", m, cols, depth, dt)
    workspace = _workspace(workspace, need, device)
    check(lib().gqs_fp8_product(x_codes, x_exps, m, codes, exps, cols, depth, transposed,
                                _ptr(bias), bdt, y.data_ptr(), dt, _ptr(workspace), max(need, 0),
                                _current(device)))
    return y


def gqs_fp8_linear_workspace_bytes(m: int, cols: int, depth: int, dtype=torch.bfloat16) -> int:
    return int(lib().gqs_fp8_linear_workspace_bytes(m, cols, depth, _dtype(dtype, "dtype")))


def gqs_fp8_linear(x: torch.Tensor, w: Fp8Weight, bias=None, *, transposed: bool = False,
                   seed=None, workspace=None, stream=None) -> torch.Tensor:
    """x w^T + bias, or with `transposed` x w + bias, of x [m, depth] whose
    row copy (with a `seed` rounded at random) is made on the way; the result
    has x's dtype."""
    dt, ldx = _matrix(x, "x")
    device = x.device
    if _elsewhere(device, stream):
        with _Elsewhere(device, stream, _tensors_of(x, w, bias, workspace)):
            return gqs_fp8_linear(x, w, bias, transposed=transposed, seed=seed,
                                  workspace=workspace)
    codes, exps, cols, depth = _weight_copy(w, device, transposed)
    m, d = x.shape
    if d != depth:
        raise ValueError(f"x is {list(x.shape)}, expected {depth} columns")
    bdt = _bias(bias, cols, device)
    y = torch.empty((m, cols), dtype=x.dtype, device=device)
    need = _need("gqs_fp8_linear_workspace_bytes", m, cols, depth, dt)
    workspace = _workspace(workspace, need, device)
    check(lib().gqs_fp8_linear(x.data_ptr(), dt, m, depth, ldx, *_rounding(seed), codes, exps,
                               cols, transposed, _ptr(bias), bdt, y.data_ptr(), _ptr(workspace),
                               max(need, 0), _current(device)))
    return y
