"""Stand-ins for the device operators of `train`, in plain 64-bit arithmetic
on the CPU, so that the wrappers around them (autograd, autocast, the modules)
run without a GPU.  `calls` names what was called, in order."""
from __future__ import annotations

import numpy as np
import torch

import train_plain as plain
from allreduce_compatible_gradient_amd import train


def _np(t):
    return t.detach().double().numpy()


def _new(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype)


def values(x, d=None):
    """What an Act8 stands for, or a tensor, in 64 bits."""
    if isinstance(x, train.Act8):
        return plain.restore(x.codes.numpy(), x.exps.numpy(), x.d)
    return _np(x)


def install(monkeypatch) -> list:
    calls = []

    def save(x, *, seed=None, out=None, stream=None):
        calls.append("save")
        train._dtype(x.dtype, "x")
        out = train.Act8.empty(*x.shape, "cpu") if out is None else out
        codes, exps = plain.save(_np(x), seed)
        out.codes.copy_(torch.from_numpy(codes))
        out.exps.copy_(torch.from_numpy(exps))
        return out

    def keep(t, out, seed):
        if out is not None:
            calls.append("keep")
            codes, exps = plain.save(_np(t), seed)
            out.codes.copy_(torch.from_numpy(codes))
            out.exps.copy_(torch.from_numpy(exps))

    def layer_norm(x, weight=None, bias=None, eps=1e-5, *, stats=True, save_x=None, seed_x=None,
                   save_y=None, seed_y=None, stream=None):
        calls.append("norm")
        train._dtype(x.dtype, "x")
        train._weights(weight, bias, x.shape[1], x.device)
        w = 1.0 if weight is None else _np(weight)
        b = 0.0 if bias is None else _np(bias)
        mean, rstd = plain.norm_stats(_np(x), eps)
        y = _new(plain.layer_norm(_np(x), w, b, eps), x.dtype)
        keep(x, save_x, seed_x)
        keep(y, save_y, seed_y)
        return y, _new(mean[:, 0], torch.float32), _new(rstd[:, 0], torch.float32)

    def layer_norm_backward(dy, x, mean, rstd, weight=None, *, weight_grad=True, bias_grad=True,
                            stream=None):
        calls.append("norm backward")
        train._dtype(dy.dtype, "dy")
        w = 1.0 if weight is None else _np(weight)
        wt = torch.float32 if weight is None else weight.dtype
        dx, dw, db = plain.layer_norm_backward(_np(dy), values(x), _np(mean)[:, None],
                                               _np(rstd)[:, None], w)
        return (_new(dx, dy.dtype), _new(dw, wt) if weight_grad else None,
                _new(db, wt) if bias_grad else None)

    def gelu(h, approximate="none", *, save_h=None, seed_h=None, save_y=None, seed_y=None,
             stream=None):
        calls.append("gelu")
        train._dtype(h.dtype, "h")
        y = _new(plain.gelu(_np(h), approximate), h.dtype)
        keep(h, save_h, seed_h)
        keep(y, save_y, seed_y)
        return y

    def gelu_backward(dy, h, approximate="none", *, stream=None):
        calls.append("gelu backward")
        return _new(_np(dy) * plain.gelu_slope(values(h), approximate), dy.dtype)

    def weight_grad(dy, x, *, dtype=torch.float32, bias=True, workspace=None, stream=None):
        calls.append("weight grad")
        train._dtype(dtype, "dtype")
        dw, db = plain.weight_grad(_np(dy), values(x))
        return _new(dw, dtype), _new(db, dtype) if bias else None

    def matrix(x, name, **_):
        return train._dtype(x.dtype, name), x.shape[1]

    monkeypatch.setattr(train, "_matrix", matrix)
    for name, f in (("act8_save", save), ("layer_norm", layer_norm),
                    ("layer_norm_backward", layer_norm_backward), ("gelu", gelu),
                    ("gelu_backward", gelu_backward), ("weight_grad", weight_grad)):
        monkeypatch.setattr(train, "gqt_" + name, f)
    return calls
