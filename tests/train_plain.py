"""Plain implementations of the training operators in 64 bits, written from
their definitions (include/gq_train.h), and bounds on what fp32 arithmetic
may be off them.  numpy on the CPU; the random uniforms come from the C
oracle's Philox."""
from __future__ import annotations

import math

import numpy as np
from scipy.special import ndtr

import oracle

U = 2.0**-24  # half a step of fp32
HALF = {"f32": 2.0**-24, "bf16": 2.0**-8}  # half a step of an output, relative


def uniforms(rows: int, cols: int, seed: int) -> np.ndarray:
    """32-bit uniforms [rows, cols]: 16-bit half j % 2 of word (j % 8) / 2 of
    Philox block j / 8, draw 0 above draw 1, the row in the worker's place."""
    key = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    out = np.zeros((rows, -(-cols // 8) * 8), dtype=np.int64)
    for r in range(rows):
        for b in range(out.shape[1] // 8):
            for draw, shift in ((0, 16), (1, 0)):
                w = oracle.philox4x32_10([b, 0, r, draw], key)
                for j in range(8):
                    half = (int(w[j // 2]) >> (16 * (j % 2))) & 0xFFFF
                    out[r, 8 * b + j] |= half << shift
    return out[:, :cols]


def save(x: np.ndarray, seed=None):
    """(codes int8 [rows, 32 G], exps uint8 [rows, G]) of x, one group at a time."""
    rows, d = x.shape
    groups = -(-d // 32)
    codes = np.zeros((rows, 32 * groups), dtype=np.int8)
    exps = np.zeros((rows, groups), dtype=np.uint8)
    u = None if seed is None else uniforms(rows, 32 * groups, seed)
    for r in range(rows):
        for g in range(groups):
            v = np.zeros(32)
            part = x[r, 32 * g:32 * g + 32].astype(np.float64)
            v[:part.size] = part
            a = np.max(np.abs(v)) if np.all(np.isfinite(v)) else math.inf
            if not math.isfinite(a):
                exps[r, g] = 255
                continue
            E = -126
            while a > 127 * 2.0**E:
                E += 1
            t = v / 2.0**E  # exact in 64 bits
            if u is None:
                q = np.rint(t)
            else:
                lo = np.floor(np.abs(t))
                F = np.floor((np.abs(t) - lo) * 2.0**32)
                q = np.copysign(lo + (u[r, 32 * g:32 * g + 32] < F), t)
            top = 63 if E == 122 else 127
            codes[r, 32 * g:32 * g + 32] = np.clip(q, -top, top)
            exps[r, g] = E + 127
    return codes, exps


def restore(codes: np.ndarray, exps: np.ndarray, d: int) -> np.ndarray:
    step = np.where(exps == 255, np.nan, np.exp2(exps.astype(np.float64) - 127))
    return (codes.astype(np.float64) * np.repeat(step, 32, axis=1))[:, :d]


def norm_stats(x, eps):
    mean = x.mean(axis=1, keepdims=True)
    var = np.square(x - mean).mean(axis=1, keepdims=True)
    return mean, 1 / np.sqrt(var + eps)


def layer_norm(x, w, b, eps):
    mean, rstd = norm_stats(x, eps)
    return (x - mean) * rstd * w + b


# Sums inside a row: at most 32 additions in a thread, 6 between lanes and 16
# between waves (rows up to 16384 columns; longer ones add d / 1024 in a thread).
def gamma(d):
    return (64 + d / 1024) * U


def layer_norm_bound(x, w, b, eps, dtype):
    """|error| of y: the mean's (gamma mean|x|), then those of the deviation,
    the variance and the four roundings after them."""
    d = x.shape[1]
    mean, rstd = norm_stats(x, eps)
    dm = gamma(d) * np.abs(x).mean(axis=1, keepdims=True) + U * np.abs(mean)
    c = np.abs(x - mean)
    # the variance: its own sum, and (mean error)^2 (the first order cancels)
    rel = 0.5 * (gamma(d) + 4 * U + np.square(dm * rstd)) + 2 * U
    scaled = c * rstd * np.abs(w)
    y = scaled + np.abs(b)
    return (dm + U * np.abs(x)) * rstd * np.abs(w) * 1.01 + scaled * (rel + 4 * U) + \
        y * (2 * U + HALF[dtype] * 1.01) + 2.0**-133


def layer_norm_backward(dy, x, mean, rstd, w):
    xh = (x - mean) * rstd
    g = dy * w
    dx = rstd * (g - g.mean(axis=1, keepdims=True) - xh * (g * xh).mean(axis=1, keepdims=True))
    return dx, (dy * xh).sum(axis=0), dy.sum(axis=0)


def layer_norm_backward_bounds(dy, x, mean, rstd, w, dtype, wdtype):
    """Bounds for (dx, dw, db); mean and rstd are inputs, so xh is off by its
    two roundings.  A column's sum over the rows is a chain of at most `rows`
    additions and at most 1100 blocks' partial sums."""
    rows, d = dy.shape
    xh = np.abs((x - mean) * rstd)
    g = np.abs(dy * w)
    s1, s2 = g.mean(axis=1, keepdims=True), (g * xh).mean(axis=1, keepdims=True)
    err = rstd * ((g + s1 + xh * s2) * 8 * U + gamma(d) * (s1 + xh * s2))
    dx = layer_norm_backward(dy, x, mean, rstd, w)[0]
    chain = (min(rows, 1100) + 32) * U
    terms = np.abs(dy) * xh
    dw = terms.sum(axis=0) * (chain + 4 * U)
    db = np.abs(dy).sum(axis=0) * chain
    _, ew, eb = layer_norm_backward(dy, x, mean, rstd, w)
    return (err + np.abs(dx) * HALF[dtype] * 1.01 + 2.0**-133,
            dw + np.abs(ew) * HALF[wdtype] * 1.01 + 2.0**-133,
            db + np.abs(eb) * HALF[wdtype] * 1.01 + 2.0**-133)


def gelu(h, form):
    if form == "none":
        return h * ndtr(h)
    u = math.sqrt(2 / math.pi) * (h + 0.044715 * h**3)
    return h / (1 + np.exp(np.minimum(-2 * u, 700.0)))


def gelu_slope(h, form):
    if form == "none":
        return ndtr(h) + h * np.exp(-0.5 * h * h) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    e = np.exp(-2 * np.abs(c * (h + 0.044715 * h**3)))
    s, r = np.where(h < 0, e, 1) / (1 + e), np.where(h < 0, 1, e) / (1 + e)
    return s + 2 * h * s * r * c * (1 + 3 * 0.044715 * h * h)


def gelu_bounds(h, form):
    """Bounds on fp32 gelu and its slope, before the output's rounding: the
    exponential is off by its argument's rounding (absolute, so relative in
    the result), the fitted tail by 1.5e-7, and a few roundings."""
    if form == "none":
        tail = ndtr(-np.abs(h))
        rel = 1.5e-7 + (2 * h * h + 8) * U
        phi = np.exp(-0.5 * h * h) / math.sqrt(2 * math.pi)
        e = tail * rel + 2 * U * ndtr(h)
        return np.abs(h) * (e + U), e + np.abs(h) * phi * rel + 4 * U * np.abs(gelu_slope(h, form))
    c = math.sqrt(2 / math.pi)
    au = np.abs(c * (h + 0.044715 * h**3))
    x = np.exp(-2 * au)
    small = x / (1 + x)
    rel = (12 * au + 12) * U
    s = np.where(h < 0, small, 1 - small)
    e = small * rel + 4 * U * s
    k = np.abs(2 * h * c * (1 + 3 * 0.044715 * h * h))
    return np.abs(h) * e, e + k * small * (rel + 8 * U) + 4 * U * np.abs(gelu_slope(h, form))


def weight_grad(dy, x):
    return dy.T @ x, dy.sum(axis=0)


def weight_grad_bounds(dy, x, wdtype):
    """Every product is exact; each of the m additions (three an element for
    fp32 dy) rounds by at most one step of the running sum of magnitudes."""
    m = dy.shape[0]
    dw, db = weight_grad(dy, x)
    chain = (3 * m + 8) * 2 * U
    return (np.abs(dy).T @ np.abs(x) * chain + np.abs(dw) * HALF[wdtype] * 1.01 + 2.0**-133,
            np.abs(dy).sum(axis=0) * chain + np.abs(db) * HALF[wdtype] * 1.01 + 2.0**-133)
