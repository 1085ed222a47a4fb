"""Plain implementations of the step's operators in 64 bits, written from
their definitions (include/gq_step.h), and bounds on what the kernels'
arithmetic may be off them.  numpy on the CPU."""
from __future__ import annotations

import math

import numpy as np

U = 2.0**-24  # half a step of fp32
HALF = {"f32": 2.0**-24, "bf16": 2.0**-8}  # half a step of an output, relative

M32 = np.uint64(0xFFFFFFFF)


def halves(counters, seed: int) -> np.ndarray:
    """[N, 8] 16-bit halves of the Philox4x32-10 blocks at counters [N, 4]."""
    x = [np.asarray(c, dtype=np.uint64) for c in np.asarray(counters).T]
    k = [np.uint64(seed & 0xFFFFFFFF), np.uint64((seed >> 32) & 0xFFFFFFFF)]
    for _ in range(10):
        a, c = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(c >> np.uint64(32)) ^ x[1] ^ k[0], c & M32, (a >> np.uint64(32)) ^ x[3] ^ k[1],
             a & M32]
        k = [(k[0] + np.uint64(0x9E3779B9)) & M32, (k[1] + np.uint64(0xBB67AE85)) & M32]
    w = np.stack(x, axis=1).astype(np.int64)
    return np.stack((w & 0xFFFF, w >> 16), axis=2).reshape(len(w), 8)


def grid(bits: int, bias: int, top: float) -> np.ndarray:
    """The numbers of a format of 3 mantissa bits, by code."""
    c = np.arange(2**bits)
    v = np.where(c < 8, c * 2.0 ** (-2 - bias), (1 + (c & 7) / 8) * np.exp2((c >> 3) - float(bias)))
    return v[v <= top]


E4M3, E5M3 = grid(7, 7, 448.0), grid(8, 16, 61440.0)
LOWEST = {448.0: -117, 61440.0: -108}


def block(v: np.ndarray, table: np.ndarray, u=None):
    """(codes without their signs, exponent byte) of a block."""
    a = np.max(np.abs(v)) if np.all(np.isfinite(v)) else math.inf
    if not math.isfinite(a):
        return np.zeros(v.shape, dtype=np.int64), 255
    E = LOWEST[table[-1]]
    while a > table[-1] * 2.0**E:
        E += 1
    t = np.abs(v) / 2.0**E
    lo = np.clip(np.searchsorted(table, t, side="right") - 1, 0, len(table) - 2)
    f = (t - table[lo]) / (table[lo + 1] - table[lo])
    if u is None:
        up = (f > 0.5) | ((f == 0.5) & (lo % 2 == 1))
    else:
        f = np.where(lo < 8, np.rint(f * 2.0**20) / 2.0**20, f)
        up = u + np.floor(f * 65536 + 0.5) >= 65536
    q = lo + up
    # values from 2^128 on have no float
    q = np.minimum(q, np.searchsorted(table * 2.0**E, 2.0**128) - 1)
    return q, E + 127


def step_of(exps) -> np.ndarray:
    e = np.asarray(exps, dtype=np.float64)
    return np.where(e == 255, np.nan, np.exp2(e - 127))


def signed(codes: np.ndarray) -> np.ndarray:
    """The numbers of e4m3 bytes."""
    c = codes.astype(np.int64)
    return np.where(c & 128, -1.0, 1.0) * np.append(E4M3, np.nan)[c & 127]


def _blocks(x, u):
    """e4m3 bytes and exponent bytes of the rows of x [N, size]."""
    codes = np.zeros(x.shape, dtype=np.uint8)
    exps = np.zeros(len(x), dtype=np.uint8)
    for i in range(len(x)):
        q, exps[i] = block(x[i], E4M3, None if u is None else u[i])
        codes[i] = q | np.where(np.signbit(x[i]) & (exps[i] != 255), 128, 0)
    return codes, exps


def rows(x: np.ndarray, seed=None):
    """(codes uint8 [rows, 128 G], exps uint8 [G, rows]) of x."""
    n, d = x.shape
    g = -(-d // 128)
    v = np.zeros((n, 128 * g))
    v[:, :d] = x
    u = None
    if seed is not None:
        c = np.zeros((n, 16 * g, 4), dtype=np.int64)
        c[:, :, 0] = np.arange(16 * g)
        c[:, :, 2] = np.arange(n)[:, None]
        u = halves(c.reshape(-1, 4), seed).reshape(-1, 128)
    codes, exps = _blocks(v.reshape(-1, 128), u)
    return codes.reshape(n, 128 * g), exps.reshape(n, g).T


def rows_values(codes, exps, d):
    return (signed(codes) * np.repeat(step_of(exps.T), 128, axis=1))[:, :d]


def weight(w: np.ndarray):
    """(codes [n, 128 Gk], exps [Gn, Gk], codes_t [k, 128 Gn])."""
    n, k = w.shape
    gn, gk = -(-n // 128), -(-k // 128)
    v = np.zeros((128 * gn, 128 * gk))
    v[:n, :k] = w
    squares = v.reshape(gn, 128, gk, 128).transpose(0, 2, 1, 3).reshape(gn * gk, -1)
    codes, exps = _blocks(squares, None)
    codes = codes.reshape(gn, gk, 128, 128).transpose(0, 2, 1, 3).reshape(128 * gn, -1)
    return codes[:n], exps.reshape(gn, gk), np.ascontiguousarray(codes[:, :k].T)


def weight_values(codes, exps, k):
    n = len(codes)
    step = np.repeat(np.repeat(step_of(exps), 128, axis=0), 128, axis=1)[:n]
    return (signed(codes) * step)[:, :k]


def product_bound(x, w, dtype, exact):
    """|error| of x w^T [m, n] before its bias: the fp32 sums (one rounding an
    addition, at most 2 U of the magnitudes' sum each) and the output's
    rounding; for 8-bit MFMAs also what they cut off: within a group of eight
    products, the part of each below 2^-13 of the largest's leading bit, so
    at most 7 times 2^-13 of the largest, which the group's magnitudes cover."""
    mag = np.abs(x) @ np.abs(w).T
    chain = (x.shape[1] + 64) * 2 * U
    cut = 0.0 if exact else 7 * 2.0**-13
    return mag * (chain + cut) + (np.abs(x @ w.T) + mag * cut) * HALF[dtype] * 1.01 + 2.0**-133


def moment(v: np.ndarray, second: bool, step=0, tensor=0, seed=0):
    """(codes uint8 [128 G], exps uint8 [G]) of a moment rounded at random."""
    n = len(v)
    g = -(-n // 128)
    x = np.zeros(128 * g)
    x[:n] = v
    c = np.zeros((16 * g, 4), dtype=np.int64)
    c[:, 0], c[:, 1], c[:, 2], c[:, 3] = np.arange(16 * g), step, tensor, int(second)
    u = halves(c, seed).reshape(-1, 128)
    if not second:
        codes, exps = _blocks(x.reshape(-1, 128), u)
        return codes.reshape(-1), exps
    codes, exps = np.zeros((g, 128), dtype=np.uint8), np.zeros(g, dtype=np.uint8)
    for i in range(g):
        codes[i], exps[i] = block(x[128 * i:128 * i + 128], E5M3, u[i])
    return codes.reshape(-1), exps


def moment_values(codes, exps, n, second):
    v = E5M3[codes] if second else signed(codes)
    return (v.reshape(-1, 128) * step_of(exps)[:, None]).reshape(-1)[:n]


def adamw(p, g, m, v, t, lr, beta1, beta2, eps, decay, scale=1.0):
    """(p, m, v) after step t."""
    g = g * scale
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    change = (m / (1 - beta1**t)) / (np.sqrt(v / (1 - beta2**t)) + eps)
    return p * (1 - lr * decay) - lr * change, m, v


def adamw_bounds(p, g, m, v, t, lr, beta1, beta2, eps, decay, scale=1.0):
    """Bounds for fp32 (p, m, v), before a bf16 rounding: constants, products
    and sums round by U each.  m: b1 and 1 - b1, the scaled gradient, their
    product, the sum: 5 U of the magnitudes; v the same with the gradient
    squared: 7 U.  The change: m's error, and relative ones of v's root (half
    of v's), the constants, the root, its sum with eps, the quotient: 12 U; p:
    its decay and the sum 3 U.  2^-149 for what is subnormal."""
    g = np.abs(g * scale)
    mm = beta1 * np.abs(m) + (1 - beta1) * g
    vv = beta2 * v + (1 - beta2) * g * g
    root = np.sqrt(vv / (1 - beta2**t)) + eps
    tiny = 2.0**-148
    em = 5 * U * mm * 1.01 + tiny
    ev = 7 * U * vv * 1.01 + tiny
    with np.errstate(divide="ignore", invalid="ignore"):
        change = np.where(root > 0, mm / (1 - beta1**t) / root, 0.0)
        # an absolute error of v moves its root by at most tiny / root
        sub = np.where(vv > 0, tiny / vv, 0.0)
    ep = lr * change * ((5 + 12) * U + sub) * 1.02 + 3 * U * (np.abs(p) + lr * change) * 1.02
    return ep + tiny, em, ev
