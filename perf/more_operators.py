"""Cases of the step's operators: products in 8-bit floating point with a scale
for each block of 128, and AdamW over many tensors with states in 32 or 8
bits, the gradients clipped by their norm.

Every case is one pass as a training or serving program makes it.  ``run``
computes it in plain torch operations, or, where ``own`` is true, through
``allreduce_compatible_gradient_amd.fp8`` and ``.optim``; ``exact`` computes
the same outputs from the definitions in 64 bits.

e4m3 blocks: a block's values share a power of two 2^E.  With a the largest
|x| of the block, E is the smallest integer >= -117 with a <= 448 2^E, and a
value is kept as e4m3(x 2^-E).  The blocks of activations and gradients are
128 columns of a row, those of a weight squares of 128 x 128, those of a first
moment 128 elements.  A second moment has blocks of 128 elements too, with
codes of 5 exponent and 3 mantissa bits and no sign, up to 61440 (multiples of
2^-18 below 2^-15), and E >= -108.

Rounding is to nearest (ties to even) or, given a seed, at random without
bias: with f the fraction of the way from the lower neighbour of |x| 2^-E to
the upper, up where u + floor(f 2^16 + 1/2) >= 2^16.  u are the 16-bit halves
of Philox4x32-10 words, eight to a counter: for a matrix (column / 8, 0, row,
0); for an element i of the optimizer's tensor k in step t (i / 8, t, k, draw)
with draw 0 for the first moment, 1 for the second, 2 for a bf16 parameter,
whose 16 dropped bits get u added.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
DEVICE = "cuda"
LR, BETA1, BETA2, EPS, DECAY, MAX_NORM = 1e-3, 0.9, 0.999, 1e-8, 0.01, 1.0


# ---------------------------------------------------------------------------
# the cases

def _linear(name, what, m, n, k, dtype):
    return {"name": name, "op": "linear", "what": what, "m": m, "n": n, "k": k, "dtype": dtype}


def _adamw(name, blocks, d, hidden, dtype, grad, bits, clip, step):
    return {"name": name, "op": "adamw", "blocks": blocks, "d": d, "hidden": hidden,
            "dtype": dtype, "grad": grad, "bits": bits, "clip": clip, "step": step}


def listed():
    return [
        # one token through an up projection, weights laid out before: latency
        _linear("linear 1x1024 to 4096 bf16", "forward", 1, 4096, 1024, "bf16"),
        # sixteen sequences' next tokens through a down projection
        _linear("linear 16x4096 to 1024 bf16", "forward", 16, 1024, 4096, "bf16"),
        # a larger serving batch, between the two regimes
        _linear("linear 96x4096 to 4096 bf16", "forward", 96, 4096, 4096, "bf16"),
        # odd sizes of all three axes, fp32
        _linear("linear 1000x777 to 1001 f32", "forward", 1000, 1001, 777, "f32"),
        # evaluation of a large batch
        _linear("linear 8192x1024 to 4096", "forward", 8192, 4096, 1024, "bf16"),
        # a training step: weights cast anew, y and dx, dy rounded at random
        _linear("linear step 4096 1024x1024 f32", "step", 4096, 1024, 1024, "f32"),
        _linear("linear step 8192 4096x4096", "step", 8192, 4096, 4096, "bf16"),
        # an update of one small block's six tensors: latency
        _adamw("adamw 1 block 64x100 f32", 1, 64, 100, "f32", "f32", 32, False, 1),
        # a stack of MLP blocks trained in fp32, clipped
        _adamw("adamw 4x1024x4096 f32 clip", 4, 1024, 4096, "f32", "f32", 32, True, 10),
        # the depth and width of a medium language model, bf16 weights rounded at random
        _adamw("adamw 24x1024x4096 bf16", 24, 1024, 4096, "bf16", "bf16", 32, False, 1000),
        # 8-bit states, bf16 weights, clipped
        _adamw("adamw 8-bit 4x1024x4096 bf16", 4, 1024, 4096, "bf16", "bf16", 8, True, 100),
        # 8-bit states of odd tensors, fp32 weights, bf16 gradients
        _adamw("adamw 8-bit 3x1001x777 f32", 3, 1001, 777, "f32", "bf16", 8, False, 2),
    ]


def _log_uniform(rng, lo, hi):
    """A whole number in [lo, hi], uniform in its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.5:
        dtype, what = rng.choice(["bf16", "bf16", "f32"]), rng.choice(["forward", "step"])
        n, k = _log_uniform(rng, 16, 8192), _log_uniform(rng, 16, 8192)
        most = 8192 * 4096 * 4096 // (2 if dtype == "f32" else 1) // (n * k)
        case = _linear("", what, _log_uniform(rng, 1, min(16384, most)), n, k, dtype)
    else:
        bits, dtype = rng.choice([8, 8, 32]), rng.choice(["bf16", "f32"])
        d, hidden = _log_uniform(rng, 16, 2048), _log_uniform(rng, 16, 8192)
        most = (4 if bits == 8 else 14) * 2 * 1024 * 4096 // (2 * d * hidden + 3 * d + hidden)
        case = _adamw("", _log_uniform(rng, 1, max(1, min(24, most))), d, hidden, dtype,
                      "bf16" if dtype == "bf16" else rng.choice(["bf16", "f32"]), bits,
                      rng.random() < 0.5, _log_uniform(rng, 1, 10000))
    del case["name"]
    return case


# ---------------------------------------------------------------------------
# inputs

def _activations(rows, d, g):
    """Normal values with a mean, and a few channels far larger than the rest."""
    scale = torch.ones(d, device=DEVICE)
    scale[torch.rand(d, device=DEVICE, generator=g) < 0.01] = 20.0
    x = torch.randn(rows, d, device=DEVICE, generator=g)
    return x.mul_(scale).add_(0.1 * torch.randn(d, device=DEVICE, generator=g))


def _sizes(case):
    """The tensors of a stack of MLP blocks: norm, up, down."""
    d, h = case["d"], case["hidden"]
    return [d, d, h * d, h, d * h, d] * case["blocks"]


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    t = DTYPES[case["dtype"]]
    state = dict(case, seed=seed * 0x9E3779B9 + 7)
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        state["x"] = _activations(m, k, g).to(t)
        w = (torch.randn(n, k, device=DEVICE, generator=g) / math.sqrt(k)).to(t)
        state["b"] = (0.1 * torch.randn(n, device=DEVICE, generator=g)).to(t)
        if case["what"] == "step":
            state["w"] = w
            token = torch.exp(torch.randn(m, 1, device=DEVICE, generator=g))
            dy = torch.randn(m, n, device=DEVICE, generator=g)
            state["dy"] = dy.mul_(0.001 * token).to(t)
        else:  # a serving program keeps its weights' codes
            q, e = _to_e4m3(_squares(w.float()), None)
            state["codes"] = _from_squares(q, n, -(-k // 128) * 128).to(torch.float8_e4m3fn)
            state["exps"] = (e + 127).reshape(-(-n // 128), -1).to(torch.uint8)
        return state
    # parameters, gradients and states as views of one buffer each, every
    # tensor beginning at a multiple of 128 elements; zeros between
    sizes = _sizes(case)
    starts = np.concatenate(([0], np.cumsum([-(-n // 128) * 128 for n in sizes]))).tolist()
    total = starts[-1]
    gt = DTYPES[case["grad"]]
    held = torch.zeros(total, dtype=torch.bool, device=DEVICE)
    for n, at in zip(sizes, starts):
        held[at:at + n] = True

    def values(scale, kind=torch.randn):
        return torch.where(held, kind(total, device=DEVICE, generator=g), 0.0).mul_(scale)
    # each block of gradients has a size of its own, as channels do
    size = torch.exp(torch.randn(total // 128, device=DEVICE, generator=g)).repeat_interleave(128)
    state["p"] = values(0.02).to(t)
    state["g"] = values(0.001 * size).to(gt)
    first = case["step"] == 1
    m = values(0.0 if first else 0.0003 * size)
    v = values(0.0 if first else 1e-6 * size * size, torch.rand)
    if case["bits"] == 8:
        q, e = _to_e4m3(m.view(-1, 128), state["seed"] + 1)
        state["m"] = q.reshape(-1).to(torch.float8_e4m3fn)
        state["m_exps"] = (e + 127).reshape(-1).to(torch.uint8)
        q, e = _to_e5m3(v.view(-1, 128), state["seed"] + 2)
        state["v"] = _e5m3_codes(q).reshape(-1)
        state["v_exps"] = (e + 127).reshape(-1).to(torch.uint8)
    else:
        state["m"], state["v"] = m, v
    state["sizes"], state["starts"] = sizes, starts
    for key in ("p", "g", "m", "v"):
        state[key + "_views"] = [state[key][a:a + (-(-n // 128) * 128 if case["bits"] == 8 and
                                                   key in "mv" else n)]
                                 for n, a in zip(sizes, starts)]
    if case["bits"] == 8:
        for key in ("m", "v"):
            state[key + "_exps_views"] = [state[key + "_exps"][a // 128:b // 128]
                                          for a, b in zip(starts, starts[1:])]
    return state


# ---------------------------------------------------------------------------
# the plain forms

def _philox(c0, c1, c2, c3, seed):
    """The four 32-bit words (int64 tensors) of Philox4x32-10 at counter
    (c0, c1, c2, c3) under the 64-bit key `seed`."""
    low = 0xFFFFFFFF
    k0, k1 = seed & low, (seed >> 32) & low
    c1, c3 = torch.full_like(c0, c1), torch.full_like(c0, c3)
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # the low 64 bits of each product
        c0, c1, c2, c3 = ((p1 >> 32) & low) ^ c1 ^ k0, p1 & low, ((p0 >> 32) & low) ^ c3 ^ k1, \
            p0 & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return c0, c1, c2, c3


def _halves(c0, c1, c2, c3, seed):
    """Eight 16-bit uniforms (fp32, exact) for each counter, last axis 8 times as long."""
    words = torch.stack([w.int() for w in _philox(c0, c1, c2, c3, seed)], dim=-1)
    return torch.stack((words & 0xFFFF, (words >> 16) & 0xFFFF), dim=-1).flatten(-3).float()


def _matrix_halves(rows, cols, seed):
    row = torch.arange(rows, device=DEVICE)[:, None]
    block = torch.arange(-(-cols // 8), device=DEVICE)[None, :]
    return _halves(block.expand(rows, -1), 0, row.expand(-1, block.shape[1]), 0, seed)


def _element_halves(s, draw_index):
    """Those of the optimizer's tensors, [total]."""
    eighths = torch.tensor(s["starts"], device=DEVICE) // 8
    tensor = torch.repeat_interleave(torch.arange(len(s["sizes"]), device=DEVICE),
                                     eighths.diff(), output_size=s["starts"][-1] // 8)
    i = torch.arange(s["starts"][-1] // 8, device=DEVICE) - eighths[tensor]
    return _halves(i, s["step"], tensor, draw_index, s["seed"])


def _pow2(e):
    """2^e in fp32, exactly, for whole -126 <= e <= 127."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _step_exponent(v, top, lowest):
    """E of each block (the last axis): the smallest with max <= top 2^E."""
    a = v.abs().amax(dim=-1, keepdim=True)
    mantissa, exponent = torch.frexp(a)  # a = mantissa 2^exponent, mantissa in [0.5, 1)
    tm, te = math.frexp(top)
    e = exponent - te + (mantissa > tm)
    return torch.where(a == 0, torch.full_like(e, lowest), e.clamp(min=lowest))


def _round_float(t, least, u):
    """t >= 0 on the grid of 3 mantissa bits with exponents from `least` on."""
    exponent = (torch.frexp(t)[1] - 1).clamp(min=least)
    ulp = _pow2(exponent - 3)
    c = t / ulp
    if u is None:
        return c.round() * ulp
    lo = c.floor()
    return (lo + (u + torch.floor((c - lo) * 65536 + 0.5) >= 65536)) * ulp


def _to_e4m3(v, seed, u=None):
    """fp32 e4m3 values and E of blocks along v's last axis."""
    e = _step_exponent(v, 448.0, -117)
    if seed is not None and u is None:
        u = _matrix_halves(v.shape[0], v[0].numel(), seed)[:, :v[0].numel()].reshape(v.shape)
    t = v * _pow2(-e)
    q = _round_float(t.abs(), -6, u)
    return torch.copysign(torch.where(e == 120, q.clamp(max=240.0), q), t), e


def _to_e5m3(v, seed, u=None):
    e = _step_exponent(v, 61440.0, -108)
    if u is None:
        u = _matrix_halves(v.shape[0], v.shape[1], seed)
    return _round_float(v * _pow2(-e), -15, u), e


def _e5m3_codes(q):
    mantissa, exponent = torch.frexp(q)
    normal = (exponent + 15) * 8 + (mantissa * 16 - 8).int()
    return torch.where(q < 2.0**-15, (q * 2.0**18).int(), normal).to(torch.uint8)


def _e5m3_values(codes):
    c = codes.int()
    normal = (1 + (c & 7).float() / 8) * _pow2((c >> 3) - 16)
    return torch.where(c < 8, c.float() * 2.0**-18, normal)


def _stepped(q, exps):
    """Blocks [..., 128] of values times their steps."""
    return q * _pow2(exps.int() - 127)


def _blocks_of_rows(v):
    rows, d = v.shape
    return torch.nn.functional.pad(v, (0, -d % 128)).reshape(rows, -1, 128)


def _squares(w):
    n, k = w.shape
    w = torch.nn.functional.pad(w, (0, -k % 128, 0, -n % 128))
    return w.reshape(-(-n // 128), 128, -1, 128).transpose(1, 2).flatten(2)


def _from_squares(q, n, k):
    return q.unflatten(2, (128, 128)).transpose(1, 2).flatten(2).flatten(0, 1)[:n, :k]


def _rows_values(x, seed):
    q, e = _to_e4m3(_blocks_of_rows(x.float()), seed)
    return (q * _pow2(e)).flatten(1)[:, :x.shape[1]]


def _plain_linear(s):
    n, k = s["n"], s["k"]
    if s["what"] == "step":
        q, e = _to_e4m3(_squares(s["w"].float()), None)
        w = _from_squares((q * _pow2(e)), n, k)
    else:
        step = s["exps"].repeat_interleave(128, dim=0)[:n, :, None]
        w = _stepped(s["codes"].float().reshape(n, -1, 128), step).flatten(1)[:, :k]
    y = _rows_values(s["x"], None) @ w.t() + s["b"].float()
    if s["what"] == "forward":
        return {"y": y.to(s["x"].dtype)}
    dx = _rows_values(s["dy"], s["seed"]) @ w
    return {"y": y.to(s["x"].dtype), "dx": dx.to(s["x"].dtype)}


def _plain_adamw(s):
    t, out = s["step"], {}
    g = s["g"].float()
    if s["clip"]:
        norm = torch.sqrt((g * g).sum(dtype=torch.float64))
        g = g * (MAX_NORM / (norm + 1e-6)).clamp(max=1.0).float()
        out["norm"] = norm.float()
    m, v = s["m"], s["v"]
    if s["bits"] == 8:
        m = _stepped(m.float().view(-1, 128), s["m_exps"][:, None]).view(-1)
        v = _stepped(_e5m3_values(v).view(-1, 128), s["v_exps"][:, None]).view(-1)
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * (g * g)
    c1, c2 = 1 - BETA1**t, 1 - BETA2**t
    change = m / (torch.sqrt(v) / math.sqrt(c2) + EPS)
    p = s["p"].float() * (1 - LR * DECAY) - (LR / c1) * change
    if s["p"].dtype == torch.bfloat16:
        bits = p.view(torch.int32) + _element_halves(s, 2).int()
        p = (bits & -65536).view(torch.float32)
    s["p"].copy_(p)
    if s["bits"] == 8:
        q, e = _to_e4m3(m.view(-1, 128), None, _element_halves(s, 0).view(-1, 128))
        s["m"].copy_(q.view(-1))
        s["m_exps"].copy_((e + 127).view(-1))
        m = (q * _pow2(e)).view(-1).to(torch.bfloat16)
        q, e = _to_e5m3(v.view(-1, 128), None, _element_halves(s, 1).view(-1, 128))
        s["v"].copy_(_e5m3_codes(q).view(-1))
        s["v_exps"].copy_((e + 127).view(-1))
        v = (q * _pow2(e)).view(-1).to(torch.bfloat16)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    s["step"] = t + 1
    return {"p": s["p"], "m": m, "v": v, **out}


def _plain(s):
    return _plain_linear(s) if s["op"] == "linear" else _plain_adamw(s)


# ---------------------------------------------------------------------------
# the framework's calls

def _own_linear(s):
    from allreduce_compatible_gradient_amd import fp8
    if s["what"] == "forward":
        w = fp8.Fp8Weight(s["codes"], s["exps"], s["k"])
        return {"y": fp8.gqs_fp8_linear(s["x"], w, s["b"])}
    w = fp8.gqs_fp8_weight(s["w"])
    return {"y": fp8.gqs_fp8_linear(s["x"], w, s["b"]),
            "dx": fp8.gqs_fp8_linear(s["dy"], w, transposed=True, seed=s["seed"])}


def _own_adamw(s):
    from allreduce_compatible_gradient_amd import optim
    out, scale = {}, None
    if s["clip"]:
        out["norm"], scale = optim.gqs_grad_norm(s["g_views"], max_norm=MAX_NORM)
    m, v = s["m_views"], s["v_views"]
    if s["bits"] == 8:
        m = [optim.Moment8(*x) for x in zip(m, s["m_exps_views"], s["sizes"])]
        v = [optim.Moment8(*x) for x in zip(v, s["v_exps_views"], s["sizes"])]
    optim.gqs_adamw(s["p_views"], s["g_views"], m, v, step=s["step"], lr=LR,
                    betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY, scale=scale,
                    seed=s["seed"])
    s["step"] += 1
    out["p"], out["m"], out["v"] = s["p"], s["m"], s["v"]
    if s["bits"] == 8:
        for key in ("m", "v"):
            whole = optim.Moment8(s[key], s[key + "_exps"], s[key].numel())
            out[key] = optim.gqs_moment8_restore(whole, torch.bfloat16)
    return out


def run(state):
    if not own:
        return _plain(state)
    return _own_linear(state) if state["op"] == "linear" else _own_adamw(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    size = {"bf16": 2, "f32": 4}
    b = size[case["dtype"]]
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        if case["what"] == "forward":  # x, the weight's codes, the bias, y
            return {"bytes": (m * k + n + m * n) * b + n * k, "flops": 2 * m * n * k}
        # x, dy, w and the bias read, y and dx written
        return {"bytes": (2 * m * k + 2 * m * n + n * k + n) * b, "flops": 4 * m * n * k}
    count = sum(_sizes(case))
    # p read and written, g read, both states read and written; those in 8
    # bits are also returned as bf16 values
    states = 2 * (1 + 1 / 128 + 1) * 2 if case["bits"] == 8 else 16
    return {"bytes": count * (2 * b + size[case["grad"]] + states), "flops": 20 * count}


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def _exact_halves(count, c0, c1, c2, c3, seed):
    """[count, 8] 16-bit halves as doubles; c0 to c3 whole numbers or arrays."""
    u32, s32 = np.uint64(0xFFFFFFFF), np.uint64(32)
    x = [np.broadcast_to(np.asarray(c, dtype=np.uint64), (count,)) for c in (c0, c1, c2, c3)]
    key = [np.uint64(seed & 0xFFFFFFFF), np.uint64((seed >> 32) & 0xFFFFFFFF)]
    for _ in range(10):
        a, c = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(c >> s32) ^ x[1] ^ key[0], c & u32, (a >> s32) ^ x[3] ^ key[1], a & u32]
        key = [(key[0] + np.uint64(0x9E3779B9)) & u32, (key[1] + np.uint64(0xBB67AE85)) & u32]
    words = np.stack([w.astype(np.uint32) for w in x], axis=1)
    return torch.from_numpy(words.view("<u2").astype(np.int32)).to(DEVICE).double()


def _two_to(e):
    """2^e in 64 bits, exactly, for whole e of any type."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _grid(bits, bias, top):
    """All values of a format of 3 mantissa bits, ascending."""
    c = torch.arange(2**bits, dtype=torch.float64, device=DEVICE)
    e, f = torch.floor(c / 8), c % 8
    v = torch.where(e == 0, f / 8 * 2.0 ** (1 - bias), (1 + f / 8) * _two_to(e - bias))
    return v[v <= top]


def _exact_blocks(v, grid, lowest, u):
    """The values kept of v [blocks, size], block by block; u as v or None."""
    a = v.abs().max(dim=1, keepdim=True).values
    top = grid[-1]
    e = torch.floor(torch.log2((a / top).clamp(min=2.0**-200))) - 1  # below E, whatever log2 rounds
    for _ in range(3):
        e = torch.where(_two_to(e) * top < a, e + 1, e)
    e = e.clamp(min=lowest)
    t = v.abs() / _two_to(e)
    lo = (torch.searchsorted(grid, t, right=True) - 1).clamp(max=len(grid) - 2)
    below, above = grid[lo], grid[lo + 1]
    f = (t - below) / (above - below)
    if u is None:
        up = (f > 0.5) | ((f == 0.5) & (lo % 2 == 1))
    else:
        up = u + torch.floor(f * 65536 + 0.5) >= 65536
    q = torch.where(up, above, below)
    if lowest == -117:
        q = torch.where((e == 120) & (q > 240), 240.0, q)
    return torch.sign(v) * q * _two_to(e)


def _exact_rows(x, seed):
    rows, d = x.shape
    wide = -(-d // 128) * 128
    v = torch.zeros(rows, wide, dtype=torch.float64, device=DEVICE)
    v[:, :d] = x.double()
    u = None
    if seed is not None:
        each = wide // 8
        u = _exact_halves(rows * each, np.tile(np.arange(each), rows), 0,
                          np.repeat(np.arange(rows), each), 0, seed).reshape(-1, 128)
    return _exact_blocks(v.reshape(-1, 128), _grid(7, 7, 448.0), -117, u).reshape(rows, -1)[:, :d]


def _exact_linear(s):
    n, k = s["n"], s["k"]
    if s["what"] == "step":
        gn, gk = -(-n // 128), -(-k // 128)
        w = torch.zeros(gn * 128, gk * 128, dtype=torch.float64, device=DEVICE)
        w[:n, :k] = s["w"].double()
        w = w.reshape(gn, 128, gk, 128).permute(0, 2, 1, 3).reshape(gn * gk, -1)
        w = _exact_blocks(w, _grid(7, 7, 448.0), -117, None).reshape(gn, gk, 128, 128)
        w = w.permute(0, 2, 1, 3).reshape(gn * 128, -1)[:n, :k].contiguous()
    else:
        step = _two_to(s["exps"].int() - 127)
        step = torch.kron(step, torch.ones(128, 128, dtype=torch.float64, device=DEVICE))
        w = (s["codes"].double() * step[:n])[:, :k].contiguous()
    out = {"y": torch.mm(_exact_rows(s["x"], None), w.t()) + s["b"].double()}
    if s["what"] == "step":
        out["dx"] = torch.mm(_exact_rows(s["dy"], s["seed"]), w)
    return out


def _exact_adamw(s):
    t, out = s["step"], {}
    p, g, m, v = (s[key].double() for key in ("p", "g", "m", "v"))
    if s["bits"] == 8:
        m = m * _two_to(s["m_exps"].int() - 127).repeat_interleave(128)
        v = _grid(8, 16, 61440.0)[s["v"].long()] * _two_to(
            s["v_exps"].int() - 127).repeat_interleave(128)
    if s["clip"]:
        out["norm"] = torch.linalg.vector_norm(g)
        g = g * min(1.0, MAX_NORM / (float(out["norm"]) + 1e-6))
    m = m + (1 - BETA1) * (g - m)
    v = v + (1 - BETA2) * (g.square() - v)
    mean, var = m / (1 - BETA1**t), v / (1 - BETA2**t)
    p = p - LR * (mean / (var.sqrt() + EPS) + DECAY * p)
    if s["bits"] == 8 or s["p"].dtype == torch.bfloat16:
        eighths = np.diff(s["starts"]) // 8
        tensor = np.repeat(np.arange(len(eighths)), eighths)
        i = np.arange(len(tensor)) - np.repeat(np.array(s["starts"][:-1]) // 8, eighths)

        def halves(draw_index):
            return _exact_halves(len(tensor), i, t, tensor, draw_index, s["seed"])
    if s["p"].dtype == torch.bfloat16:
        # the 16 bits below bf16's last place, as fp32 holds them
        ulp = _two_to(torch.frexp(p.abs().clamp(min=2.0**-126))[1] - 8)
        c = torch.floor(p.abs() / ulp * 65536)
        p = torch.sign(p) * torch.floor((c + halves(2).reshape(-1)) / 65536) * ulp
    if s["bits"] == 8:
        m = _exact_blocks(m.view(-1, 128), _grid(7, 7, 448.0), -117,
                          halves(0).reshape(-1, 128)).view(-1)
        v = _exact_blocks(v.view(-1, 128), _grid(8, 16, 61440.0), -108,
                          halves(1).reshape(-1, 128)).view(-1)
    return {"p": p, "m": m, "v": v, **out}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_linear(s) if s["op"] == "linear" else _exact_adamw(s)
