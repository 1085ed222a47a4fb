"""Layer norm where a block takes several rows in turn, the last turn not full:
every shape of its kernels, with rows loaded ahead or not, from x or its copy,
against 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import train_plain as plain  # noqa: E402
from allreduce_compatible_gradient_amd import train  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5


def host(t):
    return t.detach().double().cpu().numpy()


def draw(rows, d, seed, dtype, mean=0.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    t = (torch.randn(rows, d, device=DEV, generator=g) + mean).to(DT[dtype])
    return t, host(t)


def within(got, want, bound, what):
    got = host(got)
    assert got.shape == want.shape, what
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist())


# at least two turns of all blocks that the card holds, forward (without copies
# and with) and backward, the last one short; 7001 x 4096 with copies four turns
SHAPES = [(140_001, 24), (70_001, 40), (70_001, 64), (20_003, 250), (8_200, 512), (10_301, 770),
          (8_199, 1_500), (4_099, 2_048), (3_001, 4_000), (7_001, 4_096), (2_500, 6_100),
          (1_100, 8_192)]


@pytest.mark.parametrize("rows,d", SHAPES + [(1_100, 16_384), (2_100, 16_400)])
@pytest.mark.parametrize("dtype,wdtype,seeds", [("bf16", "f32", (5, 6)), ("f32", "f32", (None, 7)),
                                                ("bf16", "bf16", None)])
def test_forward(rows, d, dtype, wdtype, seeds):
    t, x = draw(rows, d, d, dtype, mean=0.5)
    w, wn = draw(1, d, d + 1, wdtype)
    b, bn = draw(1, d, d + 2, wdtype)
    kw = {}
    if seeds:
        kw = {"save_x": train.Act8.empty(rows, d, DEV), "seed_x": seeds[0],
              "save_y": train.Act8.empty(rows, d, DEV), "seed_y": seeds[1]}
    y, mean, rstd = train.gqt_layer_norm(t, w[0], b[0], EPS, **kw)
    within(y, plain.layer_norm(x, wn, bn, EPS), plain.layer_norm_bound(x, wn, bn, EPS, dtype), "y")
    em, er = plain.norm_stats(x, EPS)
    size = plain.gamma(d) * np.abs(x).mean(axis=1)
    within(mean, em[:, 0], size + plain.U, "mean")
    dm = size + plain.U * np.abs(em[:, 0])
    within(rstd, er[:, 0], er[:, 0] * (plain.gamma(d) + 8 * plain.U + (dm * er[:, 0])**2), "rstd")
    if seeds:  # the copies are those that one row a thread's turn writes
        for a, v, s in ((kw["save_x"], t, seeds[0]), (kw["save_y"], y, seeds[1])):
            ref = train.gqt_act8_save(v, seed=s)
            assert torch.equal(a.codes, ref.codes) and torch.equal(a.exps, ref.exps)


@pytest.mark.parametrize("rows,d", SHAPES + [(1_100, 8_200)])
@pytest.mark.parametrize("dtype,wdtype,kept", [("bf16", "f32", False), ("bf16", "bf16", True),
                                               ("f32", "f32", False), ("f32", "f32", True)])
def test_backward(rows, d, dtype, wdtype, kept):
    t, x = draw(rows, d, d + 10, dtype, mean=-0.3)
    dyt, dy = draw(rows, d, d + 11, dtype)
    w, wn = draw(1, d, d + 12, wdtype)
    _, mean, rstd = train.gqt_layer_norm(t, w[0], None, EPS)
    if kept:
        t = train.gqt_act8_save(t, seed=d)
        x = host(train.gqt_act8_restore(t, torch.float32))
    got = train.gqt_layer_norm_backward(dyt, t, mean, rstd, w[0])
    args = dy, x, host(mean)[:, None], host(rstd)[:, None], wn
    for g, e, bound, what in zip(got, plain.layer_norm_backward(*args),
                                 plain.layer_norm_backward_bounds(*args, dtype, wdtype),
                                 ("dx", "dw", "db")):
        within(g, e, bound, what)
