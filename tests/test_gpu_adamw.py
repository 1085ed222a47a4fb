"""AdamW, its moments in 8 bits and the gradients' norm on the GPU against
their plain 64-bit forms (tests/step_plain.py)."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import step_plain as plain  # noqa: E402
from allreduce_compatible_gradient_amd import _step, optim  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SEED = 0x0123456789ABCDEF
HYPER = dict(lr=3e-3, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    _step.lib()


def host(t):
    return t.detach().double().cpu().numpy()


def formula(p, g, m, v, t, scale=1.0, of=plain.adamw):
    return of(p, g, m, v, t, HYPER["lr"], *HYPER["betas"], HYPER["eps"], HYPER["weight_decay"],
              scale)


def draw(n, seed, pd="f32", gd="f32", fresh=False):
    """Device p, g, m, v of n elements: gradients over many sizes, some zero."""
    rng = np.random.default_rng(seed)
    g = rng.standard_normal(n) * np.exp2(rng.integers(-20, 3, n).astype(float))
    g[rng.random(n) < 0.1] = 0
    m = np.zeros(n) if fresh else rng.standard_normal(n) * 1e-2
    v = np.zeros(n) if fresh else rng.random(n) * 1e-4
    p = rng.standard_normal(n)

    def to(x, dtype=torch.float32):
        return torch.from_numpy(x).to(DEV).to(dtype)
    return to(p, DT[pd]), to(g, DT[gd]), to(m), to(v)


def off(t, by):
    """The same values at an address off by some elements."""
    big = torch.empty(t.numel() + by, dtype=t.dtype, device=t.device)
    big[by:] = t
    return big[by:]


def moments8(m, v, step=7, tensor=0):
    """Moment8 pairs of host values, made by the plain form."""
    out = []
    for x, second in ((m, False), (v, True)):
        codes, exps = plain.moment(x, second, step, tensor, 99)
        codes = torch.from_numpy(codes).to(DEV)
        out.append(optim.Moment8(codes if second else codes.view(torch.float8_e4m3fn),
                                 torch.from_numpy(exps).to(DEV), len(x)))
    return out


def near(got, want, bound, what=""):
    got = host(got)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (what, int(bad.sum()), float((np.abs(got - want) / bound).max()),
                           np.argwhere(bad)[:4].tolist())


SIZES = [[1], [7, 1, 8, 9], [0, 5, 0, 128, 0], [8191, 8192, 8193, 127, 129], [40000, 3]]


@pytest.mark.parametrize("clip", [False, True])
@pytest.mark.parametrize("pd,gd", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"),
                                   ("bf16", "f32")])
@pytest.mark.parametrize("step", [1, 2, 1000])
def test_moments_in_32_bits(step, pd, gd, clip):
    for s, sizes in enumerate(SIZES):
        data = [draw(n, 10 * s + i, pd, gd, step == 1) for i, n in enumerate(sizes)]
        data = [tuple(off(t, i % 3) for t in d) for i, d in enumerate(data)]
        before = [[host(t) for t in d] for d in data]
        scale = torch.tensor([0.37], device=DEV) if clip else None
        optim.gqs_adamw(*map(list, zip(*data)), step=step, scale=scale, **HYPER)
        for d, b in zip(data, before):
            c = 1.0 if scale is None else float(scale)
            want = formula(*b, step, c)
            ep, em, ev = formula(*b, step, c, of=plain.adamw_bounds)
            if pd == "bf16":
                ep = ep * 1.01 + np.abs(want[0]) * 2.0**-8 * 1.01
            near(d[0], want[0], ep, "p")
            near(d[2], want[1], em, "m")
            near(d[3], want[2], ev, "v")
            assert np.array_equal(host(d[1]), b[1])


@pytest.mark.parametrize("pd,gd", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("step", [1, 50])
def test_moments_in_8_bits(step, pd, gd):
    """The update takes the moments before their rounding; the codes are those
    of the plain form, or, where fp32's last bits decide, their neighbours."""
    for s, sizes in enumerate(SIZES):
        data = [draw(n, 10 * s + i, pd, gd, step == 1) for i, n in enumerate(sizes)]
        ms, vs, before = [], [], []
        for i, (p, g, m, v) in enumerate(data):
            m8, v8 = moments8(host(m), host(v))
            ms.append(m8)
            vs.append(v8)
            before.append((host(p), host(g), host(optim.gqs_moment8_restore(m8, torch.float32)),
                           host(optim.gqs_moment8_restore(v8, torch.float32))))
        ps, gs = [d[0] for d in data], [d[1] for d in data]
        optim.gqs_adamw(ps, gs, ms, vs, step=step, seed=SEED, **HYPER)
        for i, b in enumerate(before):
            n = len(b[0])
            if n == 0:
                continue
            p, m, v = formula(*b, step)
            ep, em, ev = formula(*b, step, of=plain.adamw_bounds)
            if pd == "bf16":
                ep = ep * 1.01 + np.abs(p) * 2.0**-7 * 1.01  # at random: a whole step
            near(ps[i], p, ep, "p")
            for got, x, second in ((ms[i], m, False), (vs[i], v, True)):
                codes, exps = plain.moment(x, second, step, i, SEED)
                assert np.array_equal(got.exps.cpu().numpy(), exps)
                c = got.codes.view(torch.uint8).cpu().numpy()
                same = (c == codes) | ((c | codes) == 128)
                assert same.mean() > 1 - 1e-4 - 1.0 / len(c), (second, same.mean())
                assert (np.abs(c.astype(int) - codes) <= 1)[~same].all()
                want = plain.moment_values(codes, exps, n, second)
                r = host(optim.gqs_moment8_restore(got, torch.bfloat16))
                assert np.array_equal(r[same[:n]], want[same[:n]])
                assert not c[n:].any()


def test_a_list_is_its_parts():
    """More tensors than a launch takes, empty ones among them: what each
    alone would give, random numbers by the number in the list."""
    sizes = [(37 * i) % 300 if i % 11 else 0 for i in range(150)]
    data = [draw(n, i, "bf16") for i, n in enumerate(sizes)]
    m8 = [moments8(host(d[2]), host(d[3]), tensor=i) for i, d in enumerate(data)]
    want = []
    for i, (d, (m, v)) in enumerate(zip(data, m8)):
        e = torch.empty(0, dtype=torch.bfloat16, device=DEV)
        none = optim.Moment8.zeros(0, DEV, False), optim.Moment8.zeros(0, DEV, True)
        p, mm, vv = d[0].clone(), *(optim.Moment8(x.codes.clone(), x.exps.clone(), x.n)
                                    for x in (m, v))
        optim.gqs_adamw([e] * i + [p], [torch.empty(0, device=DEV)] * i + [d[1]],
                        [none[0]] * i + [mm], [none[1]] * i + [vv], step=3, seed=5, **HYPER)
        want.append((p, mm, vv))
    optim.gqs_adamw([d[0] for d in data], [d[1] for d in data], [x[0] for x in m8],
                    [x[1] for x in m8], step=3, seed=5, **HYPER)
    for d, (m, v), (p, mm, vv) in zip(data, m8, want):
        assert torch.equal(d[0], p) and torch.equal(m.exps, mm.exps)
        assert torch.equal(m.codes.view(torch.uint8), mm.codes.view(torch.uint8))
        assert torch.equal(v.codes, vv.codes) and torch.equal(v.exps, vv.exps)


def test_random_bf16_parameters():
    """Steps of a hundredth of a last place count in expectation; to nearest
    they are lost."""
    n = 1 << 16
    hyper = dict(lr=2.0**-7 / 100, betas=(0.0, 0.0), eps=0.0, weight_decay=0.0)
    g = torch.ones(n, device=DEV)
    p = torch.full((n,), 1.5, dtype=torch.bfloat16, device=DEV)
    still = p.clone()
    for step in range(1, 21):
        for t, seed in ((p, SEED), (still, None)):
            m, v = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
            optim.gqs_adamw([t], [g], [m], [v], step=step, seed=seed, **hyper)
    assert (still == 1.5).all()
    moved = 1.5 - host(p).mean()
    # 20 steps of 2^-7 / 100 in places of 2^-7: a binomial's 5 deviations
    assert abs(moved - 0.2 * 2.0**-7) < 5 * 2.0**-7 * math.sqrt(0.2 / n)


def test_second_moments_decay():
    """With no gradients a second moment in 8 bits shrinks on average as in 32
    bits: rounded to nearest it would stay."""
    n, steps = 1 << 14, 50
    v8 = moments8(np.zeros(n), np.linspace(0.5, 1, n))[1]
    m8 = optim.Moment8.zeros(n, DEV, False)
    p, g = torch.ones(n, device=DEV), torch.zeros(n, device=DEV)
    start = host(optim.gqs_moment8_restore(v8)).mean()
    for step in range(1, steps + 1):
        optim.gqs_adamw([p], [g], [m8], [v8], step=step, lr=0.0, betas=(0.9, 0.999), seed=3)
    got = host(optim.gqs_moment8_restore(v8)).mean() / start
    # each step rounds to a neighbour with variance at most step^2 / 4, a step
    # of at most an eighth of the value
    assert abs(got - 0.999**steps) < 5 * 0.125 / 2 * math.sqrt(steps / n)


def test_non_finite_gradients():
    """An inf or NaN stays within its element, in 8 bits within its block."""
    n = 600
    for bits in (32, 8):
        for bad in (float("nan"), float("inf")):
            p, g, m, v = draw(n, 3)
            g[200] = bad
            if bits == 8:
                m, v = moments8(host(m), host(v))
            optim.gqs_adamw([p], [g], [m], [v], step=2, seed=1, **HYPER)
            assert torch.isnan(p[200]) and int(torch.isnan(p).sum()) == 1
            if bits == 8:
                for x in (m, v):
                    r = torch.isnan(optim.gqs_moment8_restore(x, torch.float32))
                    assert r[128:256].all() and int(r.sum()) == 128
                g[200] = 0.0
                optim.gqs_adamw([p], [g], [m], [v], step=3, seed=1, **HYPER)
                assert int(torch.isnan(p).sum()) == 128
            else:
                assert not torch.isfinite(m[200]) and int((~torch.isfinite(v)).sum()) == 1


def test_zero_everything():
    """No gradient, no moment, eps 0: 0 / 0 is the formula's NaN; with eps the
    parameter only decays."""
    p = torch.ones(100, device=DEV)
    z = [torch.zeros(100, device=DEV) for _ in range(3)]
    optim.gqs_adamw([p], [z[0]], [z[1]], [z[2]], step=1, lr=0.5, weight_decay=0.5)
    assert (p == 0.75).all()
    optim.gqs_adamw([p], [z[0]], [z[1]], [z[2]], step=1, lr=0.5, eps=0.0)
    assert torch.isnan(p).all()


def test_step_and_rate_on_the_device():
    """lr and step as tensors give what numbers give, and a captured graph
    reads them at every replay."""
    p, g, m, v = draw(5000, 1, "bf16")
    m8, v8 = moments8(host(m), host(v))
    lr = torch.tensor([HYPER["lr"]], device=DEV)
    step = torch.zeros(1, dtype=torch.int64, device=DEV)
    rest = {k: x for k, x in HYPER.items() if k != "lr"}
    copies = [(p.clone(), m.clone(), v.clone()) for _ in range(2)]
    eights = [[optim.Moment8(x.codes.clone(), x.exps.clone(), x.n) for x in (m8, v8)]
              for _ in range(2)]
    q8 = [p.clone() for _ in range(2)]

    def run(i, lr, step):
        pp, mm, vv = copies[i]
        optim.gqs_adamw([pp], [g], [mm], [vv], step=step, lr=lr, seed=SEED, **rest)
        optim.gqs_adamw([q8[i]], [g], [eights[i][0]], [eights[i][1]], step=step, lr=lr, seed=SEED,
                        **rest)
    step.fill_(1)
    run(0, lr, step)  # warm, and the first step
    run(1, HYPER["lr"], 1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.add_(1)
        run(0, lr, step)
    for t in range(2, 6):
        rate = float(np.float32(HYPER["lr"] / t))
        lr.fill_(rate)
        graph.replay()
        run(1, rate, t)
        torch.cuda.synchronize()
        # pow on the device and on the host may differ in the factors' last bit
        for a, b in zip(copies[0][1:], copies[1][1:]):
            assert torch.equal(a, b)
        near(copies[0][0], host(copies[1][0]), np.abs(host(copies[1][0])) * 2.0**-7 * 1.01)
        for a, b in zip(eights[0], eights[1]):
            assert torch.equal(a.codes.view(torch.uint8), b.codes.view(torch.uint8))


def test_streams_hold_what_they_use():
    stream = torch.cuda.Stream()
    p, g, m, v = draw(100000, 9)
    q, mm, vv = p.clone(), m.clone(), v.clone()
    optim.gqs_adamw([q], [g], [mm], [vv], step=4, **HYPER)
    want = optim.gqs_grad_norm([g], max_norm=0.5)
    torch.cuda.synchronize()
    got = optim.gqs_grad_norm([g], max_norm=0.5, stream=stream)
    optim.gqs_adamw([p], [g], [m], [v], step=4, stream=stream, **HYPER)
    stream.synchronize()
    assert torch.equal(p, q) and torch.equal(m, mm) and torch.equal(v, vv)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ---------------------------------------------------------------------------
# the norm

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sizes", [[1], [3, 0, 8, 9], [16384, 16385, 16383], [5] * 200, [1000003]])
def test_norm(sizes, dtype):
    gs = [off(draw(n, i)[1].to(DT[dtype]), i % 3) for i, n in enumerate(sizes)]
    norm, scale = optim.gqs_grad_norm(gs, max_norm=0.25)
    want = math.sqrt(sum(float(np.square(host(g)).sum()) for g in gs))
    assert abs(float(norm) - want) <= want * 2.0**-24 * 1.01
    c = min(1.0, 0.25 / (want + 1e-6))
    assert abs(float(scale) - c) <= c * 2.0**-24 * 1.01
    again, none = optim.gqs_grad_norm(gs)
    assert torch.equal(again, norm) and none is None


def test_norm_of_extremes():
    big = torch.full((1000,), 3e38, device=DEV)
    norm, scale = optim.gqs_grad_norm([big], max_norm=1.0)
    assert torch.isinf(norm) and 0 < float(scale) < 1e-38 or float(scale) == 0.0
    small = torch.full((1000,), 1e-40, device=DEV)  # its square has no float
    norm, scale = optim.gqs_grad_norm([small], max_norm=1.0)
    assert abs(float(norm) - math.sqrt(1000) * float(small[0].double())) < 1e-45 * 2
    assert float(scale) == 1.0
    for bad, n, s in ((float("inf"), math.inf, 0.0), (float("nan"), math.nan, math.nan)):
        small[77] = bad
        norm, scale = optim.gqs_grad_norm([small], max_norm=1.0)
        assert np.array_equal([float(norm), float(scale)], [n, s], equal_nan=True)
    assert float(optim.gqs_grad_norm([torch.zeros(9, device=DEV)], max_norm=2.0)[1]) == 1.0


def test_refusals():
    p, g, m, v = draw(300, 1)
    m8, v8 = moments8(host(m), host(v))
    ok = dict(step=1, lr=1e-3)
    for call, kind in (
            (lambda: optim.gqs_adamw([p], [g[:200]], [m], [v], **ok), ValueError),
            (lambda: optim.gqs_adamw([p], [g], [m[:200]], [v], **ok), ValueError),
            (lambda: optim.gqs_adamw([p], [g], [m], [], **ok), ValueError),
            (lambda: optim.gqs_adamw([p], [g], [m], [v8], **ok), TypeError),
            (lambda: optim.gqs_adamw([p], [g], [m8], [v8], **ok), ValueError),  # no seed
            (lambda: optim.gqs_adamw([p], [g], [v8], [m8], seed=1, **ok), TypeError),
            (lambda: optim.gqs_adamw([p.half()], [g], [m], [v], **ok), TypeError),
            (lambda: optim.gqs_adamw([p], [g], [m.double()], [v], **ok), TypeError),
            (lambda: optim.gqs_adamw([p, p.bfloat16()], [g, g], [m, m], [v, v], **ok), TypeError),
            (lambda: optim.gqs_adamw([p.view(2, 150).t()], [g], [m], [v], **ok), ValueError),
            (lambda: optim.gqs_adamw([p, p], [g, g], [m, m.clone()], [v, v.clone()], **ok), Exception),
            (lambda: optim.gqs_adamw([p], [g], [m], [m], **ok), Exception),
            (lambda: optim.gqs_adamw([p], [g], [m], [v], step=0, lr=1e-3), Exception),
            (lambda: optim.gqs_adamw([p], [g], [m], [v], scale=g, **ok), ValueError),
            (lambda: optim.gqs_adamw([p], [g], [m], [v], step=torch.ones(1, device=DEV), lr=1e-3),
             ValueError),
            (lambda: optim.gqs_adamw([p], [g.cpu()], [m], [v], **ok), ValueError),
            (lambda: optim.gqs_grad_norm([g, g.bfloat16()]), TypeError),
            (lambda: optim.gqs_grad_norm([g], max_norm=-1.0), Exception),
            (lambda: optim.gqs_moment8_restore(m), ValueError)):
        was = p.clone()
        with pytest.raises(kind):
            call()
        assert torch.equal(p, was)


def test_a_tensor_past_32_bits():
    """2^32 bytes of bf16 and more elements than 31 bits count: its end, and
    the random numbers there."""
    n = (1 << 31) + 1000
    p = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    g = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    m, v = optim.Moment8.zeros(n, DEV, False), optim.Moment8.zeros(n, DEV, True)
    g[-1], g[(1 << 31) + 3], g[5] = 1.0, 2.0, 3.0
    optim.gqs_adamw([p], [g], [m], [v], step=1, lr=0.5, weight_decay=0.0, seed=2)
    at = torch.tensor([5, (1 << 31) + 3, n - 1], device=DEV)
    assert (p[at].float() + 0.5).abs().max() < 2.0**-8
    assert int(torch.count_nonzero(p)) == 3
    first = optim.Moment8(m.codes[-1024:], m.exps[-8:], 1024 - (-n % 128))
    got = host(optim.gqs_moment8_restore(first))
    want = np.zeros(len(got))
    want[-1], want[(1 << 31) + 3 - n] = 0.1, 0.2
    assert (np.abs(got - want) <= want / 8).all()
    norm, _ = optim.gqs_grad_norm([g])
    assert abs(float(norm) - math.sqrt(14)) < 1e-6
