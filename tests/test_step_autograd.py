"""The step's operators as a training program has them: `linear` and `Mlp8`
with fp8 products under autograd, and the optimizer.  On the CPU with plain
stand-ins in the operators' place, on the GPU as they are."""
import copy
import io

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import step_plain as plain  # noqa: E402
import train_plain  # noqa: E402
import train_standins  # noqa: E402
from allreduce_compatible_gradient_amd import fp8, optim, train  # noqa: E402

E4M3 = torch.float8_e4m3fn


def host(t):
    return t.detach().double().cpu().numpy()


def _new(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype)


def install(monkeypatch) -> list:
    """fp8's and optim's device calls in plain 64-bit arithmetic."""
    calls = train_standins.install(monkeypatch)

    def weight(w, *, transposed=True, out=None, stream=None):
        calls.append("weight copy")
        train._dtype(w.dtype, "w")
        codes, exps, codes_t = (torch.from_numpy(a) for a in plain.weight(host(w)))
        return fp8.Fp8Weight(codes.view(E4M3), exps, w.shape[1],
                             codes_t.view(E4M3) if transposed else None)

    def linear(x, w, bias=None, *, transposed=False, seed=None, workspace=None, stream=None):
        calls.append("fp8 dx" if transposed else "fp8 product")
        train._dtype(x.dtype, "x")
        if transposed:
            step = plain.step_of(w.exps.numpy()).repeat(128, axis=0).repeat(128, axis=1)
            codes = plain.signed(w.codes_t.view(torch.uint8).numpy()[:, :w.n]).T
            v = codes * step[:w.n, :w.k]
        else:
            v = plain.weight_values(w.codes.view(torch.uint8).numpy(), w.exps.numpy(), w.k).T
        y = plain.rows_values(*plain.rows(host(x), seed), x.shape[1]) @ v
        return _new(y if bias is None else y + host(bias), x.dtype)

    def adamw(params, grads, exp_avgs, exp_avg_sqs, *, step, lr, betas=(0.9, 0.999), eps=1e-8,
              weight_decay=1e-2, scale=None, seed=None, stream=None):
        calls.append(("adamw", len(params), int(step), seed))
        c = 1.0 if scale is None else float(scale)
        for p, g, m, v in zip(params, grads, exp_avgs, exp_avg_sqs):
            assert p.is_contiguous() and g.is_contiguous() and p.shape == g.shape
            shape, flat = p.shape, isinstance(m, torch.Tensor)
            old = (m, v) if flat else (_moment(m), _moment(v))
            new = plain.adamw(host(p).ravel(), host(g).ravel(), host(old[0]), host(old[1]),
                              int(step), float(lr), *betas, eps, weight_decay, c)
            p.copy_(_new(new[0].reshape(shape), p.dtype))
            for t, x, second in ((m, new[1], False), (v, new[2], True)):
                if flat:
                    t.copy_(_new(x, t.dtype))
                else:
                    codes, exps = plain.moment(x, second, int(step), 0, seed)
                    t.codes.view(torch.uint8).copy_(torch.from_numpy(codes))
                    t.exps.copy_(torch.from_numpy(exps))

    def norm(grads, *, max_norm=None, stream=None):
        n = float(np.sqrt(sum(np.square(host(g)).sum() for g in grads)))
        scale = None if max_norm is None else torch.tensor(min(1.0, max_norm / (n + 1e-6)))
        return torch.tensor(n, dtype=torch.float32), scale

    monkeypatch.setattr(fp8, "gqs_fp8_weight", weight)
    monkeypatch.setattr(fp8, "gqs_fp8_linear", linear)
    monkeypatch.setattr(optim, "gqs_adamw", adamw)
    monkeypatch.setattr(optim, "gqs_grad_norm", norm)
    return calls


def _moment(m):
    if m.codes.is_cuda:
        return optim.gqs_moment8_restore(m, torch.float32)
    return _new(plain.moment_values(m.codes.view(torch.uint8).numpy(), m.exps.numpy(), m.n,
                                    m.second), torch.float32)


@pytest.fixture(params=["cpu", pytest.param("cuda", marks=pytest.mark.gpu)])
def device(request, monkeypatch):
    if request.param == "cpu":
        install(monkeypatch)
        monkeypatch.setattr(optim, "_on_device", lambda p: True)
    elif not torch.cuda.is_available():
        pytest.skip("no GPU")
    return request.param


def leaf(device, *shape, seed, dtype=torch.float32, scale=1.0):
    x = np.random.default_rng(seed).standard_normal(shape) * scale
    return torch.from_numpy(x).to(device).to(dtype).requires_grad_()


def within(got, want, bound, what=""):
    got = host(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (what, int(bad.sum()), float((np.abs(got - want) / bound).max()))


def copies(x, w, dy, seed):
    """The values the copies of x [m, k], w [n, k] and dy stand for."""
    vx = plain.rows_values(*plain.rows(x), x.shape[1])
    codes, exps, _ = plain.weight(w)
    vdy = plain.rows_values(*plain.rows(dy, seed), dy.shape[1])
    return vx, plain.weight_values(codes, exps, w.shape[1]), vdy


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("seed", [None, 77])
def test_linear(device, seed, dtype):
    """y, dx from the e4m3 copies, dw and db from the 8-bit copy of x."""
    kind = "f32" if dtype == torch.float32 else "bf16"
    x = leaf(device, 2, 9, 200, seed=1, dtype=dtype)
    w, b = leaf(device, 70, 200, seed=2, dtype=dtype), leaf(device, 70, seed=3, dtype=dtype)
    y = train.linear(x, w, b, seed=seed, fp8=True)
    assert y.shape == (2, 9, 70) and y.dtype == dtype
    dy = leaf(device, 2, 9, 70, seed=4, dtype=dtype, scale=0.01).detach()
    y.backward(dy)
    x2, dy2 = host(x).reshape(18, 200), host(dy).reshape(18, 70)
    vx, vw, vdy = copies(x2, host(w), dy2, None if seed is None else train._mix_seed(seed, 4))
    bound = plain.product_bound(vx, vw, kind, kind == "f32") + np.abs(host(b)) * (
        plain.U + plain.HALF[kind] * 1.01)
    within(y.reshape(18, 70), vx @ vw.T + host(b), bound, "y")
    within(x.grad.reshape(18, 200), vdy @ vw, plain.product_bound(vdy, vw.T, kind, kind == "f32"),
           "dx")
    kept = train_plain.restore(*train_plain.save(x2, seed), 200)
    want = train_plain.weight_grad(dy2, kept)
    for got, a, e in zip((w.grad, b.grad), want,
                         train_plain.weight_grad_bounds(dy2, kept, kind)):
        assert got.dtype == dtype
        within(got, a, e, "dw, db")


def test_linear_gradients_against_differences(device):
    """Of values the formats hold, y is exact, so differences are too: d y / d
    x = w wherever x's codes move with x."""
    x = torch.tensor([[1.0, 2.0, -4.0, 0.5]], device=device, requires_grad=True)
    w = torch.tensor([[1.0, -2.0, 0.5, 4.0], [8.0, 1.0, 1.0, -1.0]], device=device)
    y = train.linear(x, w, fp8=True)
    y.backward(torch.tensor([[1.0, 2.0]], device=device))
    for k in range(4):
        e = torch.zeros_like(x)
        e[0, k] = x.detach()[0, k]  # doubled: still a power of two
        moved = train.linear(x.detach() + e, w, fp8=True) - y.detach()
        slope = (moved * torch.tensor([[1.0, 2.0]], device=device)).sum() / e[0, k]
        assert float(slope) == float(x.grad[0, k])


def test_linear_parts(device):
    """No gradients, some of them, no bias, one row, no rows, strided weights,
    shared inputs and a gradient expanded from a scalar."""
    x, w = leaf(device, 5, 40, seed=1), leaf(device, 30, 40, seed=2)
    with torch.no_grad():
        y = train.linear(x, w, fp8=True)
    assert torch.equal(y, train.linear(x, w, fp8=True).detach())
    train.linear(x, w.detach(), fp8=True).sum().backward()
    assert w.grad is None
    once = x.grad.clone()
    train.linear(x.detach(), w, fp8=True).sum().backward()
    assert torch.equal(x.grad, once) and w.grad is not None
    x.grad = None
    (train.linear(x, w, fp8=True) + train.linear(x, w, fp8=True)).sum().backward()
    assert torch.equal(x.grad, 2 * once)
    t = w.detach().t().contiguous().t()
    assert torch.equal(train.linear(x, t, fp8=True), train.linear(x, w, fp8=True))
    assert train.linear(x[0], w, fp8=True).shape == (30,)
    empty = torch.zeros(0, 40, device=device, requires_grad=True)
    for fp8_ in (True, False):
        y = train.linear(empty, w, fp8=fp8_)
        assert y.shape == (0, 30)
        y.sum().backward()  # its gradient has strides of 0
        assert empty.grad.shape == (0, 40)


@pytest.mark.parametrize("x_dtype", [torch.float32, torch.bfloat16])
def test_linear_under_autocast(device, x_dtype):
    x = leaf(device, 12, 40, seed=1, dtype=x_dtype)
    w, b = leaf(device, 24, 40, seed=2), leaf(device, 24, seed=3)
    with torch.autocast(device, torch.bfloat16):
        y = train.linear(x, w, b, fp8=True)
    assert y.dtype == torch.bfloat16
    y.float().square().sum().backward()
    assert x.grad.dtype == x_dtype and w.grad.dtype == b.grad.dtype == torch.float32
    want = train.linear(x.detach().bfloat16(), w.detach().bfloat16(), b.detach().bfloat16(),
                        fp8=True)
    assert torch.equal(y.detach(), want)


@pytest.mark.parametrize("plain_up", [True, False])
def test_block(device, plain_up):
    """Mlp8 with fp8 products: as one operator or by its parts the same
    gradients, near those of the library's products."""
    torch.manual_seed(0)
    ordinary = train.Mlp8(48, 160, seed=5, device=device, dtype=torch.float32)
    block = train.Mlp8(48, 160, seed=5, device=device, dtype=torch.float32, fp8=True)
    block.load_state_dict(ordinary.state_dict())
    if not plain_up:
        block.down.register_forward_hook(lambda *a: None)
    x = leaf(device, 3, 11, 48, seed=1)
    y = block(x)
    y.square().mean().backward()
    got = [x.grad] + [p.grad for p in block.parameters()]
    x0 = x.detach().clone().requires_grad_()
    y0 = ordinary(x0)
    y0.square().mean().backward()
    # each of the products' operands is off by at most 1/16 of itself, at
    # random: a few percent of a sum in all
    assert float(((y - y0).norm() / (y0 - x0).norm()).detach()) < 0.1
    for a, b in zip(got, [x0.grad] + [p.grad for p in ordinary.parameters()]):
        assert a.shape == b.shape and float((a - b).norm() / b.norm()) < 0.15


def test_held_weights(device):
    block = train.Mlp8(40, 130, device=device, dtype=torch.float32, fp8=True)
    x = leaf(device, 4, 40, seed=1).detach()
    with torch.no_grad():
        y = block(x)
        block.hold_fp8()
        assert torch.equal(block(x), y)
        block.up.weight.zero_()
        assert torch.equal(block(x), y)   # as they were
        block.hold_fp8(False)
        assert not torch.equal(block(x), y)
        block.hold_fp8()
        with torch.autocast(device, torch.bfloat16):
            assert block(x).shape == x.shape
    assert block(x).requires_grad  # with gradients: of the weights as they are
    assert not any("held" in k for k in block.state_dict())
    with pytest.raises(ValueError):
        train.Mlp8(8, 16, device=device).hold_fp8()


def test_held_copies_are_dropped_with_their_weights(device):
    """By a state that is loaded and by a cast; a layer that is no plain
    Linear is not held."""
    make = lambda: train.Mlp8(40, 150, device=device, dtype=torch.float32, fp8=True)  # noqa: E731
    block, other = make(), make()
    x = leaf(device, 4, 40, seed=1).detach()
    with torch.no_grad():
        y = other(x)
        block.hold_fp8()
        assert not torch.equal(block(x), y)
        block.load_state_dict(other.state_dict())
        assert torch.equal(block(x), y)
        block.hold_fp8().double().float().up.weight.zero_()
        assert not torch.equal(block(x), y)
        block.load_state_dict(other.state_dict())
        block.up = torch.nn.Sequential(other.up)
        assert torch.allclose(block.hold_fp8()(x), y, atol=0.1)
        del block.__dict__["fp8"], block.__dict__["_held"]  # as an older pickle
        assert torch.isfinite(block(x)).all()


# ---------------------------------------------------------------------------
# the optimizer

def parameters(device, dtype=torch.float32):
    ps = [torch.nn.Parameter(leaf(device, *s, seed=k, dtype=dtype).detach())
          for k, s in enumerate([(7, 5), (300,), (1,), (2, 3, 4, 5)])]
    # laid out channels last, and transposed
    ps[3].data = ps[3].data.contiguous(memory_format=torch.channels_last)
    ps[0].data = ps[0].data.t().contiguous().t()
    return ps


def give(ps, seed, same_layout=True):
    for k, p in enumerate(ps):
        g = leaf(p.device.type, *p.shape, seed=100 * seed + k, dtype=p.dtype, scale=0.1).detach()
        p.grad = torch.empty_like(p).copy_(g) if same_layout else g


@pytest.mark.parametrize("clip", [None, 0.5])
def test_optimizer_against_torch(device, clip):
    """32-bit moments: torch's AdamW, and its clipping, in 64 bits."""
    ps = parameters(device)
    qs = [torch.nn.Parameter(p.detach().double()) for p in ps]
    opt = optim.AdamW(ps, lr=1e-2, betas=(0.8, 0.9), eps=1e-6, weight_decay=0.1, max_norm=clip)
    ref = torch.optim.AdamW(qs, lr=1e-2, betas=(0.8, 0.9), eps=1e-6, weight_decay=0.1)
    for step in range(1, 5):
        give(ps, step, same_layout=step % 2 == 0)
        for p, q in zip(ps, qs):
            q.grad = p.grad.double()
        if step == 3:  # one without a gradient keeps its count
            ps[1].grad = qs[1].grad = None
        if clip:
            n = torch.nn.utils.clip_grad_norm_(qs, clip)
        opt.step()
        ref.step()
        if clip:
            assert abs(float(opt.last_norm) - float(n)) < 1e-6 * float(n)
    assert opt.state[ps[1]]["step"] == 3 and opt.state[ps[0]]["step"] == 4
    for p, q in zip(ps, qs):
        # four steps of fp32 roundings, each below 2^-20 of a change of lr
        assert float((p.double() - q).abs().max()) < 4 * (1e-2 * 2.0**-19 + 2.0**-22 * 4)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_optimizer_in_8_bits(device, dtype):
    """The first step has exact moments: its update is that of 32 bits."""
    ps = parameters(device, dtype)
    qs = [p.detach().double().clone() for p in ps]
    opt = optim.AdamW(ps, lr=1e-2, bits=8, seed=3)
    give(ps, 1)
    opt.step()
    for p, q in zip(ps, qs):
        g = p.grad.double()
        want = q * (1 - 1e-4) - 1e-2 * g / (g.abs() + 1e-8)
        tol = 2.0**-7 if dtype == torch.bfloat16 else 2.0**-21
        assert float(((p.double() - want).abs() - tol * (want.abs() + 1e-2)).max()) <= 0
        m, v = opt.moments(p)
        assert m.codes.dtype == E4M3 and v.codes.dtype == torch.uint8 and m.n == p.numel()
        assert m.codes.numel() == -(-p.numel() // 128) * 128
    give(ps, 2)
    opt.step()
    assert all(torch.isfinite(p).all() for p in ps)


@pytest.mark.parametrize("bits", [32, 8])
def test_optimizer_goes_on_from_its_state(device, bits):
    ps = parameters(device, torch.bfloat16)
    opt = optim.AdamW(ps, lr=1e-2, bits=bits, seed=4)
    for step in range(1, 3):
        give(ps, step)
        opt.step()
    file = io.BytesIO()
    torch.save(opt.state_dict(), file)
    file.seek(0)
    other = [torch.nn.Parameter(p.detach().clone(memory_format=torch.preserve_format)) for p in ps]
    again = optim.AdamW(other, lr=5.0, bits=bits, seed=4)
    again.load_state_dict(torch.load(file, weights_only=True))
    twin = copy.deepcopy(opt.state_dict())
    for p, q in zip(ps, other):
        for key, value in opt.state[p].items():
            got = again.state[q][key]
            assert type(got) is type(value)
            if isinstance(value, torch.Tensor):
                assert got.dtype == value.dtype and got.data_ptr() != value.data_ptr()
    give(ps, 9)
    give(other, 9)
    opt.step()
    again.step()
    for p, q in zip(ps, other):
        assert torch.equal(p, q)
    assert twin["state"][0]["step"] == 2
    with pytest.raises(ValueError):
        optim.AdamW(parameters(device), bits=40 - bits).load_state_dict(opt.state_dict())


@pytest.mark.parametrize("bits", [32, 8])
def test_optimizer_copies_and_pickles(device, bits):
    ps = parameters(device)
    opt = optim.AdamW(ps, lr=1e-2, bits=bits, seed=4, max_norm=1.0)
    give(ps, 1)
    opt.step()
    file = io.BytesIO()
    torch.save(opt, file)
    file.seek(0)
    for twin in (copy.deepcopy(opt), torch.load(file, weights_only=False)):
        assert (twin.bits, twin.seed, twin.max_norm, twin.capturable) == (bits, 4, 1.0, False)
        qs = twin.param_groups[0]["params"]
        twin_of = [p.detach().clone() for p in ps]
        for p, q, r in zip(ps, qs, twin_of):
            assert torch.equal(p, q) and q is not p
            q.grad = p.grad.clone()
        twin.step()
        assert all(not torch.equal(q, r) for q, r in zip(qs, twin_of))


@pytest.mark.parametrize("first", [False, True])
def test_optimizer_counts_go_over(device, first):
    """Steps counted on the host go on on the device, and the other way."""
    ps = parameters(device)
    opt = optim.AdamW(ps, lr=1e-2, bits=8, seed=4, capturable=first)
    for step in (1, 2):
        give(ps, step)
        opt.step()
    qs = [torch.nn.Parameter(p.detach().clone(memory_format=torch.preserve_format)) for p in ps]
    other = optim.AdamW(qs, lr=1e-2, bits=8, seed=4, capturable=not first)
    other.load_state_dict(opt.state_dict())
    give(ps, 3)
    give(qs, 3)
    opt.step()
    other.step()
    for p, q in zip(ps, qs):
        assert torch.equal(p, q)
    assert ("step" in other.param_groups[0]) == (not first)
    assert all(("step" in other.state[q]) == first for q in qs)
    if not first:
        ps[0].grad = None
        opt.step()
        with pytest.raises(ValueError):
            other.load_state_dict(opt.state_dict())


def test_optimizer_groups(device):
    """Groups with settings of their own, types side by side, a closure, and
    parameters without gradients."""
    a, b = parameters(device)[:2]
    c = torch.nn.Parameter(leaf(device, 50, seed=9, dtype=torch.bfloat16).detach())
    still = torch.nn.Parameter(torch.ones(3, device=device))
    opt = optim.AdamW([{"params": [a, c]}, {"params": [b, still], "lr": 0.0, "weight_decay": 0.0}],
                      lr=1e-2, max_norm=1e9)
    give([a, b, c], 1)
    before = b.detach().clone()

    def closure():
        return torch.tensor(3.0)
    assert float(opt.step(closure)) == 3.0
    assert torch.equal(b, before) and (still == 1).all() and not opt.state[still]
    n = float(torch.cat([p.grad.double().flatten() for p in (a, b, c)]).norm())
    assert abs(float(opt.last_norm) - n) < 1e-6 * n
    assert optim.AdamW([still]).step() is None


def test_optimizer_refusals(device):
    p = torch.nn.Parameter(torch.ones(4, device=device))
    for kw in (dict(bits=4), dict(lr=-1.0), dict(lr=float("nan")), dict(betas=(0.9, 1.0)),
               dict(betas=(0.9,)), dict(eps=-1.0), dict(weight_decay=float("inf")),
               dict(max_norm=-1.0), dict(lr=torch.tensor(1e-3))):
        with pytest.raises(ValueError):
            optim.AdamW([p], **kw)
    wide = torch.nn.Parameter(torch.ones(4, 6, device=device)[:, ::2])
    wide.grad = torch.ones(4, 3, device=device)
    with pytest.raises(ValueError):
        optim.AdamW([wide]).step()
    p.grad = torch.sparse_coo_tensor([[0]], [1.0], (4,), device=device)
    with pytest.raises(RuntimeError):
        optim.AdamW([p]).step()


def test_optimizer_refuses_captures_that_would_go_wrong(device, monkeypatch):
    """A graph would zero what a first step makes at each replay, and keep the
    number of a step that the host counts."""
    p, q = (torch.nn.Parameter(torch.ones(4, device=device)) for _ in range(2))
    p.grad = torch.ones(4, device=device)
    ready, fixed = optim.AdamW([p, q], capturable=True), optim.AdamW([p])
    ready.step()
    fixed.step()
    before = p.detach().clone()
    with monkeypatch.context() as m:
        m.setattr(optim, "_capturing", lambda device: True)
        for opt in (fixed, optim.AdamW([p], capturable=True), optim.AdamW([p], bits=8)):
            with pytest.raises(RuntimeError):
                opt.step()
        ready.step()
        q.grad = torch.ones(4, device=device)
        with pytest.raises(RuntimeError):
            ready.step()
    assert (q == 1).all() and not torch.equal(p, before)
    assert int(ready.param_groups[0]["step"]) == 2


def test_optimizer_refuses_host_parameters():
    p = torch.nn.Parameter(torch.ones(4))
    p.grad = torch.ones(4)
    with pytest.raises(ValueError):
        optim.AdamW([p]).step()


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_a_captured_training_step(bits):
    """Forward, backward and update of an fp8 block in one graph: each replay
    is the eager step with the same numbers, the count and lr on the device."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dev, steps = "cuda", 4
    data = [torch.randn(64, 96, device=dev) for _ in range(steps + 1)]

    def program():
        torch.manual_seed(1)
        block = train.Mlp8(96, 300, random=False, device=dev, dtype=torch.float32, fp8=True)
        lr = torch.tensor([1e-2], device=dev)
        opt = optim.AdamW(block.parameters(), lr=lr, bits=bits, max_norm=1.0, capturable=True)
        return block, lr, opt

    def step(block, opt, x):
        opt.zero_grad(set_to_none=True)
        loss = (block(x) - 1).square().mean()
        loss.backward()
        opt.step()
        return loss.detach()

    block, lr, opt = program()
    eager = []
    for k, x in enumerate(data):
        lr.fill_(1e-2 / (k + 1))
        eager.append(float(step(block, opt, x)))
    want = [p.detach().clone() for p in block.parameters()]
    del block, opt

    block, lr, opt = program()
    x = data[0].clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        first = float(step(block, opt, x))  # makes the states, outside of the graph
        opt.zero_grad(set_to_none=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss = step(block, opt, x)
    got = [first]
    for k in range(1, steps + 1):
        x.copy_(data[k])
        lr.fill_(1e-2 / (k + 1))
        graph.replay()
        torch.cuda.synchronize()
        got.append(float(loss))
    assert got == eager
    assert int(opt.param_groups[0]["step"]) == steps + 1
    for p, q in zip(block.parameters(), want):
        assert torch.equal(p, q)


@pytest.mark.gpu
@pytest.mark.parametrize("more", [["--fp8"], ["--adamw", "32", "--clip", "1.0"],
                                  ["--fp8", "--adamw", "8"]])
def test_example_runs(more):
    """Ragged sizes; every loss is finite."""
    import importlib.util
    import os
    import torch.distributed as dist
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location(
        "train_mlp8", os.path.join(root, "examples", "train_mlp8.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    torch.cuda.set_device(0)
    store = dist.TCPStore("127.0.0.1", 0, 1, is_master=True)
    dist.init_process_group("nccl", store=store, rank=0, world_size=1)
    try:
        losses = example.run(example.arguments(
            ["--blocks", "2", "--d", "72", "--hidden", "200", "--tokens", "333", "--steps", "5"]
            + more))
    finally:
        dist.destroy_process_group()
    assert len(losses) == 5 and all(np.isfinite(losses))
