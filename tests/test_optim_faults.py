"""What an optimizer's step may not do: change a weight behind autograd's
back, stop half-way, take the state of another layout or optimizer.  The
binding runs up to its launch on the CPU, or with plain stand-ins; on the GPU
as it is."""
import types

import pytest

torch = pytest.importorskip("torch")

from allreduce_compatible_gradient_amd import optim  # noqa: E402
from test_step_autograd import device, give, install, leaf, parameters  # noqa: E402,F401


class Launches:
    """The library's entry points as far as the binding sees them: what they
    were given, and that they took it."""

    def __init__(self):
        self.args = []

    def gqs_adamw(self, tensors, count, p_dtype, g_dtype, args, *rest):
        self.args.append({name: getattr(args, name) for name, _ in args._fields_})
        return 0


@pytest.fixture
def launches(monkeypatch):
    """gqs_adamw on host tensors up to its launch."""
    here = Launches()
    monkeypatch.setattr(optim, "lib", lambda: here)
    monkeypatch.setattr(optim, "_device_of", lambda *a: types.SimpleNamespace(index=-1))
    monkeypatch.setattr(optim, "_elsewhere", lambda *a: False)
    monkeypatch.setattr(optim, "_current", lambda device: 0)
    monkeypatch.setattr(optim, "_on_device", lambda p: True)
    return here


# ---------------------------------------------------------------------------
# parameters are changed in place, and autograd is told

def test_a_step_counts_as_a_change(launches):
    p, q = torch.nn.Parameter(torch.ones(3)), torch.nn.Parameter(torch.ones(2, 3).t())
    before = p._version, q._version
    optim.gqs_adamw([p], [torch.ones(3)], [torch.zeros(3)], [torch.zeros(3)], step=1, lr=1e-3)
    assert p._version > before[0] and q._version == before[1]
    p.grad, q.grad = torch.ones(3), torch.ones(3, 2)
    optim.AdamW([p, q]).step()
    assert p._version > before[0] + 1 and q._version > before[1]
    assert len(launches.args) == 2


def _backward_after_a_step(device):
    layer = torch.nn.Linear(4, 4, device=device)
    x = torch.ones(2, 4, device=device, requires_grad=True)
    for p in layer.parameters():
        p.grad = torch.ones_like(p)
    y = layer(x)
    optim.AdamW(layer.parameters()).step()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_a_graph_from_before_a_step_is_refused(launches):
    _backward_after_a_step("cpu")


@pytest.mark.gpu
def test_a_graph_from_before_a_step_is_refused_on_the_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    _backward_after_a_step("cuda")
    p = torch.ones(9, device="cuda")
    optim.gqs_adamw([p], [p.clone()], [torch.zeros_like(p)], [torch.zeros_like(p)], step=1,
                    lr=1e-3, stream=torch.cuda.Stream())
    assert p._version > 0


# ---------------------------------------------------------------------------
# bf16 parameters to nearest, whatever the moments are

def test_rounding_of_parameters_is_its_own_choice(launches):
    p, g = torch.ones(3, dtype=torch.bfloat16), torch.ones(3)
    eights = [optim.Moment8.zeros(3, "cpu", k) for k in (False, True)]
    wide = [torch.zeros(3) for _ in range(2)]
    for moments, kw, want in ((eights, dict(seed=1), 1), (eights, dict(seed=1, random=False), 0),
                              (eights, dict(seed=1, random=True), 1), (wide, dict(), 0),
                              (wide, dict(seed=1), 1), (wide, dict(seed=1, random=False), 0)):
        optim.gqs_adamw([p], [g], [moments[0]], [moments[1]], step=1, lr=1e-3, **kw)
        assert launches.args[-1]["random"] == want, kw
    with pytest.raises(ValueError):
        optim.gqs_adamw([p], [g], [wide[0]], [wide[1]], step=1, lr=1e-3, random=True)
    for bits in (8, 32):
        for random in (False, True):
            q = torch.nn.Parameter(p.clone())
            q.grad = torch.ones_like(q)
            optim.AdamW([q], bits=bits, random=random).step()
            assert launches.args[-1]["random"] == random, (bits, random)
            assert launches.args[-1]["bits"] == bits


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 32])
def test_parameters_to_nearest_on_the_gpu(bits):
    """The first step has exact moments, and its change is that of 64 bits: p
    lies within half a last place of it and fp32's few."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    p = torch.nn.Parameter(torch.randn(5000, device="cuda").bfloat16())
    p.grad = torch.randn(5000, device="cuda").bfloat16()
    old, g = p.detach().double(), p.grad.double()
    optim.AdamW([p], lr=1e-2, bits=bits, random=False, seed=3).step()
    want = old * (1 - 1e-4) - 1e-2 * g / (g.abs() + 1e-8)
    half = torch.exp2(torch.floor(torch.log2(want.abs())) - 8)
    # constants, moments, root, quotient and sums: below 2^-18 of the change
    # and 2^-22 of p
    slack = 2.0**-18 * 1e-2 + 2.0**-22 * old.abs()
    assert ((p.double() - want).abs() <= half + slack).all()


# ---------------------------------------------------------------------------
# moments lie in the order of the parameter that they were made for

def relaid(p):
    """p's values in other memory orders."""
    orders = [p.detach().contiguous(), p.detach().transpose(0, -1).contiguous().transpose(0, -1)]
    if p.dim() == 4:
        orders.append(p.detach().contiguous(memory_format=torch.channels_last))
    return orders


@pytest.mark.parametrize("bits", [32, 8])
def test_a_state_goes_to_a_parameter_of_another_order(device, bits):  # noqa: F811
    ps = parameters(device)
    opt = optim.AdamW(ps, lr=1e-2, bits=bits, seed=4)
    for step in (1, 2):
        give(ps, step)
        opt.step()
    saved = opt.state_dict()
    twins = []
    for k in range(3):
        qs = [torch.nn.Parameter(relaid(p)[min(k, p.dim() // 2)].clone(
            memory_format=torch.preserve_format)) for p in ps]
        again = optim.AdamW(qs, lr=1e-2, bits=bits, seed=4)
        again.load_state_dict(saved)
        for step in (3, 4):
            give(qs, step, same_layout=step == 3)
            again.step()
        twins.append((again, qs))
    for step in (3, 4):
        give(ps, step)
        opt.step()
    for again, qs in twins:
        for p, q in zip(ps, qs):
            assert torch.equal(p, q), (p.stride(), q.stride())
            for a, b in zip(opt.moments(p), again.moments(q)):
                same = (torch.equal(a, b) if bits == 32 else
                        torch.equal(a.codes.view(torch.uint8), b.codes.view(torch.uint8)))
                assert same


@pytest.mark.parametrize("bits", [32, 8])
def test_a_parameter_that_is_laid_out_anew(device, bits):  # noqa: F811
    ps, qs = parameters(device), parameters(device)
    one, other = (optim.AdamW(x, lr=1e-2, bits=bits, seed=4) for x in (ps, qs))
    for step in range(1, 5):
        give(ps, step)
        give(qs, step)
        one.step()
        other.step()
        for q in qs:
            q.data = relaid(q)[step % len(relaid(q))].clone(memory_format=torch.preserve_format)
    for p, q in zip(ps, qs):
        assert torch.equal(p, q)


@pytest.mark.parametrize("bits", [32, 8])
def test_a_state_of_other_sizes_is_refused(device, bits):  # noqa: F811
    ps = parameters(device)
    opt = optim.AdamW(ps, bits=bits)
    give(ps, 1)
    opt.step()
    for shape in ((7, 6), (5, 7), (35, 40), (35,)):
        qs = parameters(device)
        qs[0] = torch.nn.Parameter(leaf(device, *shape, seed=1).detach())
        again = optim.AdamW(qs, bits=bits)
        with pytest.raises(ValueError):
            again.load_state_dict(opt.state_dict())
        assert not again.state
    # a state without shapes, as older ones: by the numbers of elements
    old = opt.state_dict()
    for state in old["state"].values():
        del state["shape"], state["order"]
    with pytest.raises(ValueError):
        again = optim.AdamW([torch.nn.Parameter(leaf(device, 300, seed=1).detach())]
                            + parameters(device)[1:], bits=bits)
        again.load_state_dict(old)
    same = optim.AdamW(parameters(device), bits=bits)
    same.load_state_dict(old)
    give(same.param_groups[0]["params"], 2)
    same.step()


# ---------------------------------------------------------------------------
# a step is taken as a whole or not at all

def test_a_step_that_is_refused_changes_nothing(device):  # noqa: F811
    """Whatever comes last: another type, another device, a setting."""
    def param(dtype=torch.float32, on=device):
        p = torch.nn.Parameter(torch.ones(5, device=on, dtype=dtype))
        p.grad = torch.ones_like(p)
        return p

    def sparse():
        p = param()
        p.grad = torch.sparse_coo_tensor([[0]], [1.0], (5,), device=device)
        return p
    rate = torch.tensor(1e-3, device=device, dtype=torch.float64)
    for bad, kw, setting in ((param(torch.float16), {}, {}), (param(torch.float64), {}, {}),
                             (param(on="meta"), dict(capturable=True), {}), (sparse(), {}, {}),
                             (param(), {}, dict(lr=-1.0)), (param(), {}, dict(lr=rate)),
                             (param(), dict(capturable=True), dict(lr=rate)),
                             (param(), {}, dict(betas=(0.9, 1.0))),
                             (param(), {}, dict(weight_decay=float("nan")))):
        for apart in (False, True):
            if setting and not apart:
                continue
            p = param()
            groups = [{"params": [p]}, {"params": [bad]}] if apart else [p, bad]
            if apart and bad.device.type == "meta" and device == "cpu":
                continue  # a group each: no fault
            opt = optim.AdamW(groups, **kw)
            opt.param_groups[-1].update(setting)
            with pytest.raises((TypeError, ValueError, RuntimeError)):
                opt.step()
            assert (p == 1).all() and not opt.state and "step" not in opt.param_groups[0]


# ---------------------------------------------------------------------------
# steps counted on the device: each parameter's own

def _run_with_gaps(device, capturable, bits, present):
    ps = parameters(device)
    opt = optim.AdamW([{"params": ps[:3]}, {"params": ps[3:]}], lr=1e-2, bits=bits, seed=4,
                      capturable=capturable)
    for step, these in enumerate(present, 1):
        give(ps, step)
        for k, p in enumerate(ps):
            if k not in these:
                p.grad = None
        opt.step()
    return ps, opt


def count_of(opt, p):
    group = next(g for g in opt.param_groups if any(q is p for q in g["params"]))
    return int(opt.state[p].get("step", group.get("step")))


GAPS = [[(0, 3), (0, 1, 3), (0, 1, 2, 3)],            # first gradients that come late
        [(0, 1, 2, 3), (0, 1), (0, 1), (0, 1, 2, 3)],  # and that stay away
        [(0,), (1,), (0,), (1, 2), (0, 1, 2, 3)]]


@pytest.mark.parametrize("present", GAPS)
def test_counts_on_the_device_are_those_on_the_host(device, present):  # noqa: F811
    ps, opt = _run_with_gaps(device, False, 32, present)
    qs, other = _run_with_gaps(device, True, 32, present)
    for k, (p, q) in enumerate(zip(ps, qs)):
        assert count_of(opt, p) == count_of(other, q) == sum(k in these for these in present)
        # powers on the device and on the host may differ in a factor's last bit
        assert ((p - q).abs() <= 2.0**-21 * (q.abs() + 1e-2)).all()
    for kind in (False, True):  # a state goes over, and goes on
        rs = [torch.nn.Parameter(q.detach().clone(memory_format=torch.preserve_format))
              for q in qs]
        again = optim.AdamW([{"params": rs[:3]}, {"params": rs[3:]}], lr=1e-2, seed=4,
                            capturable=kind)
        again.load_state_dict(other.state_dict())
        give(rs, 9)
        again.step()
        assert [count_of(again, r) for r in rs] == [count_of(other, q) + 1 for q in qs]


def test_counts_do_not_part_in_a_capture(device, monkeypatch):  # noqa: F811
    ps, opt = _run_with_gaps(device, True, 32, GAPS[1])
    before = [p.detach().clone() for p in ps]
    ps[0].grad = None
    with monkeypatch.context() as m:
        m.setattr(optim, "_capturing", lambda device: True)
        with pytest.raises(RuntimeError):
            opt.step()
    assert all(torch.equal(p, q) for p, q in zip(ps, before))


@pytest.mark.gpu
def test_captured_steps_count_for_each():
    """A graph goes on with counts that have parted."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ps, opt = _run_with_gaps("cuda", True, 32, GAPS[0])
    qs, other = _run_with_gaps("cuda", True, 32, GAPS[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step()
    for _ in range(3):
        graph.replay()
        other.step()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(ps, qs))
    assert [count_of(opt, p) for p in ps] == [6, 5, 4, 6]


# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["AdamW", "Adam", "SGD", "Adagrad"])
@pytest.mark.parametrize("capturable", [False, True])
def test_another_optimizers_state_is_refused(device, kind, capturable):  # noqa: F811
    """Where it is loaded, not in the next step; shapes of one dimension, too."""
    for which in ([1], [0], [0, 1, 2, 3]):
        ps = [parameters(device)[k] for k in which]
        give(ps, 1)
        of = getattr(torch.optim, kind)(ps, lr=1e-2, **({"momentum": 0.9} if kind == "SGD" else {}))
        of.step()
        opt = optim.AdamW(ps, capturable=capturable)
        with pytest.raises(ValueError):
            opt.load_state_dict(of.state_dict())
        assert not opt.state
        opt.step()
