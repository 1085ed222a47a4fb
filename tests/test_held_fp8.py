"""What Mlp8.hold_fp8 holds, and when it lets go: a layer never comes from two
states.  On the CPU with plain stand-ins, on the GPU as it is."""
import copy
import io

import pytest

torch = pytest.importorskip("torch")

from allreduce_compatible_gradient_amd import optim, train  # noqa: E402
from test_step_autograd import device, install, leaf  # noqa: E402,F401


def blocks(device, n=2):
    """Blocks of other weights and biases, and an input."""
    made = [train.Mlp8(40, 150, seed=k, device=device, dtype=torch.float32, fp8=True)
            for k in range(n)]
    return *made, leaf(device, 4, 40, seed=1).detach()


def run(block, x):
    with torch.no_grad():
        return block(x)


@pytest.mark.parametrize("name", ["up", "down"])
def test_a_replaced_layer_is_taken_as_it_is(device, name):
    block, other, x = blocks(device)
    block.hold_fp8()
    setattr(block, name, getattr(other, name))
    got = run(block, x)
    assert torch.equal(got, run(block.hold_fp8(False), x))


def test_layers_of_another_width(device):
    block, x = blocks(device, 1)
    block.hold_fp8()
    block.up = torch.nn.Linear(40, 70, device=device)
    block.down = torch.nn.Linear(70, 40, device=device)
    assert torch.equal(run(block, x), run(block.hold_fp8(False), x))


@pytest.mark.parametrize("name", ["up", "down"])
def test_a_state_loaded_into_a_layer_is_seen(device, name):
    block, *others, x = blocks(device, 3)
    for other in others:  # held again, it sees the next as well
        block.hold_fp8()
        was = run(block, x)
        getattr(block, name).load_state_dict(getattr(other, name).state_dict())
        got = run(block, x)
        assert not torch.equal(got, was) and not block._holding
        assert torch.equal(got, run(block.hold_fp8(False), x))


@pytest.mark.parametrize("name", ["up", "down"])
def test_a_layer_that_is_cast_is_seen(device, name):
    block, x = blocks(device, 1)
    block.hold_fp8()
    getattr(block, name).half().float()
    assert torch.equal(run(block, x), run(block.hold_fp8(False), x))
    block.hold_fp8()
    getattr(block, name).weight.data = getattr(block, name).weight.data * 2
    assert torch.equal(run(block, x), run(block.hold_fp8(False), x))
    block.hold_fp8()
    layer = getattr(block, name)
    layer.weight = torch.nn.Parameter(layer.weight.detach() * 2)
    assert torch.equal(run(block, x), run(block.hold_fp8(False), x))


@pytest.mark.parametrize("kind", [optim.AdamW, torch.optim.SGD])
def test_an_update_is_seen(device, kind):
    block, x = blocks(device, 1)
    opt = kind(block.parameters(), lr=0.1)
    block.hold_fp8()
    was = run(block, x)
    block(x).sum().backward()
    opt.step()
    got = run(block, x)
    assert not torch.equal(got, was)
    assert torch.equal(got, run(block.hold_fp8(False), x))


def test_a_change_in_place_reaches_neither_weight_nor_bias(device):
    """What is held is the whole layer."""
    block, other, x = blocks(device)
    block.hold_fp8()
    was = run(block, x)
    with torch.no_grad():
        for name in ("up", "down"):
            getattr(block, name).weight.copy_(getattr(other, name).weight)
            getattr(block, name).bias.copy_(getattr(other, name).bias)
    assert torch.equal(run(block, x), was)
    assert not torch.equal(run(block.hold_fp8(), x), was)


def test_layers_without_a_bias_are_held(device):
    block, x = blocks(device, 1)
    block.up = torch.nn.Linear(40, 150, bias=False, device=device)
    was = run(block, x)
    assert torch.equal(run(block.hold_fp8(), x), was) and block._holding
    block.up.bias = torch.nn.Parameter(torch.ones(150, device=device))
    assert not torch.equal(run(block, x), was)


def test_a_copy_holds_nothing(device):
    block, x = blocks(device, 1)
    block.hold_fp8()
    was = run(block, x)
    file = io.BytesIO()
    torch.save(block, file)
    file.seek(0)
    for twin in (copy.deepcopy(block), torch.load(file, weights_only=False), copy.copy(block)):
        assert twin._held is None and torch.equal(run(twin, x), was)
        assert torch.equal(run(twin.hold_fp8(), x), was)
        twin.up.load_state_dict(twin.up.state_dict())
        assert torch.equal(run(twin, x), was)
    twin = copy.deepcopy(block)
    twin.up.load_state_dict(twin.up.state_dict())
    block.hold_fp8()
    twin.down.load_state_dict(twin.down.state_dict())
    assert block._holding  # a copy's layers are its own


@pytest.mark.gpu
def test_a_captured_pass_keeps_what_it_reads():
    """A graph of a held pass replays it, whatever has ended the holding."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    block, other, x = blocks("cuda")
    block.hold_fp8()
    want = run(block, x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = run(block, x)
    block(x).sum().backward()
    block.up.load_state_dict(other.up.state_dict())
    block.down.load_state_dict(other.down.state_dict())
    for _ in range(3):
        more = [torch.randn(150, 40, device="cuda") for _ in range(8)]
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        del more
    assert not torch.equal(run(block, x), want)


def test_a_product_without_gradients_makes_no_transposed_copy(monkeypatch):
    """Whether or not its inputs could have some."""
    from allreduce_compatible_gradient_amd import fp8
    install(monkeypatch)
    made, make = [], fp8.gqs_fp8_weight
    monkeypatch.setattr(fp8, "gqs_fp8_weight",
                        lambda w, *, transposed=True: made.append(transposed)
                        or make(w, transposed=transposed))
    x, w = leaf("cpu", 4, 40, seed=1), leaf("cpu", 30, 40, seed=2)
    with torch.no_grad():
        train.linear(x, w, fp8=True)
    train.linear(x.detach(), w, fp8=True).sum().backward()
    assert made == [False, False]
    train.linear(x, w, fp8=True).sum().backward()
    assert made == [False, False, True] and x.grad is not None
