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
