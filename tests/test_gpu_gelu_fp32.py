"""fp32 GELU in its tail, where the exponential's argument decides: no more
than the roundings that fp32 cannot avoid there."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import train_plain as plain  # noqa: E402
from allreduce_compatible_gradient_amd import train  # noqa: E402

pytestmark = pytest.mark.gpu
U = plain.U


def worst(t, want, bound):
    return float((np.abs(t.double().cpu().numpy() - want) / bound).max())


@pytest.mark.parametrize("form", ["none", "tanh"])
def test_gelu_of_fp32_in_its_tail(form):
    """erf: the square in e^(-h^2/2) is rounded once, which is h^2/2 half steps
    of the result; the exponential is off by one step (2 U), the fitted tail by
    1.5e-7.  tanh: 2 u is four roundings (8 u U), and the gate's sum, reciprocal
    (one step) and product add four.  Products round once each."""
    low, high = (-12.5, -3.0) if form == "none" else (-6.0, -1.0)
    h = np.random.default_rng(1).uniform(low, high, (64, 1024)).astype(np.float32)
    t = torch.from_numpy(h).to("cuda")
    h = h.astype(np.float64)
    y = train.gqt_gelu(t, form)
    s = train.gqt_gelu_backward(torch.ones_like(t), t, form)
    if form == "none":
        e = (h * h / 2 + 2) * U
        tail = np.abs(plain.gelu(h, form) / h)
        phi = np.abs(h) * np.exp(-0.5 * h * h) / math.sqrt(2 * math.pi)
        bound_y = np.abs(h) * tail * (e + 1.5e-7 + 2 * U)
        bound_s = phi * (e + 2 * U) + tail * (e + 1.5e-7 + U)
    else:
        c = math.sqrt(2 / math.pi)
        u = np.abs(c * (h + 0.044715 * h**3))
        slope = c * (1 + 3 * 0.044715 * h * h)
        small = np.abs(plain.gelu(h, form) / h)
        e = (8 * u + 6) * U
        bound_y = np.abs(h) * small * (e + U)
        # u' has two products, a sum and three constants; its factor 2 h, the
        # complement (one minus the gate, off by e's share and three roundings)
        # and their product one each
        term = np.abs(2 * h * slope) * small * (1 - small)
        bound_s = term * (e + small * e + 12 * U) + small * e
    want_s = plain.gelu_slope(h, form)
    assert worst(y, plain.gelu(h, form), bound_y * 1.001) <= 1
    assert worst(s, want_s, (bound_s + U * np.abs(want_s)) * 1.001) <= 1
