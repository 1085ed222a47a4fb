"""gqs_adamw refuses arrays that overlap, those of the 8-bit moments' exponents
among them, before it touches the device."""
import pytest

from allreduce_compatible_gradient_amd import _step
from test_step_cpu import A, NUL, adam, words

E = A << 24  # of exponents


def call(tensors, bits=8):
    L = _step.lib()
    return L.gqs_adamw(words(tensors), len(tensors), 0, 0, adam(bits=bits), A, 16, NUL)


def tensor(k, n=1000, em=None, ev=None):
    """The k-th of a list: its arrays lie apart from the others'."""
    at = (A << 4) + (k << 40)
    return (at, at + (A << 4), at + (A << 8), at + (A << 12), E + 64 * k if em is None else em,
            E + (A << 1) + 64 * k if ev is None else ev, n)


@pytest.mark.parametrize("tensors", [
    [tensor(0, em=E, ev=E)],                                     # one for both moments
    [tensor(0, em=E, ev=E + 7)],                                 # the last of 8 bytes
    [tensor(0), tensor(1, em=E + 7)],                            # another tensor's
    [tensor(0), tensor(1, ev=E + (A << 1) + 1)],
    [tensor(0, em=(A << 4) + (A << 8) + 1023)],                  # its own codes
    [tensor(0, ev=(A << 4) + 3999)],                             # its parameter
    [tensor(k) for k in range(100)] + [tensor(200, ev=E + 64 * 99 + 7)],  # a long list
])
def test_exponents_that_overlap_are_refused(tensors):
    assert call(tensors) == 2
    assert b"overlap" in _step.lib().gqs_last_error()


def test_exponents_side_by_side_are_not():
    """Refused for another reason, in a later check: the arrays do not overlap."""
    L = _step.lib()
    for tensors in ([tensor(0, em=E, ev=E + 8)], [tensor(0), tensor(1, em=E + 8)],
                    [tensor(k) for k in range(100)]):
        bad = adam(bits=8, scale=A + 2)
        assert L.gqs_adamw(words(tensors), len(tensors), 0, 0, bad, A, 16, NUL) == 6
    # 32-bit moments have none
    bad = adam(bits=32, scale=A + 2)
    assert L.gqs_adamw(words([tensor(0, em=E, ev=E)]), 1, 0, 0, bad, A, 16, NUL) == 6
