"""The weight gradient where its kernel takes its several ways: squares of four
tiles with partial sums, tokens split over them, tokens in full steps and left
over, rows far apart, values next to fp32's subnormals.  Whole numbers keep
every sum exact, so that those results have to be equal."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from allreduce_compatible_gradient_amd import train  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def copy_of_ones(m, k):
    """The copy of a matrix of ones."""
    groups = -(-k // 32)
    codes = torch.zeros((m, 32 * groups), dtype=torch.int8, device=DEV)
    codes[:, :k] = 1
    return train.Act8(codes, torch.full((m, groups), 127, dtype=torch.uint8, device=DEV), k)


def test_fp32_next_to_the_subnormals():
    """Three bf16 parts hold an fp32 value of 2^-110 or more whole; below,
    what lies under bf16's last place, 2^-133, is left out, towards 0."""
    rng = np.random.default_rng(1)
    for m in (1, 200):  # the loop over left-over tokens, and a full step
        for e in (-149, -140, -133, -127, -126, -118, -111, -110, -109, -100):
            v = np.zeros((m, 64), np.float32)
            v[m // 2] = (rng.choice([-1, 1], 64) * (1 + rng.random(64)) * 2.0**e)
            dw, db = train.gqt_weight_grad(torch.from_numpy(v).to(DEV), copy_of_ones(m, 40))
            dw = dw.double().cpu().numpy()
            want = np.tile(v[m // 2].astype(np.float64)[:, None], (1, 40))
            if e >= -110:
                assert np.array_equal(dw, want), e
            else:
                assert (np.abs(dw - want) < 2.0**-133).all() and (np.abs(dw) <= np.abs(want)).all()
            assert np.array_equal(db.cpu().numpy(), v[m // 2])
