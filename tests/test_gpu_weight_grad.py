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


def whole_numbers(m, n, k, dtype, seed=0):
    """dy of whole numbers and a copy of halves: (dy, copy, and both in 64
    bits).  Every sum stays below 2^24 halves, so that fp32 holds it."""
    assert m * 3 * 18 * 2 < 2**24
    g = torch.Generator(device=DEV).manual_seed(seed)
    dy = torch.randint(-3, 4, (m, n), device=DEV, generator=g).to(DT[dtype])
    groups = -(-k // 32)
    codes = torch.randint(-9, 10, (m, 32 * groups), device=DEV, generator=g).to(torch.int8)
    exps = torch.randint(126, 129, (m, groups), device=DEV, generator=g).to(torch.uint8)
    x = codes.double() * torch.exp2(exps.double() - 127).repeat_interleave(32, dim=1)
    return dy, train.Act8(codes, exps, k), dy.double(), x[:, :k].contiguous()


def same(got, dy, x):
    dw, db = got
    assert torch.equal(dw.double(), dy.t().contiguous() @ x)
    assert torch.equal(db.double(), dy.sum(dim=0))


# workspace: the number of partial sums names the way that is taken
@pytest.mark.parametrize("m,n,k,dtype,partials", [
    # squares over all tokens, 15 full steps and 20 left over, with a partial
    # of db from each of 32 columns of tiles, of which the last is past k
    (500, 3950, 3900, "bf16", 32 * 3950), (500, 3950, 3900, "f32", 32 * 3950),
    # squares over a third of the tokens
    (5990, 4220, 1150, "f32", 3 * 4220 * (1150 + 10)),
    (16384, 4220, 1150, "bf16", 3 * 4220 * (1150 + 10)),
    # tiles that a block's waves share: all tokens, and four steps of them
    (1000, 1900, 1930, "bf16", 0), (1000, 1900, 1930, "f32", 0),
    (20_000, 300, 200, "bf16", 40 * 300 * (200 + 2)),
    (20_000, 300, 200, "f32", 40 * 300 * (200 + 2))])
def test_every_way_of_the_tiles(m, n, k, dtype, partials):
    assert train.gqt_weight_grad_workspace_bytes(m, n, k, DT[dtype]) == 4 * partials
    t, a, dy, x = whole_numbers(m, n, k, dtype)
    same(train.gqt_weight_grad(t, a), dy, x)
    dw, none = train.gqt_weight_grad(t, a, bias=False)
    assert none is None and torch.equal(dw.double(), dy.t().contiguous() @ x)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [(1000, 300, 200), (20_000, 300, 200), (500, 3950, 3900)])
def test_one_row_of_dy_for_all_tokens(m, n, k, dtype):
    """A stride of 0 in full steps."""
    t, a, dy, x = whole_numbers(m, n, k, dtype)
    same(train.gqt_weight_grad(t[:1].expand(m, n), a), dy[:1].expand(m, n), x)


@pytest.mark.parametrize("n", [5, 24, 300])
def test_rows_of_dy_far_apart(n):
    """2^24 elements, past a lane's offset in a step: one row at a time.  And
    just below, in full steps."""
    m, k = 140, 72
    for stride in (2**24, 2**24 - 8):
        t, a, dy, x = whole_numbers(m, n, k, "bf16")
        big = torch.empty(m * stride, dtype=torch.bfloat16, device=DEV)
        far = torch.as_strided(big, (m, n), (stride, 1))
        far.copy_(t)
        same(train.gqt_weight_grad(far, a), dy, x)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [(1000, 1900, 1930), (20_000, 300, 200), (500, 3950, 3900)])
def test_non_finite_values_in_full_steps(m, n, k, dtype):
    """An inf or NaN of dy stays in its row of dw and its db, a NaN group in
    its columns, in whichever step they are met."""
    t, a, dy, x = whole_numbers(m, n, k, dtype)
    tokens = [0, 31, 32, 129, 255, 300, m - 1]
    rows = [3, 130, 131, n - 9, n - 8, n - 2, n - 1]
    for i, (token, row) in enumerate(zip(tokens, rows)):
        t[token, row] = float("nan") if i % 3 == 2 else float("inf") if i % 2 else -float("inf")
    groups = [1, a.exps.shape[1] - 1]
    a.exps[33, groups[0]] = a.exps[m - 2, groups[1]] = 255
    dw, db = train.gqt_weight_grad(t, a)
    clean_row = torch.ones(n, dtype=torch.bool, device=DEV)
    clean_row[rows] = False
    clean = torch.ones(k, dtype=torch.bool, device=DEV)
    for g in groups:
        clean[32 * g:32 * g + 32] = False
    want = dy.t().contiguous() @ x
    assert torch.equal(dw.double()[clean_row][:, clean], want[clean_row][:, clean])
    assert dw[:, ~clean].isnan().all()
    assert torch.equal(db.double()[clean_row], dy.sum(dim=0)[clean_row])
    for i, (token, row) in enumerate(zip(tokens, rows)):
        v = t[token, row].double()
        # an inf times x, NaN where x is 0; what the others add does not matter
        assert torch.allclose(dw[row][clean].double(), (v * x[token])[clean], equal_nan=True)
        assert torch.allclose(db[row].double(), v, equal_nan=True)
