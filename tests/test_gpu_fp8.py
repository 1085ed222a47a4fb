"""Products in 8-bit floating point on the GPU against their plain 64-bit
forms (tests/step_plain.py): the copies bit for bit, the products within the
bounds of their sums; shapes where the kernels change, strides, non-finite
values, empty inputs, streams, graphs, large offsets."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import step_plain as plain  # noqa: E402
from allreduce_compatible_gradient_amd import _step, fp8  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SEED = 0x1234567890ABCDEF


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    _step.lib()


def host(t):
    return t.detach().double().cpu().numpy()


def draw(rows, d, seed, dtype="f32", scale=1.0):
    """A device matrix of values `dtype` holds, and the same values in 64
    bits: normal, with columns and blocks of other sizes and exact zeros."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, d)) * scale
    x *= np.exp2(rng.integers(-6, 7, d)) * np.exp2(rng.integers(-3, 4, (rows, 1)))
    x[rng.random((rows, d)) < 0.05] = 0.0
    t = torch.from_numpy(x).to(DEV).to(DT[dtype])
    return t, host(t)


def strided(t, how):
    rows, d = t.shape
    if how == "apart":
        big = torch.full((rows, d + 13), float("nan"), dtype=t.dtype, device=t.device)
        big[:, 5:5 + d] = t
        return big[:, 5:5 + d]
    if how == "off":
        flat = torch.empty(rows * d + 3, dtype=t.dtype, device=t.device)
        flat[3:] = t.reshape(-1)
        return flat[3:].view(rows, d)
    return t


def codes_of(t):
    return t.view(torch.uint8).cpu().numpy()


def within(got, want, bound, what=""):
    got = host(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (what, int(bad.sum()), float((np.abs(got - want) / bound).max()),
                           np.argwhere(bad)[:4].tolist())


# ---------------------------------------------------------------------------
# the copies

@pytest.mark.parametrize("how", ["plain", "apart", "off"])
@pytest.mark.parametrize("seed", [None, SEED])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,d", [(1, 1), (3, 7), (2, 127), (17, 128), (16, 129), (5, 515),
                                    (33, 641)])
def test_row_copies(rows, d, dtype, seed, how):
    t, x = draw(rows, d, rows * 1000 + d, dtype)
    codes, exps = plain.rows(x, seed)
    a = fp8.gqs_fp8_rows(strided(t, how), seed=seed)
    assert a.exps.shape == (-(-d // 128), -(-rows // 16) * 16)
    assert np.array_equal(a.exps[:, :rows].cpu().numpy(), exps)
    # the sign of what rounds to zero is free
    got = codes_of(a.codes)
    assert np.array_equal(np.where(got == 128, 0, got), np.where(codes == 128, 0, codes))
    for out in ("f32", "bf16"):
        assert np.array_equal(host(fp8.gqs_fp8_restore(a, DT[out])),
                              plain.rows_values(codes, exps, d))


@pytest.mark.parametrize("how", ["plain", "apart", "off"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,k", [(1, 1), (7, 3), (128, 128), (129, 127), (127, 129), (260, 390)])
def test_weight_copies(n, k, dtype, how):
    t, x = draw(n, k, n * 1000 + k, dtype)
    codes, exps, codes_t = plain.weight(x)
    w = fp8.gqs_fp8_weight(strided(t, how))
    assert np.array_equal(w.exps.cpu().numpy(), exps)
    for got, want in ((codes_of(w.codes), codes), (codes_of(w.codes_t), codes_t)):
        assert np.array_equal(np.where(got == 128, 0, got), np.where(want == 128, 0, want))
    assert np.array_equal(host(fp8.gqs_fp8_restore(w, torch.float32)),
                          plain.weight_values(codes, exps, k))
    alone = fp8.gqs_fp8_weight(t, transposed=False)
    assert alone.codes_t is None and np.array_equal(codes_of(alone.codes), codes_of(w.codes))


@pytest.mark.parametrize("seed", [None, SEED])
def test_extreme_values(seed):
    """The largest floats, subnormals, both zeros, blocks of one size of value
    and values half-way between codes."""
    f = np.finfo(np.float32)
    x = np.zeros((6, 256), dtype=np.float32)
    x[0, :128] = f.max
    x[0, 128:] = -f.max * np.linspace(0, 1, 128)
    x[1, :128] = f.smallest_subnormal * np.arange(128)
    x[1, 128:] = f.tiny * np.linspace(-3, 3, 128)
    x[2, 0], x[2, 1] = 448.0, -0.0
    x[2, 2:100] = (plain.E4M3[1:99] + plain.E4M3[:98]) / 2
    x[3] = 2.0**-117 * np.linspace(-500, 500, 256)
    x[4] = np.float32(1e-30)
    x[5, ::2] = 2.0**127
    codes, exps = plain.rows(x.astype(np.float64), seed)
    a = fp8.gqs_fp8_rows(torch.from_numpy(x).to(DEV), seed=seed)
    assert np.array_equal(a.exps[:, :6].cpu().numpy(), exps)
    got = host(fp8.gqs_fp8_restore(a, torch.float32))
    want = plain.rows_values(codes, exps, 256)
    assert np.isfinite(got).all()
    # scaled into subnormals, fractions below a code's last place keep 20 bits
    # or round: no draw here lies that near its border
    assert np.array_equal(got, want)


def test_non_finite_blocks():
    x = torch.ones(3, 300, device=DEV)
    x[0, 130], x[2, 299] = float("nan"), float("-inf")
    for seed in (None, SEED):
        a = fp8.gqs_fp8_rows(x, seed=seed)
        bad = torch.isnan(fp8.gqs_fp8_restore(a, torch.float32))
        want = torch.zeros(3, 300, dtype=torch.bool, device=DEV)
        want[0, 128:256], want[2, 256:] = True, True
        assert torch.equal(bad, want)
    w = fp8.gqs_fp8_weight(x)
    bad = torch.isnan(fp8.gqs_fp8_restore(w, torch.float32))
    assert bad[:, 128:].all() and not bad[:, :128].any()


def test_random_copies_are_unbiased():
    """The mean over 8192 rows of one row's values lies within 5 deviations."""
    v = torch.linspace(-1, 1, 256, device=DEV).repeat(8192, 1)
    a = fp8.gqs_fp8_rows(v, seed=11)
    r = host(fp8.gqs_fp8_restore(a, torch.float32))
    x = host(v[0])
    up, lo = r.max(axis=0), r.min(axis=0)
    assert ((lo <= x) & (x <= up)).all()
    step = up - lo
    p = np.where(step > 0, (x - lo) / np.where(step > 0, step, 1), 0)
    dev = step * np.sqrt(p * (1 - p) / 8192)
    assert (np.abs(r.mean(axis=0) - x) <= 5 * dev + step * 2.0**-16 + 1e-12).all()


# ---------------------------------------------------------------------------
# products

SHAPES = [(1, 1, 1), (1, 300, 130), (2, 16, 128), (7, 33, 1000), (16, 128, 2100), (17, 40, 129),
          (31, 257, 384), (33, 130, 260), (64, 64, 640), (65, 129, 100), (100, 520, 1537),
          (128, 256, 256), (129, 300, 515), (257, 140, 700), (300, 1030, 390), (513, 513, 513)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_products(m, n, k, dtype):
    """Forward and transposed, from a copy and from x itself."""
    tx, x = draw(m, k, m + n + k, dtype)
    tw, w = draw(n, k, m * n + k, dtype, 0.1)
    tb = torch.randn(n, device=DEV).to(DT[dtype])
    tdy, dy = draw(m, n, m + 3 * n, dtype, 0.01)
    w8 = fp8.gqs_fp8_weight(tw)
    x8 = fp8.gqs_fp8_rows(tx)
    vw = host(fp8.gqs_fp8_restore(w8, torch.float32))
    vx = host(fp8.gqs_fp8_restore(x8, torch.float32))
    want = vx @ vw.T + host(tb)
    bound = plain.product_bound(vx, vw, dtype, dtype == "f32") + np.abs(host(tb)) * (
        plain.U + plain.HALF[dtype] * 1.01)
    y = fp8.gqs_fp8_linear(tx, w8, tb)
    assert y.dtype == DT[dtype]
    within(y, want, bound, "linear")
    assert torch.equal(y, fp8.gqs_fp8_linear(tx, w8, tb))
    within(fp8.gqs_fp8_product(x8, w8, tb, dtype=DT[dtype]), want, bound, "product")
    within(fp8.gqs_fp8_product(x8, w8, dtype=DT[dtype]), want - host(tb), bound, "no bias")
    dy8 = fp8.gqs_fp8_rows(tdy, seed=SEED)
    vdy = host(fp8.gqs_fp8_restore(dy8, torch.float32))
    bound = plain.product_bound(vdy, vw.T, dtype, dtype == "f32")
    within(fp8.gqs_fp8_linear(tdy, w8, transposed=True, seed=SEED), vdy @ vw, bound, "dx")
    within(fp8.gqs_fp8_product(dy8, w8, transposed=True, dtype=DT[dtype]), vdy @ vw, bound, "dx")


@pytest.mark.parametrize("how", ["apart", "off", "one row"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m", [3, 40, 300])
def test_strides(m, dtype, how):
    tx, _ = draw(m, 333, m, dtype)
    tw, _ = draw(77, 333, 5, dtype)
    if how == "one row":
        tx = tx[:1].expand(m, -1)
        given = tx
    else:
        given = strided(tx, how)
    w8 = fp8.gqs_fp8_weight(strided(tw, how if how != "one row" else "plain"))
    plainly = fp8.gqs_fp8_weight(tw)
    got = fp8.gqs_fp8_linear(given, w8)
    assert torch.equal(got, fp8.gqs_fp8_linear(tx.contiguous(), plainly))
    assert got.is_contiguous()


def test_whole_numbers_are_exact():
    """Small whole numbers, sums below 2^8: any lost product would show, in
    both types and every way of the kernels."""
    g = torch.Generator(device=DEV).manual_seed(2)
    for m, n, k in ((1, 70, 900), (16, 200, 700), (48, 200, 700), (100, 300, 1000),
                    (300, 260, 1000), (600, 600, 600), (2000, 1100, 200)):
        x = torch.randint(-1, 2, (m, k), device=DEV, generator=g).float()
        w = torch.randint(-1, 2, (n, k), device=DEV, generator=g).float()
        want = (x.double().cpu() @ w.double().cpu().t())
        assert want.abs().max() <= 256
        for t in DT.values():
            w8 = fp8.gqs_fp8_weight(w.to(t))
            assert torch.equal(fp8.gqs_fp8_linear(x.to(t), w8).double().cpu(), want), (m, n, k, t)
            back = fp8.gqs_fp8_linear(want.sign().to(DEV).to(t), w8, transposed=True)
            expect = want.sign() @ w.double().cpu()
            ok = expect.abs() <= 256
            assert torch.equal(back.double().cpu()[ok], expect[ok]), (m, n, k, t)


def test_non_finite_values_reach_their_rows_only():
    for m in (4, 40, 300):
        for t in DT.values():
            x = torch.ones(m, 300, device=DEV, dtype=t)
            w = torch.ones(140, 300, device=DEV, dtype=t)
            clean = fp8.gqs_fp8_weight(w)
            x[1, 200] = float("inf")
            y = fp8.gqs_fp8_linear(x, clean)
            assert torch.isnan(y[1]).all() and (y[0] == 300).all() and (y[2:] == 300).all()
            w[130, 5] = float("nan")
            x[1, 200] = 1
            y = fp8.gqs_fp8_linear(x, fp8.gqs_fp8_weight(w))
            assert torch.isnan(y[:, 128:]).all() and (y[:, :128] == 300).all()


def test_a_product_past_the_largest_float():
    """Blocks at both ends of the exponents: 2^127 times 2^-126 is 2, with
    every scale of the matrix cores between."""
    for t in DT.values():
        for m in (2, 40, 300):
            x = torch.full((m, 256), 2.0**127, device=DEV, dtype=t)
            w = torch.full((130, 256), 2.0**-117, device=DEV, dtype=t)
            y = fp8.gqs_fp8_linear(x, fp8.gqs_fp8_weight(w))
            assert (y == 256 * 2.0**10).all()
            y = fp8.gqs_fp8_linear(x, fp8.gqs_fp8_weight(x[:2]))
            assert torch.isinf(y).all()


def test_empty_batches():
    w8 = fp8.gqs_fp8_weight(torch.ones(5, 9, device=DEV))
    x = torch.zeros(0, 9, device=DEV)
    assert fp8.gqs_fp8_linear(x, w8).shape == (0, 5)
    a = fp8.gqs_fp8_rows(x)
    assert a.shape == (0, 9) and fp8.gqs_fp8_restore(a).shape == (0, 9)
    assert fp8.gqs_fp8_product(a, w8).shape == (0, 5)
    assert fp8.gqs_fp8_linear(torch.zeros(0, 5, device=DEV), w8, transposed=True).shape == (0, 9)


def test_rows_behind_are_left_alone():
    """What lies behind a copy, a result and a workspace stays as it was."""
    m, n, k = 37, 45, 200
    x, w = torch.randn(m, k, device=DEV), torch.randn(n, k, device=DEV)
    L = _step.lib()
    w8 = fp8.gqs_fp8_weight(w)
    need = L.gqs_fp8_linear_workspace_bytes(m, n, k, 0)
    ws = torch.full((need + 64,), 77, dtype=torch.uint8, device=DEV)
    y = torch.full((m * n + 16,), 5.0, device=DEV)
    _step.check(L.gqs_fp8_linear(x.data_ptr(), 0, m, k, k, 0, 0, w8.codes.data_ptr(),
                                 w8.exps.data_ptr(), n, 0, None, 0, y.data_ptr(), ws.data_ptr(),
                                 need, torch.cuda.current_stream().cuda_stream))
    assert (ws[need:] == 77).all() and (y[m * n:] == 5.0).all()
    assert torch.equal(y[:m * n].view(m, n), fp8.gqs_fp8_linear(x, w8))


def test_refusals():
    w8 = fp8.gqs_fp8_weight(torch.ones(5, 9, device=DEV), transposed=False)
    x = torch.ones(3, 9, device=DEV)
    a = fp8.gqs_fp8_rows(x)
    for call, kind in ((lambda: fp8.gqs_fp8_linear(x[:, :8], w8), ValueError),
                       (lambda: fp8.gqs_fp8_linear(x.half(), w8), TypeError),
                       (lambda: fp8.gqs_fp8_linear(x.t(), w8), ValueError),
                       (lambda: fp8.gqs_fp8_linear(x, x), TypeError),
                       (lambda: fp8.gqs_fp8_linear(x, w8, torch.ones(4, device=DEV)), ValueError),
                       (lambda: fp8.gqs_fp8_linear(x, w8, torch.ones(5)), ValueError),
                       (lambda: fp8.gqs_fp8_linear(x[:, :5], w8, transposed=True), ValueError),
                       (lambda: fp8.gqs_fp8_linear(
                           torch.ones(30, 9, device=DEV), w8,
                           workspace=torch.empty(16, dtype=torch.uint8, device=DEV)), ValueError),
                       (lambda: fp8.gqs_fp8_product(w8, w8), ValueError),
                       (lambda: fp8.gqs_fp8_product(a, w8, dtype=torch.float16), TypeError),
                       (lambda: fp8.gqs_fp8_rows(x, out=fp8.Fp8.empty(4, 9, DEV)), ValueError),
                       (lambda: fp8.gqs_fp8_weight(x[:0]), ValueError),
                       (lambda: fp8.gqs_fp8_weight(x, out=w8), ValueError)):
        with pytest.raises(kind):
            call()


@pytest.mark.parametrize("m", [5, 300])
def test_other_streams(m):
    """On a given stream, with its workspace: ordered behind what that stream
    does, and the inputs are held until then."""
    stream = torch.cuda.Stream()
    w8 = fp8.gqs_fp8_weight(torch.randn(200, 300, device=DEV))
    x = torch.randn(m, 300, device=DEV)
    want = fp8.gqs_fp8_linear(x, w8)
    torch.cuda.synchronize()
    got = fp8.gqs_fp8_linear(x, w8, stream=stream)
    a = fp8.gqs_fp8_rows(x, stream=stream)
    again = fp8.gqs_fp8_product(a, w8, dtype=torch.float32, stream=stream.cuda_stream)
    stream.synchronize()
    assert torch.equal(got, want) and torch.equal(again, want)


@pytest.mark.parametrize("m", [3, 300])
def test_captured_and_replayed(m):
    """A linear step in a graph: each replay sees its inputs of then."""
    x = torch.randn(m, 260, device=DEV)
    w = torch.randn(150, 260, device=DEV)
    dy = torch.randn(m, 150, device=DEV)

    def step():
        w8 = fp8.gqs_fp8_weight(w)
        return (fp8.gqs_fp8_linear(x, w8),
                fp8.gqs_fp8_linear(dy, w8, transposed=True, seed=SEED))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, dx = step()
    for i in range(4):
        for t in (x, w, dy):
            t.copy_(torch.randn_like(t))
        graph.replay()
        want = step()
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(dx, want[1]), i


def test_offsets_past_32_bits():
    """A row copy and a result of more than 2^32 bytes: the last rows."""
    m, k, n = (1 << 18) + 300, 16500, 8200  # 4.3 G codes, 4.3 GB of bf16 results
    x = torch.zeros(m, k, device=DEV, dtype=torch.bfloat16)
    at = [0, 5, (1 << 17) + 1, m - 130, m - 1]
    for i, r in enumerate(at):
        x[r] = torch.randint(-1, 2, (k,), device=DEV, dtype=torch.int32).to(x.dtype)
        x[r, i * 100:] = 0
        x[r, k - 1] = 1
    w = torch.ones(n, k, device=DEV, dtype=torch.bfloat16)
    y = fp8.gqs_fp8_linear(x, fp8.gqs_fp8_weight(w, transposed=False))
    want = x[at].float().sum(dim=1)
    assert torch.equal(y[at].float(), want[:, None].expand(-1, n))
    assert not y[m - 129:m - 1].any() and not y[6:1000].any()


# sizes that reach every way of the product, and the depth's split, at one
# fragment more and less than whole tiles
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m,n,k", [(4097, 4100, 130), (4095, 8191, 70), (2049, 4097, 400),
                                   (1023, 1025, 1100), (300, 2050, 3000), (129, 129, 5000),
                                   (65, 300, 4100), (20, 60, 9000), (8200, 260, 256)])
def test_every_way(m, n, k, dtype):
    """Whole numbers, whose sums are exact in any order: y and dx against
    plain products."""
    g = torch.Generator(device=DEV).manual_seed(m + n + k)

    def draw_whole(rows, cols):
        x = torch.randint(-2, 3, (rows, cols), device=DEV, generator=g).float()
        return x * (torch.rand(rows, cols, device=DEV, generator=g) < 0.2)
    x, w, dy = draw_whole(m, k), draw_whole(n, k), draw_whole(m, n)
    w8 = fp8.gqs_fp8_weight(w.to(DT[dtype]))
    for got, want in ((fp8.gqs_fp8_linear(x.to(DT[dtype]), w8), x @ w.t()),
                      (fp8.gqs_fp8_linear(dy.to(DT[dtype]), w8, transposed=True), dy @ w)):
        # products are at most 4, so no sum of eight is cut off; bf16 holds
        # whole numbers up to 256
        assert torch.equal(got.float(), want.to(DT[dtype]).float())
        assert want.abs().max() > 8


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("first", [1, 17, 33, 65, 97, 129, 257])
def test_rows_have_their_own_steps(first, dtype):
    """Every number of rows of a way for few of them, each row of another
    power of two."""
    n, k = 37, 300
    g = torch.Generator(device=DEV).manual_seed(first)

    def draw_whole(rows, cols):
        x = torch.randint(-2, 3, (rows, cols), device=DEV, generator=g).float()
        return x * (torch.rand(rows, cols, device=DEV, generator=g) < 0.2)
    w = draw_whole(n, k)
    w8 = fp8.gqs_fp8_weight(w.to(DT[dtype]))
    for m in range(first, first + 32):
        x = draw_whole(m, k)
        steps = torch.exp2((torch.arange(m, device=DEV) * 5 % 23 - 11).float())[:, None]
        got = fp8.gqs_fp8_linear((x * steps).to(DT[dtype]), w8)
        assert torch.equal(got.float() / steps, (x @ w.t()).to(DT[dtype]).float()), m


# each way, with one to three columns and some rows more than whole tiles
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m,n,k", [(4097, 4101, 130), (2049, 4098, 400), (1023, 1027, 1100),
                                   (300, 2050, 3000), (129, 129, 5000), (90, 301, 700),
                                   (20, 62, 9000), (8201, 259, 256), (5, 35, 300)])
@pytest.mark.parametrize("before", [64, 65])
def test_results_end_where_they_end(m, n, k, before, dtype):
    """Nothing is stored around a result, wherever it begins, and what is
    stored is what another call stores."""
    x = torch.randn(m, k, device=DEV).to(DT[dtype])
    w8 = fp8.gqs_fp8_weight(torch.randn(n, k, device=DEV).to(DT[dtype]))
    L, code = _step.lib(), 0 if dtype == "f32" else 1
    need = L.gqs_fp8_linear_workspace_bytes(m, n, k, code)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    held = torch.full((before + m * n + 64,), 5.0, device=DEV, dtype=DT[dtype])
    y = held[before:before + m * n]
    _step.check(L.gqs_fp8_linear(x.data_ptr(), code, m, k, k, 0, 0, w8.codes.data_ptr(),
                                 w8.exps.data_ptr(), n, 0, None, 0, y.data_ptr(), ws.data_ptr(),
                                 need, torch.cuda.current_stream().cuda_stream))
    assert (held[:before] == 5.0).all() and (held[before + m * n:] == 5.0).all()
    assert torch.equal(y.view(m, n), fp8.gqs_fp8_linear(x, w8))


@pytest.mark.parametrize("m,n,k", [(1, 1, 20000), (40, 1, 20000), (300, 1, 6000), (1, 20000, 1),
                                   (20000, 1, 1), (3000, 3, 3)])
def test_narrow_products(m, n, k):
    x = torch.ones(m, k, device=DEV, dtype=torch.bfloat16)
    x[-1] = 2
    w8 = fp8.gqs_fp8_weight(torch.ones(n, k, device=DEV, dtype=torch.bfloat16))
    y = fp8.gqs_fp8_linear(x, w8).float()
    want = torch.full((m, n), float(k), device=DEV)
    want[-1] *= 2
    assert torch.equal(y, want.bfloat16().float())
