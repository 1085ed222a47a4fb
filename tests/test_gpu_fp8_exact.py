"""Products of few rows lose nothing in either type: their codes are multiplied
exactly and summed in fp32."""
import pytest

torch = pytest.importorskip("torch")

from allreduce_compatible_gradient_amd import _step, fp8  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    _step.lib()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m", [1, 2, 7, 16, 17, 32, 33, 64, 65, 96, 97, 128])
def test_small_products_beside_large_ones(m, dtype):
    """Products of +-2^16 that cancel and of 2^-2 between them: 18 bits apart,
    and sums below 2^21 of multiples of 2^-2, which fp32 holds.  The result, a
    quarter of the small ones' number, is exact in bf16."""
    n, k = 64, 512
    large = torch.tensor([256.0, 256.0, 0.5, 0.5], device=DEV).repeat(k // 4)
    signs = torch.tensor([1.0, -1.0, 1.0, 1.0], device=DEV).repeat(k // 4)
    x = large.expand(m, k).to(DT[dtype]).contiguous()
    w = (large * signs).expand(n, k).to(DT[dtype])
    w8 = fp8.gqs_fp8_weight(w)
    want = torch.full((m, n), k / 2 * 0.25, device=DEV, dtype=DT[dtype])
    assert torch.equal(fp8.gqs_fp8_linear(x, w8), want)
    assert torch.equal(fp8.gqs_fp8_product(fp8.gqs_fp8_rows(x), w8, dtype=DT[dtype]), want)
    # and transposed: every row of y's gradient the same
    back = fp8.gqs_fp8_linear(x, fp8.gqs_fp8_weight(w.t().contiguous()), transposed=True)
    assert torch.equal(back, want)
