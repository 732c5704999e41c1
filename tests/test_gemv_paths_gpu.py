"""Few BF16 rows times 4-bit weights: infinite activations beside large ones."""
import pytest
import torch

from block_scaled_fp4_tcgen05_gb300 import qfp4
from tests.test_gemv_gpu import MX, NV, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qfp4.load()
    assert qfp4.device_check() == 0


@pytest.mark.parametrize("large", [1e5, 1e20, 1e34])
@pytest.mark.parametrize("fmt", [MX, NV])
def test_infinity_beside_large_elements(fmt, large):
    """An infinity times a weight that is not zero is an infinity of its sign, whatever else is in the row."""
    g = torch.Generator(device="cuda").manual_seed(1)
    code, mma, w = weights(fmt, 300, 1024, g, *((60, 70) if fmt == MX else (0x30, 0x40)))
    for at in (9, 700):
        x = (torch.randn(3, 1024, generator=g, device="cuda").clamp(-1, 1) * large).bfloat16()
        x[0] = x[0].sign()
        x[1, at] = float("inf")
        x[2, at] = float("-inf")
        d = torch.empty(3, 300, dtype=torch.bfloat16, device="cuda")
        qfp4.gemv_nt(fmt, x, code, mma, torch.tensor([2.0 ** -20], device="cuda"), d)
        zero = w[:, at] == 0
        assert torch.isfinite(d[0]).all()
        for row, sign in ((1, 1), (2, -1)):
            assert torch.isnan(d[row][zero]).all()
            assert torch.equal(d[row][~zero].double(), sign * w[:, at][~zero].sign() * float("inf"))
