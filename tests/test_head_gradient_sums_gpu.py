"""Gradient of the head norms without eps, where places beyond the last head have no norm."""
import pytest
import torch

from block_scaled_fp4_tcgen05_gb300 import qfp4
from tests import test_head_norm_rope_gpu as heads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qfp4.load()
    assert qfp4.device_check() == 0


@pytest.mark.parametrize("H,KV", [(2, 2), (12, 2), (1, 1), (16, 8)])
@pytest.mark.parametrize("D", [48, 64, 128, 192, 256])
@pytest.mark.parametrize("inter", [False, True])
def test_without_eps(monkeypatch, D, H, KV, inter):
    """eps = 0, heads that fill no block of a warp and some that do."""
    monkeypatch.setattr(heads, "EPS", 0.0)
    s = heads.inputs(9, H, KV, D, D, True, D + H)
    _, dqw, dkw = heads.check_backward(s, 9, H, KV, D, D, inter)
    assert torch.isfinite(dqw).all() and torch.isfinite(dkw).all()
