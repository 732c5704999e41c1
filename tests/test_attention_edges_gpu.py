"""Attention of one new token where its arithmetic has little room."""
import math

import numpy as np
import pytest
import torch

from block_scaled_fp4_tcgen05_gb300 import qfp4
from tests import _cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qfp4.load()
    assert qfp4.device_check() == 0


def attend(type, q, k, v, scale, gs=1.0, window=0):
    """One sequence: q [H, D], k and v [n, KV, D] fp32 that the cache's type is given; the values it keeps."""
    (H, D), (n, KV, _) = q.shape, k.shape
    pages = -(-n // 16)
    g = torch.tensor([gs], device="cuda") if type == qfp4.CACHE_NVFP4 else None
    cache = _cache.empty(type, pages, KV, D, 16, 0xFF)
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    kv, vv = _cache.put(type, cache, 16, slots, k, v, g, g)
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    o, lse = torch.full((1, H, D), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((1, H), 7.0, device="cuda")
    ws = torch.zeros(qfp4.attention_decode_workspace_bytes(1, H, KV, D), dtype=torch.uint8, device="cuda")
    qfp4.attention_decode(type, q.bfloat16()[None], cache, 16, table, torch.tensor([n], dtype=torch.int32, device="cuda"), scale, o, ws, g, g, kv_heads=KV,
                          lse=lse, window=window)
    assert qfp4.poll_device_status() == 0
    return o[0].double(), lse[0].double(), kv.double(), vv.double()


@pytest.mark.parametrize("period", [128, 256, 512])
@pytest.mark.parametrize("type", _cache.TYPES)
def test_logits_whose_last_bit_is_16(type, period):
    """Logits 2^27 + 16 and 2^27 + 32 in units of log 2, by turns: the weights relative
    to each other are 1 and 2^-16, and all values alike, whatever a logit's last bit."""
    scale = np.float32(math.log(2.0))
    while np.float32(scale * np.float32(1.44269504088896341)) != 1.0:
        scale = np.nextafter(scale, np.float32(1.0))
    n, D = 32768, 64
    q = torch.zeros(4, D, device="cuda")
    q[:, 0], q[:, 1] = 2.0 ** 27, 16.0
    k = torch.zeros(n, 1, D, device="cuda")
    k[..., 0], k[..., 63] = 1.0, {qfp4.CACHE_BF16: 1.0, qfp4.CACHE_E4M3: 448.0, qfp4.CACHE_NVFP4: 6.0}[type]       # the types' scales become 1
    k[..., 1:16] = k[..., :1]
    q[:, 1:3] = 16.0
    k[..., 2] = (torch.arange(n, device="cuda") // period % 2)[:, None].float()
    if type == qfp4.CACHE_NVFP4:
        k[..., 15] = 6.0
    v = torch.full((n, 1, D), 448.0 if type == qfp4.CACHE_E4M3 else 6.0, device="cuda")
    o, lse, _, vv = attend(type, q, k, v, float(scale))
    assert (vv == v).all()
    assert ((o - v[0].double()).abs() <= (2.0 ** -8 + 2.0 ** -11) * v[0].double()).all(), o
    assert torch.isfinite(lse).all()
