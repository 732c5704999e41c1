"""Attention of one new token over the most tokens that a page table may have."""
import math

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


@pytest.mark.parametrize("window", [0, 1000])
@pytest.mark.parametrize("type", _cache.TYPES)
def test_longest_sequence(type, window):
    """2^30 tokens, the most that a page table may have, its pages one page over and
    over; and a length beyond that, cut to it.  Keys of zero: every weight is the
    same.  The result is the value that each type keeps of 0, 1, -2 and 4; a
    sum of up to 2^19 like terms per warp, in chains of 2^15 with a rounding of 2^-24
    each: 2^-9 on both sums."""
    page_size, D, n = 16384, 64, 1 << 30
    k = torch.zeros(page_size, 1, D, device="cuda")
    v = torch.tensor([0.0, 1.0, -2.0, 4.0], device="cuda").repeat(D // 4).expand(page_size, 1, D).contiguous()
    gs = torch.tensor([2.0 ** -6], device="cuda") if type == qfp4.CACHE_NVFP4 else None
    cache = _cache.empty(type, 2, 1, D, page_size, 0xFF)
    value = _cache.put(type, cache, page_size, torch.arange(page_size, device="cuda") + page_size, k, v, gs, gs)[1][0, 0].double()
    table = torch.ones(1, n // page_size, dtype=torch.int32, device="cuda")
    q = torch.ones(1, 2, D, dtype=torch.bfloat16, device="cuda")
    o, lse = torch.empty(1, 2, D, dtype=torch.bfloat16, device="cuda"), torch.empty(1, 2, device="cuda")
    ws = torch.zeros(qfp4.attention_decode_workspace_bytes(1, 2, 1, D), dtype=torch.uint8, device="cuda")
    for length, status in ((n, 0), (2 ** 31 - 1, -1)):
        qfp4.attention_decode(type, q, cache, page_size, table, torch.tensor([length], dtype=torch.int32, device="cuda"), 0.125, o, ws, gs, gs, lse=lse,
                              window=window)
        assert qfp4.poll_device_status() == status
        assert ((o[0].double() - value).abs() <= (2.0 ** -8 + 2.0 ** -8) * value.abs()).all()
        want = math.log(window or n)
        assert ((lse[0].double() - want).abs() <= 2.0 ** -9 + 2.0 ** -20 + 2.0 ** -22 * want).all()
        assert not ws[:16384].any()
