"""Attention of one new token where its arithmetic has little room: logits whose
last bit is 16, weights far below a sequence's largest, logits of -inf, infinite
queries.

Bounds as in test_attention_decode_gpu.py: half a step of BF16, 2^-8 |o|; the
logits' error twice over and the rounding of each weight to FP16, (2^-11 + 2^-17
(1 + T)) sum p|v| / S; and 2^-32 of the largest weight for each weight that lies
below FP16's normal range, with its value: 2^-32 sum |v| / S (E4M3: each weight
has its value's scale in it, so 2^-32 n max(p |v|) / S)."""
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


@pytest.mark.parametrize("every,n", [(64, 17), (64, 32), (16, 5000)])
@pytest.mark.parametrize("below", [12, 18, 21, 23, 25])
@pytest.mark.parametrize("type", _cache.TYPES)
def test_values_far_below_the_largest_weight(type, below, every, n):
    """A token in every so many whose weight is 2^below times that of the others, and
    whose value is zero: the others' values alone make up the result."""
    g = torch.Generator(device="cuda").manual_seed(n + below)
    H, D = 8, 128
    q = torch.randn(H, D, generator=g, device="cuda").sign().bfloat16().float()
    q[:, :64] = 1.0
    k = torch.zeros(n, 1, D, device="cuda")
    k[::every, 0, :64] = 1.0
    v = torch.randn(n, 1, D, generator=g, device="cuda")
    v[::every] = 0.0
    scale = below * math.log(2.0) / 64
    o, lse, kv, vv = attend(type, q, k, v.bfloat16().float(), scale, 0.01 if type == qfp4.CACHE_NVFP4 else 1.0)
    kv, vv = kv[:, 0], vv[:, 0]
    x = q.double() @ kv.t() * float(np.float32(scale))
    T = (q.double().abs() @ kv.abs().t() * float(np.float32(scale))).amax(-1, keepdim=True)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    S = p.sum(-1, keepdim=True)
    want, size = p @ vv / S, p @ vv.abs() / S
    if type == qfp4.CACHE_E4M3:
        lost = 2.0 ** -32 * n * (p * vv.abs().amax(-1)).amax(-1, keepdim=True) / S
    else:
        lost = 2.0 ** -32 * vv.abs().sum(0) / S
    bound = 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2.0 ** -17 * (1 + T)) * size + lost
    assert ((o - want).abs() <= bound).all(), float(((o - want).abs() / bound).max())
    assert ((lse - torch.logsumexp(x, -1)).abs() <= 2.0 ** -18 * T[:, 0] + 2.0 ** -20 + 2.0 ** -22 * lse.abs()).all()


def test_logits_of_minus_infinity():
    """Keys of -inf: their tokens have no weight; where all are such, the sequence counts as one without tokens."""
    g = torch.Generator(device="cuda").manual_seed(1)
    n, D = 300, 64
    q = torch.rand(4, D, generator=g, device="cuda").bfloat16().float() + 0.5
    q = q.bfloat16().float()
    k, v = (torch.randn(n, 1, D, generator=g, device="cuda").bfloat16().float() for _ in range(2))
    gone = torch.rand(n, generator=g, device="cuda") < 0.7
    k[gone, 0, 5] = -math.inf
    o, lse, kv, vv = attend(qfp4.CACHE_BF16, q, k, v, 0.125)
    keep = ~gone
    x = q.double() @ kv[keep, 0].t() * 0.125
    p = torch.softmax(x, -1)
    want, size = p @ vv[keep, 0], p @ vv[keep, 0].abs()
    T = (q.double().abs() @ kv[keep, 0].abs().t() * 0.125).max()
    assert ((o - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2.0 ** -17 * (1 + T)) * size).all()
    assert ((lse - torch.logsumexp(x, -1)).abs() <= 2.0 ** -18 * T + 2.0 ** -20 + 2.0 ** -22 * lse.abs()).all()
    k[:, 0, 5] = -math.inf
    o, lse, *_ = attend(qfp4.CACHE_BF16, q, k, v, 0.125)
    assert (o == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("type", _cache.TYPES)
def test_infinite_query_beside_large_elements(type):
    """Every logit is -inf by the one infinite element, whatever the others add: no token counts.  With the other sign they are +inf: NaN."""
    n, D = 100, 64
    q = torch.full((2, D), 1e6, device="cuda")
    q[0, 3], q[1, 3] = math.inf, -math.inf
    k = torch.ones(n, 1, D, device="cuda")
    k[:, 0, 3] = -1.0
    o, lse, kv, _ = attend(type, q, k, torch.ones(n, 1, D, device="cuda"), 0.125, 0.01)
    assert (kv[:, 0, 3] < 0).all()
    assert (o[0] == 0).all() and lse[0] == -math.inf
    assert torch.isnan(o[1]).all() and torch.isnan(lse[1])
