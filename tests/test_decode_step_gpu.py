"""The decoding attention layer's operators together: three steps of a layer over
a paged cache, from the hidden state to the output projection, against the same
layer in 64 bits."""
import math

import pytest
import torch

from block_scaled_fp4_tcgen05_gb300 import qfp4
from tests import _cache
from tests.test_gemv_gpu import weights

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qfp4.load()
    assert qfp4.device_check() == 0


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("type", _cache.TYPES)
def test_decoding_steps(type, captured):
    """Each step's inputs are the kernels' own outputs of the step before it in the
    64-bit layer too (the QKV rows, the cached values), so that the bounds are those
    of one operator at a time."""
    g = torch.Generator(device="cuda").manual_seed(type)
    B, H, KV, D, hidden, page_size, max_pages = 5, 8, 2, 128, 512, 16, 4
    width = (H + 2 * KV) * D
    wqkv, wo = weights(qfp4.NVFP4, width, hidden, g, 0x38, 0x40), weights(qfp4.MXFP4, hidden, H * D, g, 120, 124)
    gs_w = torch.tensor([0.02], device="cuda")
    qw, kw = ((1 + 0.2 * torch.randn(D, generator=g, device="cuda")).bfloat16() for _ in range(2))
    angle = torch.arange(max_pages * page_size, device="cuda", dtype=torch.float64)[:, None] * 100.0 ** (-torch.arange(0, D, 2, device="cuda") / D)
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()
    gs = [torch.tensor([v], device="cuda") if type == qfp4.CACHE_NVFP4 else None for v in (0.005, 0.02)]
    cache = _cache.empty(type, B * max_pages, KV, D, page_size, 0xFF)
    table = torch.randperm(B * max_pages, generator=g, device="cuda").int().view(B, max_pages)
    ws = torch.zeros(qfp4.attention_decode_workspace_bytes(B, H, KV, D), dtype=torch.uint8, device="cuda")
    start = torch.tensor([0, 1, 15, 16, 40], device="cuda")
    # the prompts, straight into the cache
    for b in range(B):
        n = int(start[b])
        if n:
            t = torch.arange(n, device="cuda")
            slots = (table[b].long()[t // page_size] * page_size + t % page_size).int()
            qfp4.kv_cache_write(type, *(torch.randn(n, KV, D, generator=g, device="cuda").bfloat16() for _ in range(2)), slots, cache, page_size, *gs)
    x = torch.empty(B, hidden, dtype=torch.bfloat16, device="cuda")
    qkv, q = torch.empty(B, width, dtype=torch.bfloat16, device="cuda"), torch.empty(B, H, D, dtype=torch.bfloat16, device="cuda")
    o, y = torch.empty(B, H, D, dtype=torch.bfloat16, device="cuda"), torch.empty(B, hidden, dtype=torch.bfloat16, device="cuda")
    positions, slots, lengths = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(3))
    scale = 1 / math.sqrt(D)

    def step():
        qfp4.gemv_nt(qfp4.NVFP4, x, wqkv[0], wqkv[1], gs_w, qkv)
        qfp4.qk_norm_rope_cache(qkv, H, KV, q, type, cache, page_size, slots, qw, kw, cos_sin, positions, *gs, eps=EPS)
        qfp4.attention_decode(type, q, cache, page_size, table, lengths, scale, o, ws, *gs)
        qfp4.gemv_nt(qfp4.MXFP4, o.view(B, H * D), wo[0], wo[1], None, y)

    graph = torch.cuda.CUDAGraph()
    for i in range(3):
        x.copy_(torch.randn(B, hidden, generator=g, device="cuda"))
        at = start + i
        positions.copy_(at)
        lengths.copy_(at + 1)
        slots.copy_(table.gather(1, (at // page_size)[:, None])[:, 0] * page_size + at % page_size)
        if captured and i == 1:
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                step()
        graph.replay() if captured and i > 0 else step()
        torch.cuda.synchronize()
        assert qfp4.poll_device_status() == 0
        close(qkv.double(), x.double() @ wqkv[2].t() * 0.02, x.double().abs() @ wqkv[2].abs().t() * 0.02)
        heads = qkv.view(B, -1, D)[:, : H + KV].double()
        z = heads / torch.sqrt((heads * heads).mean(-1, keepdim=True) + EPS) * torch.cat([qw.double().expand(H, D), kw.double().expand(KV, D)])
        c, s = (cos_sin.double()[at][:, None, k: k + D // 2] for k in (0, D // 2))
        a, b = z[..., : D // 2], z[..., D // 2:]
        close(q.double(), torch.cat([a * c - b * s, b * c + a * s], -1)[:, :H], z.abs().amax(-1, keepdim=True)[:, :H])
        for n in range(B):
            t = torch.arange(int(at[n]) + 1, device="cuda")
            where = (table[n].long()[t // page_size] * page_size + t % page_size).int()
            kc, vc = (torch.empty(t.numel(), KV, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
            qfp4.kv_cache_read(type, cache, page_size, where, kc, vc, *gs)
            # the read rounds to BF16 (2^-8 of each key and value): logits move by that much of their terms
            logits = torch.einsum("hgd,nhd->hgn", q[n].double().view(KV, -1, D), kc.double()) * scale
            terms = (torch.einsum("hgd,nhd->hgn", q[n].double().abs().view(KV, -1, D), kc.double().abs()) * scale).amax()
            p = torch.softmax(logits, -1)
            want, size = torch.einsum("hgn,nhd->hgd", p, vc.double()), torch.einsum("hgn,nhd->hgd", p, vc.double().abs())
            bound = 2.0 ** -8 * want.abs() + (2.0 ** -7 + 2.0 ** -7 * terms) * size
            assert ((o[n].double().view(KV, -1, D) - want).abs() <= bound).all()
        close(y.double(), o.double().view(B, -1) @ wo[2].t(), o.double().abs().view(B, -1) @ wo[2].abs().t())


def close(got, want, size):
    assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -16 * size).all()
