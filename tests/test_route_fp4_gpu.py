"""The router's rows and offsets given to the grouped FP4 calls: as they are
where every pair has a row, reported where some have none."""
import pytest
import torch

from block_scaled_fp4_tcgen05_gb300 import qfp4

pytestmark = pytest.mark.gpu
T, E, TOPK, N, K = 200, 6, 2, 256, 512


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qfp4.load()
    assert qfp4.device_check() == 0
    torch.cuda.synchronize()
    qfp4.poll_device_status()


def experts_product(valid):
    """(rows, their source tokens, their experts, D) of one routed FP4 product."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    w = (torch.randn(E, N, K, generator=g, device="cuda") / K ** 0.5).bfloat16()
    logits = torch.randn(T, E, generator=g, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    ids, dest, src = torch.empty(T, TOPK, **i32), torch.empty(T, TOPK, **i32), torch.empty(T * TOPK, **i32)
    counts, offs, n = torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(1, **i32)
    gates, mean, loss = torch.empty(T, TOPK, device="cuda"), torch.empty(E, device="cuda"), torch.empty(1, device="cuda")
    ws = torch.empty(qfp4.moe_route_workspace_bytes(T, E, TOPK), dtype=torch.uint8, device="cuda")
    qfp4.moe_route(logits, TOPK, ids, gates, counts, offs, dest, src, n, mean, loss, ws, valid=valid)
    rows, size = T * TOPK, qfp4.block_size(qfp4.MXFP4)
    ones = torch.ones(E, device="cuda")
    a = x[src.clamp(min=0).long()].contiguous()
    qa = torch.zeros(rows, K // 2, dtype=torch.uint8, device="cuda")
    sa = torch.zeros(qfp4.sf_mma_grouped_bytes(rows, E, K // size), dtype=torch.uint8, device="cuda")
    qfp4.quantize_grouped(qfp4.MXFP4, a, offs, ones, qa, sa)
    qb, sb = torch.empty(E * N, K // 2, dtype=torch.uint8, device="cuda"), []
    for e in range(E):
        s = torch.empty(qfp4.sf_mma_bytes(N, K // size), dtype=torch.uint8, device="cuda")
        qfp4.quantize(qfp4.MXFP4, w[e], None, qb[e * N:(e + 1) * N], s, qfp4.SF_MMA)
        sb.append(s)
    d = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device="cuda")
    qfp4.gemm_nt_grouped(qfp4.MXFP4, offs, rows, T, N, K, qa, sa, qb, torch.cat(sb), None, None, d)
    torch.cuda.synchronize()
    return x.double(), w.double(), src.long(), counts, d


def test_offsets_of_a_full_batch():
    x, w, src, counts, d = experts_product(None)
    assert qfp4.poll_device_status() == 0
    expert = torch.repeat_interleave(torch.arange(E, device="cuda"), counts.long())
    want = torch.einsum("rk,rnk->rn", x[src], w[expert])
    # an E2M1 code under a power-of-two scale is off by less than a quarter of its
    # value (or of its block's smallest step): a half for the two operands, and
    # random signs along K
    rel = float((d.double() - want).norm() / want.norm())
    assert rel <= 0.5, rel


def test_offsets_of_a_batch_with_padding_are_reported():
    valid = torch.ones(T, dtype=torch.uint8, device="cuda")
    valid[7] = 0
    *_, d = experts_product(valid)
    assert qfp4.poll_device_status() == -1 and qfp4.poll_device_status() == 0
    assert bool((d == 7.0).all())
