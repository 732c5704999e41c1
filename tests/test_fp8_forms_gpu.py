"""8-bit products in the kernel forms that real sizes take, at the smallest
sizes that take them: what is added to (`accumulate`) and the experts' weight
gradients on CTA pairs, 128 and 256 columns wide, by TMA and in pieces."""
import pytest
import torch

from block_scaled_fp4_tcgen05_gb300 import qfp4

pytestmark = pytest.mark.gpu

BLOCK = 128
TYPES = {qfp4.E4M3: (torch.float8_e4m3fn, 448.0), qfp4.E5M2: (torch.float8_e5m2, 57344.0)}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qfp4.load()
    assert qfp4.device_check() == 0


def settled():
    torch.cuda.synchronize()
    return qfp4.poll_device_status()


def operand(rows, K, kind, seed, per_block=False, groups=0):
    g = torch.Generator().manual_seed(seed)
    lead = (groups,) if groups else ()
    top = TYPES[kind][1]
    q = (torch.randn(*lead, rows, K, generator=g) * (top / 16)).clamp(-top, top).to(TYPES[kind][0])
    kb = -(-K // BLOCK)
    shape = (*lead, -(-rows // BLOCK), kb) if per_block else (*lead, kb, rows)
    return q, torch.exp2(torch.rand(*shape, generator=g) * 8 - 4) / top


def expand(q, s, per_block):
    rows, K = q.shape[-2:]
    if per_block:
        f = s.double().repeat_interleave(BLOCK, -2)[..., :rows, :].repeat_interleave(BLOCK, -1)[..., :K]
    else:
        f = s.double().transpose(-1, -2).repeat_interleave(BLOCK, -1)[..., :K]
    return q.double() * f


def check(d, a, b, K, fp32, start=None):
    """Half a step of the output, 2^-24 of the terms per sum, scale and block's
    own sum, as include/qfp4.h states."""
    exact, terms = a @ b.t(), a.abs() @ b.abs().t()
    if start is not None:
        exact, terms = exact + start.double(), terms + start.double().abs()
    tol = exact.abs() * 2.0 ** (-24 if fp32 else -8) + (-(-K // BLOCK) + 18) * 2.0 ** -24 * terms
    err = (d.cpu().double() - exact).abs()
    assert bool((err <= tol).all()), float((err / tol.clamp(min=1e-300)).max())


# On pairs: too short a K, or too many tiles, for the kernel of few rows to
# split K.  N % 4 == 0 leaves by TMA, the others in pieces; the last three are
# 256 columns wide.
PAIRS = [(300, 520, 384), (300, 519, 384), (129, 130, 272), (2048, 1300, 272), (2048, 1299, 272), (2500, 1408, 144)]


@pytest.mark.parametrize("M,N,K", PAIRS)
@pytest.mark.parametrize("b_rows", [128, 1])
@pytest.mark.parametrize("ta,tb", [(qfp4.E4M3, qfp4.E5M2), (qfp4.E5M2, qfp4.E4M3), (qfp4.E5M2, qfp4.E5M2)])
def test_pairs(M, N, K, b_rows, ta, tb):
    qa, sa = operand(M, K, ta, M)
    qb, sb = operand(N, K, tb, N, per_block=b_rows == 128)
    a, b = expand(qa, sa, False), expand(qb, sb, b_rows == 128)
    args = [t.cuda() for t in (qa, sa, qb, sb)]
    start = torch.randn(M, N, generator=torch.Generator().manual_seed(3)) * 100
    for out, accumulate in ((qfp4.OUT_BF16, False), (qfp4.OUT_FP32, False), (qfp4.OUT_FP32, True)):
        fp32 = out == qfp4.OUT_FP32
        d = start.cuda() if accumulate else torch.full((M, N), float("nan"), dtype=torch.float32 if fp32 else torch.bfloat16, device="cuda")
        qfp4.gemm_nt_fp8(ta, tb, M, N, K, *args, d, b_rows=b_rows, out=out, accumulate=accumulate)
        assert settled() == 0
        check(d, a, b, K, fp32, start if accumulate else None)


def test_pairs_beside_memory_of_others():
    """Nothing but D is written: rows before and after it stay."""
    M, N, K = 2050, 1300, 144
    qa, sa = operand(M, K, qfp4.E5M2, 1)
    qb, sb = operand(N, K, qfp4.E4M3, 2)
    whole = torch.full((M + 8, N), 7.0, device="cuda")
    d = whole[4:-4]
    qfp4.gemm_nt_fp8(qfp4.E5M2, qfp4.E4M3, M, N, K, *(t.cuda() for t in (qa, sa, qb, sb)), d, b_rows=1, out=qfp4.OUT_FP32,
                     accumulate=True)
    assert settled() == 0
    assert bool((whole[:4] == 7.0).all()) and bool((whole[-4:] == 7.0).all())
    check(d, expand(qa, sa, False), expand(qb, sb, False), K, True, torch.full((M, N), 7.0))


@pytest.mark.parametrize("M,N,K", [(5, 200, 272), (100, 260, 640), (300, 520, 384), (300, 519, 384), (2048, 1300, 272)])
@pytest.mark.parametrize("b_rows", [128, 1])
def test_accumulate_keeps_what_nothing_is_added_to(M, N, K, b_rows):
    """Zero codes add nothing: D stays bit for bit, numbers below 2^-126 too."""
    z = torch.zeros(max(M, N), K, dtype=torch.uint8, device="cuda")
    kb = -(-K // BLOCK)
    sa = torch.ones(kb, M, device="cuda")
    sb = torch.ones(*((-(-N // BLOCK), kb) if b_rows == 128 else (kb, N)), device="cuda")
    g = torch.Generator().manual_seed(N)
    start = torch.randn(M, N, generator=g) * torch.exp2(torch.randint(-148, 100, (M, N), generator=g).float())
    start[:, 3] = float("inf")
    d = start.cuda()
    qfp4.gemm_nt_fp8(qfp4.E4M3, qfp4.E4M3, M, N, K, z[:M], sa, z[:N], sb, d, b_rows=b_rows, out=qfp4.OUT_FP32, accumulate=True)
    assert settled() == 0
    assert torch.equal(d.cpu(), start)


@pytest.mark.parametrize("M,N", [(136, 24), (136, 23), (512, 1300)])
def test_kgrouped_accumulate_keeps_the_empty_experts(M, N):
    """An expert without rows: its D stays bit for bit, numbers below 2^-126 and
    negative zeros too."""
    offsets = [0, 0, 200, 200, 333]
    G, rows = 4, 340
    cols = qfp4.fp8_grouped_cols(rows, G)
    qa, sa = operand(M, cols, qfp4.E5M2, 1)
    qb, sb = operand(N, cols, qfp4.E4M3, 2)
    g = torch.Generator().manual_seed(N)
    start = torch.randn(G, M, N, generator=g) * torch.exp2(torch.randint(-148, 10, (G, M, N), generator=g).float())
    start[:, 0] = -0.0
    d = start.cuda()
    offs = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    qfp4.gemm_nt_fp8_kgrouped(qfp4.E5M2, qfp4.E4M3, offs, rows, M, N, qa.cuda(), sa.cuda(), qb.cuda(), sb.cuda(), d, accumulate=True)
    assert settled() == 0
    for e in (0, 2):
        assert torch.equal(d[e].cpu().view(torch.int32), start[e].view(torch.int32))
    a, b = expand(qa, sa, False), expand(qb, sb, False)
    for e, lo, hi in ((1, 0, 256), (3, 256, 512)):
        check(d[e], a[:, lo:hi], b[:, lo:hi], hi - lo, True, start[e])


# 256 columns wide: more than 76 tiles of 128, and no more than 76 of 256
@pytest.mark.parametrize("offsets,M,N", [([0, 5, 5, 300, 560], 512, 1300), ([0, 128, 257, 257, 700], 512, 1299),
                                         ([0, 1, 130], 1000, 1284), ([0] + [2 * i for i in range(1, 65)], 200, 256)])
@pytest.mark.parametrize("ta,tb", [(qfp4.E5M2, qfp4.E4M3), (qfp4.E4M3, qfp4.E5M2)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_kgrouped(offsets, M, N, ta, tb, accumulate):
    G, rows = len(offsets) - 1, offsets[-1] + 9
    cols = qfp4.fp8_grouped_cols(rows, G)
    tiles = [0]
    for lo, hi in zip(offsets, offsets[1:]):
        tiles.append(tiles[-1] + -(-(hi - lo) // BLOCK))
    qa, sa = operand(M, cols, ta, 3)
    qb, sb = operand(N, cols, tb, 4)
    start = torch.randn(G, M, N, generator=torch.Generator().manual_seed(1)) * 10
    d = start.cuda() if accumulate else torch.full((G, M, N), float("nan"), device="cuda")
    offs = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    qfp4.gemm_nt_fp8_kgrouped(ta, tb, offs, rows, M, N, qa.cuda(), sa.cuda(), qb.cuda(), sb.cuda(), d, accumulate=accumulate)
    assert settled() == 0
    a, b = expand(qa, sa, False), expand(qb, sb, False)
    for e in range(G):
        k = slice(tiles[e] * BLOCK, tiles[e + 1] * BLOCK)
        check(d[e], a[:, k], b[:, k], (tiles[e + 1] - tiles[e]) * BLOCK, True, start[e] if accumulate else None)


# by rows, 256 columns wide
@pytest.mark.parametrize("offsets,N,K", [([0, 700, 701, 2048], 1300, 272), ([0, 0, 1000, 2050], 1283, 144)])
@pytest.mark.parametrize("fp32", [False, True])
def test_grouped(offsets, N, K, fp32):
    G, rows = len(offsets) - 1, offsets[-1] + 5
    qa, sa = operand(rows, K, qfp4.E5M2, 3)
    qb, sb = operand(N, K, qfp4.E5M2, 4, per_block=True, groups=G)
    d = torch.full((rows, N), 7.0, dtype=torch.float32 if fp32 else torch.bfloat16, device="cuda")
    offs = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    qfp4.gemm_nt_fp8_grouped(qfp4.E5M2, qfp4.E5M2, offs, rows, 0, N, K, *(t.cuda() for t in (qa, sa, qb, sb)), d,
                             out=qfp4.OUT_FP32 if fp32 else qfp4.OUT_BF16)
    assert settled() == 0
    a, b = expand(qa, sa, False), expand(qb, sb, True)
    for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        if hi > lo:
            check(d[lo:hi], a[lo:hi], b[e], K, fp32)
    assert bool((d[offsets[-1]:] == 7.0).all())
