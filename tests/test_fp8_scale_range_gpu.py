"""The 8-bit products at the ends of the range of scales that include/qfp4.h
states their accuracy for."""
import pytest
import torch

from block_scaled_fp4_tcgen05_gb300 import qfp4

pytestmark = pytest.mark.gpu

BLOCK = 128
TYPES = {qfp4.E4M3: (torch.float8_e4m3fn, 448.0), qfp4.E5M2: (torch.float8_e5m2, 57344.0)}
# every kernel form: few rows in both orientations (one and two widths), the
# unswapped tile of 128 rows, CTA pairs 128 and 256 columns wide
SIZES = [(5, 200, 272), (24, 136, 1040), (100, 260, 640), (300, 520, 384), (2048, 1300, 272)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qfp4.load()
    assert qfp4.device_check() == 0


def codes(rows, K, kind, g, small):
    """Ordinary codes, or magnitudes of a few of the type's smallest steps."""
    dtype, top = TYPES[kind]
    x = torch.randn(rows, K, generator=g)
    return (x * (2.0 ** -8 if kind == qfp4.E4M3 else 2.0 ** -15) if small else (x * top / 16).clamp(-top, top)).to(dtype)


def spread(shape, power, g):
    return torch.exp2(torch.rand(*shape, generator=g) * 2 + power)


def expand(q, s, per_block):
    rows, K = q.shape
    if per_block:
        f = s.double().repeat_interleave(BLOCK, 0)[:rows].repeat_interleave(BLOCK, 1)[:, :K]
    else:
        f = s.double().t().repeat_interleave(BLOCK, 1)[:, :K]
    return q.double() * f


def check(d, a, b, K, fp32):
    """The bound that include/qfp4.h states: half a step of the output, 2^-24 of
    the terms per sum and scale, and the smallest steps below 2^-126."""
    blocks = -(-K // BLOCK)
    exact, terms = a @ b.t(), a.abs() @ b.abs().t()
    tol = exact.abs() * 2.0 ** (-24 if fp32 else -8) + (blocks + 18) * 2.0 ** -24 * terms
    tol += (blocks + 2) * 2.0 ** -149 + (0 if fp32 else 2.0 ** -134)
    err = (d.cpu().double() - exact).abs()
    assert bool((err <= tol).all()), float((err / tol).nan_to_num(nan=float("inf")).max())


# Powers of two of the two scales, small codes.  ANY: the product of the scales
# is zero, subnormal, or beyond the largest number, while D is none of these
# (b_rows = 1).  NORMAL: it nearly is.
ANY = [(-74, -70, False), (-94, -48, False), (-48, -94, False), (60, 66, True), (85, 46, True)]
NORMAL = [(-64, -62, False), (-94, -32, False), (-32, -94, False), (60, 63, True), (86, 37, True), (-94, 80, False)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("b_rows,pa,pb,small", [(1, *r) for r in ANY + NORMAL] + [(128, *r) for r in NORMAL])
def test_products_of_scales_at_the_ends_of_the_range(M, N, K, b_rows, pa, pb, small):
    g = torch.Generator().manual_seed(M + N - pa)
    ta, tb = qfp4.E5M2, qfp4.E4M3
    qa, qb = codes(M, K, ta, g, small), codes(N, K, tb, g, small)
    kb = -(-K // BLOCK)
    sa = spread((kb, M), pa, g)
    sb = spread((-(-N // BLOCK), kb) if b_rows == 128 else (kb, N), pb, g)
    sa[:, 1::3] = 2.0 ** max(-94, min(80, -pb - 4))     # rows whose products are ordinary, in every warp
    d = torch.full((M, N), float("nan"), device="cuda")
    qfp4.gemm_nt_fp8(ta, tb, M, N, K, qa.cuda(), sa.cuda(), qb.cuda(), sb.cuda(), d, b_rows=b_rows, out=qfp4.OUT_FP32)
    torch.cuda.synchronize()
    assert qfp4.poll_device_status() == 0
    check(d, expand(qa, sa, False), expand(qb, sb, b_rows == 128), K, True)


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("b_rows", [128, 1])
def test_zero_codes_add_nothing(M, N, K, b_rows):
    """Blocks without a code, under the largest scales whose product is finite
    (b_rows = 1: any) and under those the quantisers give blocks of zeros."""
    g = torch.Generator().manual_seed(M * 3 + N)
    qa, qb = codes(M, K, qfp4.E4M3, g, False), codes(N, K, qfp4.E4M3, g, False)
    kb = -(-K // BLOCK)
    sa = spread((kb, M), -10, g)
    sb = spread((-(-N // BLOCK), kb) if b_rows == 128 else (kb, N), -9, g)
    qa[:, :BLOCK] = 0
    sa[0] = 2.0 ** 120
    if b_rows == 128:
        sb[:, 0] = 2.0 ** 7
    else:
        sb[0] = 2.0 ** 30
    sa[1:, ::2] = 2.0 ** -116                                   # the scale of a block of zeros
    qa[::2] = 0
    d = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    qfp4.gemm_nt_fp8(qfp4.E4M3, qfp4.E4M3, M, N, K, qa.cuda(), sa.cuda(), qb.cuda(), sb.cuda(), d, b_rows=b_rows)
    torch.cuda.synchronize()
    assert qfp4.poll_device_status() == 0
    assert not d[::2].any()
    check(d, expand(qa, sa, False), expand(qb, sb, b_rows == 128), K, False)


@pytest.mark.parametrize("offsets,most,N", [([0, 3, 3, 20], 0, 200), ([0, 90, 130], 90, 136), ([0, 700, 701, 2048], 0, 1300)])
def test_grouped(offsets, most, N):
    K, M, G = 400, offsets[-1], len(offsets) - 1
    g = torch.Generator().manual_seed(N)
    qa, qb = codes(M, K, qfp4.E5M2, g, False), codes(G * N, K, qfp4.E4M3, g, False).view(G, N, K)
    sa, sb = spread((4, M), -90, g), spread((G, -(-N // BLOCK), 4), -36, g)
    sa[:, ::4] = 2.0 ** 30
    d = torch.full((M, N), float("nan"), device="cuda")
    offs = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    qfp4.gemm_nt_fp8_grouped(qfp4.E5M2, qfp4.E4M3, offs, M, most, N, K, qa.cuda(), sa.cuda(), qb.cuda(), sb.cuda(), d,
                             out=qfp4.OUT_FP32)
    torch.cuda.synchronize()
    assert qfp4.poll_device_status() == 0
    a = expand(qa, sa, False)
    for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        if hi > lo:
            check(d[lo:hi], a[lo:hi], expand(qb[e], sb[e], True), K, True)
