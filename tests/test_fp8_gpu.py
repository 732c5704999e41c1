"""8-bit floating point with a scale per 128 elements: the quantisers bit for
bit against their rule, the products against 64-bit sums."""
import numpy as np
import pytest
import torch

from block_scaled_fp4_tcgen05_gb300 import qfp4

pytestmark = pytest.mark.gpu

BLOCK = 128
TYPES = {qfp4.E4M3: (torch.float8_e4m3fn, 448.0), qfp4.E5M2: (torch.float8_e5m2, 57344.0)}
FLOOR = np.float32(2.0 ** -100)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qfp4.load()
    assert qfp4.device_check() == 0


def settled():
    torch.cuda.synchronize()
    return qfp4.poll_device_status()


# ------------------------------------------------------------------ quantisers

def values(rows, cols, seed, sigma=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * sigma
    far = torch.rand(rows, cols, generator=g) < 0.01
    return torch.where(far, x * 20, x).bfloat16()


def scales_of(amax, kind, pow2):
    """fp32 scale and factor of each block, by the rule."""
    top = np.float32(TYPES[kind][1])
    a = np.maximum(amax.astype(np.float32), FLOOR)
    t = (a / top).astype(np.float32)
    with np.errstate(divide="ignore", over="ignore"):
        if not pow2:
            return t, (top / a).astype(np.float32)
        mantissa, exponent = np.frexp(t.astype(np.float64))
        s = np.where(np.isinf(t), np.inf, 2.0 ** np.where(mantissa == 0.5, exponent - 1.0, exponent))
        return s.astype(np.float32), (1.0 / s).astype(np.float32)


def encode(x, factor, kind):
    """Decoded codes (64 bits) of fp32 x under its blocks' factors."""
    dtype, top = TYPES[kind]
    with np.errstate(invalid="ignore"):
        y = (x.astype(np.float32) * factor.astype(np.float32)).astype(np.float32)
    y = torch.from_numpy(y)
    return torch.where(y.isnan(), y, y.clamp(-top, top)).to(dtype).double().numpy()


def rows_rule(x, kind, pow2):
    """Codes [M, K] (decoded) and scales [ceil(K/128), M]."""
    x = x.float().numpy()
    M, K = x.shape
    kb = -(-K // BLOCK)
    mag = np.zeros((M, kb * BLOCK), np.float32)
    mag[:, :K] = np.nan_to_num(np.abs(x), nan=0.0, posinf=np.inf)
    s, f = scales_of(mag.reshape(M, kb, BLOCK).max(2), kind, pow2)
    return encode(x, np.repeat(f, BLOCK, 1)[:, :K], kind), s.T


def same(got, want):
    return np.array_equal(got, want, equal_nan=True)


def run_quantize(x, kind, pow2, rows=True, cols=True, index=None):
    M, K = (x.shape[0] if index is None else len(index)), x.shape[1]
    dtype = TYPES[kind][0]
    q = torch.full((M, K), 1.0, device="cuda").to(dtype) if rows else None
    sf = torch.full((-(-K // BLOCK), M), -1.0, device="cuda") if rows else None
    qt = torch.full((K, -(-M // 16) * 16), 1.0, device="cuda").to(dtype) if cols else None
    sft = torch.full((-(-M // BLOCK), K), -1.0, device="cuda") if cols else None
    ix = None if index is None else torch.tensor(index, dtype=torch.int32, device="cuda")
    qfp4.fp8_quantize(kind, x.cuda(), q, sf, qt, sft, scale=qfp4.SCALE_POW2 if pow2 else qfp4.SCALE_FP32, row_index=ix)
    return q, sf, qt, sft


def check_quantized(x, out, kind, pow2):
    q, sf, qt, sft = out
    M, K = x.shape
    if q is not None:
        want, scale = rows_rule(x, kind, pow2)
        assert same(sf.cpu().numpy(), scale)
        assert same(q.cpu().double().numpy(), want)
    if qt is not None:
        want, scale = rows_rule(x.t().contiguous(), kind, pow2)
        assert same(sft.cpu().numpy(), scale)
        assert same(qt.cpu().double().numpy()[:, :M], want)
        assert not qt.view(torch.uint8)[:, M:].any()


@pytest.mark.parametrize("kind", [qfp4.E4M3, qfp4.E5M2])
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("M,K", [(1, 16), (1, 4096), (15, 144), (127, 128), (128, 256), (129, 1040), (300, 48), (513, 2000)])
def test_quantize_follows_its_rule(kind, pow2, M, K):
    x = values(M, K, 31 * M + K)
    for rows, cols in ((True, False), (False, True), (True, True)):
        check_quantized(x, run_quantize(x, kind, pow2, rows, cols), kind, pow2)
    assert settled() == 0


@pytest.mark.parametrize("kind", [qfp4.E4M3, qfp4.E5M2])
@pytest.mark.parametrize("pow2", [False, True])
def test_quantize_extremes(kind, pow2):
    """Zero blocks, the smallest and largest values, infinities and NaN."""
    x = values(256, 256, 5)
    x[0] = 0.0
    x[1] = -0.0
    x[2] = 2.0 ** -133                      # BF16 subnormals
    x[3] = 2.0 ** -100
    x[4] = 3.38e38
    x[5, :128] = float("inf")
    x[6, 7] = float("-inf")
    x[7, 200] = float("nan")
    x[8, :] = float("nan")
    x[9, 0] = 448.0
    x[10, 0] = 448.0 * (1 + 2 ** -7)
    x[11] *= 2.0 ** -60
    check_quantized(x, run_quantize(x, kind, pow2), kind, pow2)
    assert settled() == 0


def test_quantize_gathers_rows():
    x = values(50, 400, 9)
    index = [3, 49, 0, -1, 3, 3, 17, -7] + list(range(49, -1, -1)) * 3
    want = torch.stack([x[i] if i >= 0 else torch.zeros(400, dtype=torch.bfloat16) for i in index])
    for rows, cols in ((True, False), (False, True), (True, True)):
        check_quantized(want, run_quantize(x, qfp4.E4M3, False, rows, cols, index), qfp4.E4M3, False)
    assert settled() == 0
    # an index beyond X is reported; its row is zero and the others stand
    index[4] = 50
    want[4] = 0.0
    check_quantized(want, run_quantize(x, qfp4.E4M3, False, True, True, index), qfp4.E4M3, False)
    assert settled() == -1
    assert settled() == 0


def group_tiles(offsets):
    """First 128-column tile of each group, and how many there are."""
    at = [0]
    for lo, hi in zip(offsets, offsets[1:]):
        at.append(at[-1] + -(-(hi - lo) // BLOCK))
    return at


@pytest.mark.parametrize("offsets,K", [([0, 5], 144), ([0, 0, 128, 128, 257, 300], 272), ([0, 1, 2, 3], 16),
                                       ([0, 0, 0], 32), ([0] + [3 * i for i in range(1, 257)], 48), ([0, 700, 1500], 640)])
@pytest.mark.parametrize("pow2,rows,gather", [(False, True, False), (True, False, True)])
def test_quantize_grouped(offsets, K, pow2, rows, gather):
    """Each group's blocks along the columns begin anew; what no group reaches
    stays as it was."""
    kind, G, used = qfp4.E4M3, len(offsets) - 1, offsets[-1]
    M = used + 20
    x = values(M, K, 3 * M)
    index = torch.randperm(M, generator=torch.Generator().manual_seed(1)) if gather else torch.arange(M)
    cols = qfp4.fp8_grouped_cols(M, G)
    seven = torch.full((1,), 7.0).to(TYPES[kind][0])
    q = seven.expand(M, K).contiguous().cuda() if rows else None
    sf = torch.full((-(-K // BLOCK), M), -1.0, device="cuda") if rows else None
    qt, sft = seven.expand(K, cols).contiguous().cuda(), torch.full((cols // BLOCK, K), -1.0, device="cuda")
    offs = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    qfp4.fp8_quantize_grouped(kind, x.cuda(), offs, qt, sft, q, sf, scale=qfp4.SCALE_POW2 if pow2 else qfp4.SCALE_FP32,
                              row_index=index.int().cuda() if gather else None)
    assert settled() == 0
    want = x[index]
    tiles = group_tiles(offsets)
    qt, sft = qt.cpu(), sft.cpu()
    for e in range(G):
        lo, hi = offsets[e], offsets[e + 1]
        if lo == hi:
            continue
        codes, scale = rows_rule(want[lo:hi].t().contiguous(), kind, pow2)
        at = tiles[e] * BLOCK
        assert same(qt[:, at:at + hi - lo].double().numpy(), codes)
        assert not qt[:, at + hi - lo:tiles[e + 1] * BLOCK].view(torch.uint8).any()
        assert same(sft[tiles[e]:tiles[e + 1]].numpy(), scale)
    assert bool((qt[:, tiles[-1] * BLOCK:].float() == 7.0).all()) and bool((sft[tiles[-1]:] == -1.0).all())
    if rows:
        codes, scale = rows_rule(want[:used], kind, pow2)
        assert same(q[:used].cpu().double().numpy(), codes) and same(sf[:, :used].cpu().numpy(), scale)
        assert bool((q[used:].float() == 7.0).all()) and bool((sf[:, used:] == -1.0).all())


@pytest.mark.parametrize("kind", [qfp4.E4M3, qfp4.E5M2])
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("G,N,K", [(1, 1, 16), (1, 128, 128), (3, 200, 272), (2, 16, 1040), (1, 385, 144)])
def test_quantize_weight_follows_its_rule(kind, pow2, G, N, K):
    w = values(G * N, K, 77 * N + K, 0.02).view(G, N, K)
    nb, kb, nt = -(-N // BLOCK), -(-K // BLOCK), -(-N // 16) * 16
    dtype = TYPES[kind][0]
    for transpose in (False, True):
        q = torch.empty(G, N, K, dtype=dtype, device="cuda")
        sf = torch.full((G, nb, kb), -1.0, device="cuda")
        qt = torch.full((G, K, nt), 1.0, device="cuda").to(dtype) if transpose else None
        sft = torch.full((G, kb, nb), -1.0, device="cuda") if transpose else None
        qfp4.fp8_quantize_weight(kind, w.cuda(), q, sf, qt, sft, scale=qfp4.SCALE_POW2 if pow2 else qfp4.SCALE_FP32)
        assert settled() == 0
        x = w.float().numpy()
        full = np.zeros((G, nb * BLOCK, kb * BLOCK), np.float32)
        full[:, :N, :K] = np.abs(x)
        s, f = scales_of(full.reshape(G, nb, BLOCK, kb, BLOCK).max((2, 4)), kind, pow2)
        want = encode(x, np.repeat(np.repeat(f, BLOCK, 1), BLOCK, 2)[:, :N, :K], kind)
        assert same(sf.cpu().numpy(), s)
        assert same(q.cpu().double().numpy(), want)
        if transpose:
            assert same(sft.cpu().numpy(), s.transpose(0, 2, 1))
            assert same(qt.cpu().double().numpy()[:, :, :N], want.transpose(0, 2, 1))
            assert not qt.view(torch.uint8)[:, :, N:].any()


# -------------------------------------------------------------------- products

def operand(rows, K, kind, seed, per_block=False, groups=0):
    """Codes over the type's whole range of finite values, scales over eight
    powers of two."""
    g = torch.Generator().manual_seed(seed)
    lead = (groups,) if groups else ()
    top = TYPES[kind][1]
    x = torch.randn(*lead, rows, K, generator=g) * (top / 16)
    q = x.clamp(-top, top).to(TYPES[kind][0])
    kb = -(-K // BLOCK)
    shape = (*lead, -(-rows // BLOCK), kb) if per_block else (*lead, kb, rows)
    s = torch.exp2(torch.rand(*shape, generator=g) * 8 - 4) / top
    return q, s


def decoded(q, s, per_block):
    K, rows = q.shape[-1], q.shape[-2]
    if per_block:
        f = s.double().repeat_interleave(BLOCK, -2)[..., :rows, :].repeat_interleave(BLOCK, -1)[..., :K]
    else:
        f = s.double().transpose(-1, -2).repeat_interleave(BLOCK, -1)[..., :K]
    return q.double() * f


def bound(exact, terms, K, fp32):
    """Half a step of the output type, and the fp32 sums: 2^-24 of the terms'
    magnitudes for each block joined, two for its scales, and 16 for the
    tensor cores' sum of one block (eight additions truncated at 2^-23)."""
    return exact.abs() * 2.0 ** (-24 if fp32 else -8) + (-(-K // BLOCK) + 18) * 2.0 ** -24 * terms


def check_product(d, a, b, K, fp32, start=None):
    exact, terms = a @ b.t(), a.abs() @ b.abs().t()
    if start is not None:
        exact, terms = exact + start, terms + start.abs()
    err = (d.cpu().double() - exact).abs()
    worst = float((err / bound(exact, terms, K, fp32).clamp(min=1e-300)).max())
    assert worst <= 1.0, worst


def product(ta, tb, M, N, K, b_rows, fp32, seed=1, start=None):
    qa, sa = operand(M, K, ta, seed)
    qb, sb = operand(N, K, tb, seed + 1, per_block=b_rows == 128)
    d = torch.full((M, N), float("nan"), dtype=torch.float32 if fp32 else torch.bfloat16, device="cuda")
    if start is not None:
        d.copy_(start)
    args = [t.cuda() for t in (qa, sa, qb, sb)]
    qfp4.gemm_nt_fp8(ta, tb, M, N, K, *args, d, b_rows=b_rows, out=qfp4.OUT_FP32 if fp32 else qfp4.OUT_BF16,
                     accumulate=start is not None)
    assert settled() == 0
    check_product(d, decoded(qa, sa, False), decoded(qb, sb, b_rows == 128), K, fp32, start)


SIZES = [(1, 1, 16), (1, 128, 128), (1, 4096, 512), (2, 24, 48), (7, 200, 144), (8, 128, 2048), (16, 640, 1040),
         (33, 257, 272), (64, 384, 4096), (100, 128, 128), (128, 256, 640), (129, 127, 256), (200, 1000, 400),
         (256, 256, 128), (257, 513, 1024), (384, 640, 2000), (700, 130, 3200), (513, 2056, 16)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("b_rows", [128, 1])
def test_product(M, N, K, b_rows):
    product(qfp4.E4M3, qfp4.E4M3, M, N, K, b_rows, False, M + N + K)
    product(qfp4.E4M3, qfp4.E4M3, M, N, K, b_rows, True, M + N)


# sixteen tiles of 128 x 128 (their clusters of eight do not run at once), K split in two and not split, both widths
@pytest.mark.parametrize("M,N,K", [(128, 2048, 2048), (512, 512, 2048), (300, 1664, 512), (384, 4096, 256), (600, 2560, 384), (40, 60000, 256)])
@pytest.mark.parametrize("b_rows", [128, 1])
def test_product_however_k_is_split(M, N, K, b_rows):
    product(qfp4.E4M3, qfp4.E4M3, M, N, K, b_rows, b_rows == 1, N)


@pytest.mark.parametrize("ta,tb", [(qfp4.E4M3, qfp4.E5M2), (qfp4.E5M2, qfp4.E4M3), (qfp4.E5M2, qfp4.E5M2)])
@pytest.mark.parametrize("M,N,K", [(3, 136, 272), (40, 256, 1024), (300, 520, 400), (512, 512, 512)])
def test_product_types(ta, tb, M, N, K):
    product(ta, tb, M, N, K, 128, False)
    product(ta, tb, M, N, K, 1, True)


@pytest.mark.parametrize("M,N,K", [(1, 130, 64), (60, 256, 2048), (300, 520, 400), (512, 768, 512)])
@pytest.mark.parametrize("b_rows", [128, 1])
def test_product_accumulates(M, N, K, b_rows):
    start = torch.randn(M, N, generator=torch.Generator().manual_seed(3)).double() * 100
    start = start.float().double()
    product(qfp4.E4M3, qfp4.E4M3, M, N, K, b_rows, True, 4, start)


def test_empty_sums():
    d = torch.full((5, 7), 3.0, dtype=torch.bfloat16, device="cuda")
    z = torch.zeros(16, dtype=torch.uint8, device="cuda")
    s = torch.zeros(16, device="cuda")
    qfp4.gemm_nt_fp8(qfp4.E4M3, qfp4.E4M3, 5, 7, 0, z, s, z, s, d)
    assert settled() == 0 and not d.any()
    f = torch.full((5, 7), 3.0, device="cuda")
    qfp4.gemm_nt_fp8(qfp4.E4M3, qfp4.E4M3, 5, 7, 0, z, s, z, s, f, out=qfp4.OUT_FP32, accumulate=True)
    assert settled() == 0 and bool((f == 3.0).all())
    qfp4.gemm_nt_fp8(qfp4.E4M3, qfp4.E4M3, 5, 7, 0, z, s, z, s, f, out=qfp4.OUT_FP32)
    assert settled() == 0 and not f.any()


@pytest.mark.parametrize("M,N,K", [(4, 128, 256), (300, 256, 400)])
def test_nan_stays_in_its_row_and_column(M, N, K):
    """A NaN code of A spoils its row of D, one of B its column, nothing else; a
    scale of inf (a block that held an infinity) spoils its row."""
    qa, sa = operand(M, K, qfp4.E4M3, 1)
    qb, sb = operand(N, K, qfp4.E4M3, 2, per_block=True)
    qa.view(torch.uint8)[1, 3] = 0x7F
    qb.view(torch.uint8)[5, K - 1] = 0xFF
    sa[0, 2] = float("inf")
    d = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    qfp4.gemm_nt_fp8(qfp4.E4M3, qfp4.E4M3, M, N, K, *(t.cuda() for t in (qa, sa, qb, sb)), d)
    assert settled() == 0
    bad = ~torch.isfinite(d.cpu())
    want = torch.zeros(M, N, dtype=torch.bool)
    want[1] = True
    want[2] = True
    want[:, 5] = True
    assert torch.equal(bad, want)


GROUPS = [
    ([0, 5], 136, 272), ([0, 0, 0, 1], 128, 128), ([0, 300, 300, 450, 451], 264, 400), ([0, 128, 256, 384], 256, 256),
    ([0, 1, 2, 3, 4, 5, 6, 7, 8], 512, 1040), ([0, 700, 701, 1500], 512, 512), ([0] + [7 * i for i in range(1, 257)], 64, 144),
    ([0, 0, 0], 128, 128), ([0, 257, 513, 513, 1100], 1000, 640),
]


@pytest.mark.parametrize("offsets,N,K", GROUPS)
@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("unused", [0, 37])
def test_grouped(offsets, N, K, fp32, unused):
    """Experts with no rows, one row, rows that end inside a tile; rows beyond
    the last offset stay as they were."""
    used, G = offsets[-1], len(offsets) - 1
    rows = used + unused
    if rows == 0:
        rows = 1
    qa, sa = operand(rows, K, qfp4.E4M3, 3)
    qb, sb = operand(N, K, qfp4.E4M3, 4, per_block=True, groups=G)
    d = torch.full((rows, N), 7.0, dtype=torch.float32 if fp32 else torch.bfloat16, device="cuda")
    offs = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    most = max(b - a for a, b in zip(offsets, offsets[1:]))
    for bound_rows in (0, most):
        d.fill_(7.0)
        qfp4.gemm_nt_fp8_grouped(qfp4.E4M3, qfp4.E4M3, offs, rows, bound_rows, N, K,
                                 *(t.cuda() for t in (qa, sa, qb, sb)), d, out=qfp4.OUT_FP32 if fp32 else qfp4.OUT_BF16)
        assert settled() == 0
        a, b = decoded(qa, sa, False), decoded(qb, sb, True)
        for e in range(G):
            lo, hi = offsets[e], offsets[e + 1]
            if hi > lo:
                check_product(d[lo:hi], a[lo:hi], b[e], K, fp32)
        assert bool((d[used:] == 7.0).all())


@pytest.mark.parametrize("fp32", [False, True])
def test_grouped_many_tiles_of_a_short_sum(fp32):
    """Groups of up to 128 rows, more tiles than three rounds: bounded, by pairs of CTAs."""
    rows = [(37 * i) % 129 for i in range(64)]
    test_grouped([sum(rows[:i]) for i in range(65)], 1100, 272, fp32, 5)


@pytest.mark.parametrize("offsets,most", [([1, 4, 8], 0), ([0, 6, 4], 0), ([0, 4, 9], 0), ([0, -2, 8], 0), ([0, 2, 8], 5)])
def test_grouped_refuses_bad_offsets(offsets, most):
    K, N, rows = 128, 128, 8
    qa, sa = operand(rows, K, qfp4.E4M3, 3)
    qb, sb = operand(N, K, qfp4.E4M3, 4, per_block=True, groups=2)
    d = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device="cuda")
    offs = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    qfp4.gemm_nt_fp8_grouped(qfp4.E4M3, qfp4.E4M3, offs, rows, most, N, K, *(t.cuda() for t in (qa, sa, qb, sb)), d)
    assert settled() == -1
    assert bool((d == 7.0).all())
    assert settled() == 0


@pytest.mark.parametrize("offsets,M,N", [([0, 5], 136, 24), ([0, 0, 128, 128, 257, 300], 264, 130), ([0, 1, 2, 3], 16, 256),
                                         ([0, 0, 0], 40, 128), ([0] + [3 * i for i in range(1, 257)], 48, 64),
                                         ([0, 700, 1500], 300, 515), ([0, 900, 900, 2500], 512, 256)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_kgrouped(offsets, M, N, accumulate):
    """Each expert's weight gradient; none where no row came to it."""
    G, used = len(offsets) - 1, offsets[-1]
    rows = used + 9
    cols, tiles = qfp4.fp8_grouped_cols(rows, G), group_tiles(offsets)
    qa, sa = operand(M, cols, qfp4.E5M2, 3)
    qb, sb = operand(N, cols, qfp4.E4M3, 4)
    for t in (qa, qb):          # what no group reaches may hold anything
        t.view(torch.uint8)[:, tiles[-1] * BLOCK:] = 0x7F
    start = torch.randn(G, M, N, generator=torch.Generator().manual_seed(1)) * 10
    d = start.cuda() if accumulate else torch.full((G, M, N), float("nan"), device="cuda")
    offs = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    qfp4.gemm_nt_fp8_kgrouped(qfp4.E5M2, qfp4.E4M3, offs, rows, M, N, qa.cuda(), sa.cuda(), qb.cuda(), sb.cuda(), d,
                              accumulate=accumulate)
    assert settled() == 0
    a, b = decoded(qa, sa, False), decoded(qb, sb, False)
    for e in range(G):
        k = slice(tiles[e] * BLOCK, tiles[e + 1] * BLOCK)
        check_product(d[e], a[:, k], b[:, k], (tiles[e + 1] - tiles[e]) * BLOCK, True, start[e].double() if accumulate else None)


@pytest.mark.parametrize("offsets", [[1, 4, 8], [0, 6, 4], [0, 4, 9], [0, -2, 8]])
def test_grouped_training_refuses_bad_offsets(offsets):
    offs = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    qt = torch.full((64, qfp4.fp8_grouped_cols(8, 2)), 9, dtype=torch.uint8, device="cuda")
    sft = torch.full((qt.shape[1] // BLOCK, 64), -1.0, device="cuda")
    qfp4.fp8_quantize_grouped(qfp4.E4M3, values(8, 64, 1).cuda(), offs, qt, sft)
    assert settled() == -1 and bool((qt == 9).all()) and bool((sft == -1.0).all())
    d = torch.full((2, 64, 64), 7.0, device="cuda")
    qfp4.gemm_nt_fp8_kgrouped(qfp4.E4M3, qfp4.E4M3, offs, 8, 64, 64, qt, sft, qt, sft, d)
    assert settled() == -1 and bool((d == 7.0).all())
    assert settled() == 0


def test_training_products():
    """Forward, input gradient and weight gradient of one layer from one
    quantisation of X, W and dY, sizes that no tile divides."""
    M, N, K = 300, 200, 272
    x, w, dy = values(M, K, 1), values(N, K, 2, 0.02), values(M, N, 3, 1e-3)
    pad = torch.zeros(M, 208, dtype=torch.bfloat16)      # dY with zero columns beyond N, a multiple of 16
    pad[:, :N] = dy
    qx = run_quantize(x, qfp4.E4M3, False)
    qd = run_quantize(pad, qfp4.E5M2, False)
    q, sf = torch.empty(N, K, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(2, 3, device="cuda")
    qt, sft = torch.empty(K, 208, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(3, 2, device="cuda")
    qfp4.fp8_quantize_weight(qfp4.E4M3, w.cuda(), q, sf, qt, sft)
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    dx = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    dw = torch.empty(208, K, device="cuda")
    qfp4.gemm_nt_fp8(qfp4.E4M3, qfp4.E4M3, M, N, K, qx[0], qx[1], q, sf, y)
    qfp4.gemm_nt_fp8(qfp4.E5M2, qfp4.E4M3, M, K, 208, qd[0], qd[1], qt, sft, dx)
    qfp4.gemm_nt_fp8(qfp4.E5M2, qfp4.E4M3, 208, K, 304, qd[2], qd[3], qx[2], qx[3], dw, b_rows=1, out=qfp4.OUT_FP32)
    assert settled() == 0
    w64 = decoded(q.cpu(), sf.cpu(), True)
    check_product(y, decoded(qx[0].cpu(), qx[1].cpu(), False), w64, K, False)
    check_product(dx, decoded(qd[0].cpu(), qd[1].cpu(), False), decoded(qt.cpu(), sft.cpu(), True), 208, False)
    check_product(dw, decoded(qd[2].cpu(), qd[3].cpu(), False), decoded(qx[2].cpu(), qx[3].cpu(), False), 304, True)
    # against the unquantised product: an E4M3 code is within 2^-4 of its
    # value and an E5M2 code within 2^-3, or within half the smallest step;
    # a sum of K such terms with random signs stays far inside their sum
    for got, want in ((y, x.double() @ w.double().t()), (dx, dy.double() @ w.double()),
                      (dw[:N], dy.double().t() @ x.double())):
        rel = float((got.cpu().double() - want).norm() / want.norm())
        assert rel <= 2.0 ** -3, rel


def test_repeats_bit_for_bit_and_on_another_stream():
    M, N, K = 37, 1000, 4096
    qa, sa = (t.cuda() for t in operand(M, K, qfp4.E4M3, 1))
    qb, sb = (t.cuda() for t in operand(N, K, qfp4.E4M3, 2, per_block=True))
    outs = []
    side = torch.cuda.Stream()
    for stream in (None, side, None):
        d = torch.empty(M, N, device="cuda")
        torch.cuda.synchronize()
        qfp4.gemm_nt_fp8(qfp4.E4M3, qfp4.E4M3, M, N, K, qa, sa, qb, sb, d, out=qfp4.OUT_FP32, stream=stream)
        assert settled() == 0
        outs.append(d)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_captured_in_a_graph():
    """Quantiser and product, captured and replayed on new inputs."""
    M, N, K = 64, 256, 512
    x = values(M, K, 1).cuda()
    q, sf = torch.empty(M, K, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(4, M, device="cuda")
    qb, sb = (t.cuda() for t in operand(N, K, qfp4.E4M3, 2, per_block=True))
    d = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")

    def step():
        qfp4.fp8_quantize(qfp4.E4M3, x, q, sf)
        qfp4.gemm_nt_fp8(qfp4.E4M3, qfp4.E4M3, M, N, K, q, sf, qb, sb, d)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (3, 4):
        x.copy_(values(M, K, seed))
        step()
        torch.cuda.synchronize()
        want = d.clone()
        d.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(d, want)
    assert settled() == 0


@pytest.mark.parametrize("kind", ["gemm", "quant"])
def test_offsets_beyond_32_bits(kind):
    """Operands of more than 2^31 elements: the last rows are right."""
    if kind == "quant":
        M, K = 140000, 16384
        x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
        tail = values(128, K, 5)
        x[-128:] = tail.cuda()
        q = torch.empty(M, K, dtype=torch.float8_e4m3fn, device="cuda")
        sf = torch.empty(K // BLOCK, M, device="cuda")
        qt = torch.empty(K, M, dtype=torch.float8_e4m3fn, device="cuda")
        sft = torch.empty(-(-M // BLOCK), K, device="cuda")
        qfp4.fp8_quantize(qfp4.E4M3, x, q, sf, qt, sft)
        assert settled() == 0
        want, scale = rows_rule(tail, qfp4.E4M3, False)
        assert same(q[-128:].cpu().double().numpy(), want) and same(sf[:, -128:].cpu().numpy(), scale)
        assert not q[:-128].view(torch.uint8).any()
        block = torch.zeros(128, K, dtype=torch.bfloat16)      # the last block of the columns: 96 rows
        last = M - M // BLOCK * BLOCK or BLOCK
        want, scale = rows_rule(tail[-last:].t().contiguous(), qfp4.E4M3, False)
        assert same(qt[:, -last:].cpu().double().numpy(), want) and same(sft[-1].cpu().numpy(), scale[0])
        return
    M, N, K = 140000, 256, 16384
    qa = torch.zeros(M, K, dtype=torch.float8_e4m3fn, device="cuda")
    sa = torch.ones(K // BLOCK, M, device="cuda")
    ta, ts = operand(200, K, qfp4.E4M3, 1)
    qa[-200:] = ta.cuda()
    sa[:, -200:] = ts.cuda()
    qb, sb = operand(N, K, qfp4.E4M3, 2, per_block=True)
    d = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    qfp4.gemm_nt_fp8(qfp4.E4M3, qfp4.E4M3, M, N, K, qa, sa, qb.cuda(), sb.cuda(), d)
    assert settled() == 0
    check_product(d[-200:], decoded(ta, ts, False), decoded(qb, sb, True), K, False)
    assert not d[:-200].any()
