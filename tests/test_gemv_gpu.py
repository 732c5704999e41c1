"""Few BF16 rows times 4-bit weights against the product in 64 bits.

Bound, as the header states it: half a step of BF16; one rounding of at most 2^-23
per 16 elements of K in the tensor cores' sums and 16 for what follows; and what
an element far below its row's largest loses in FP16, 2^-33 of the largest."""
import pytest
import torch

from block_scaled_fp4_tcgen05_gb300 import qfp4

pytestmark = pytest.mark.gpu
MX, NV = qfp4.MXFP4, qfp4.NVFP4
GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qfp4.load()
    assert qfp4.device_check() == 0


def weights(fmt, N, K, g, lo=None, hi=None):
    """Any codes, scale bytes of a range: packed, MMA scales, values in 64 bits."""
    block = qfp4.block_size(fmt)
    code = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    lo, hi = (lo, hi) if lo is not None else (118, 136) if fmt == MX else (0, 0x7F)
    sf = torch.randint(lo, hi, (N, K // block), generator=g, device="cuda", dtype=torch.uint8)
    mma = torch.zeros(max(1, qfp4.sf_mma_bytes(N, K // block)), dtype=torch.uint8, device="cuda")
    qfp4.sf_interleave(sf, N, K // block, mma)
    table = torch.cat([GRID, -GRID]).cuda()
    w = torch.stack([table[(code & 15).long()], table[(code >> 4).long()]], -1).flatten(1)
    # powers of two by their exponent field: pow on the GPU is off by a last bit
    scale = ((sf.long() - 127 + 1023) << 52).view(torch.float64) if fmt == MX else sf.view(torch.float8_e4m3fn).double()
    return code, mma, (w.view(N, K // block, block) * scale[..., None]).flatten(1)


def check(fmt, x, code, mma, w, gs, d=None):
    M, K = x.shape
    N = code.shape[0]
    d = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda") if d is None else d
    qfp4.gemv_nt(fmt, x, code, mma, gs, d)
    f = 1.0 if gs is None or fmt == MX else gs.double()
    want = x.double() @ w.t() * f
    size = x.double().abs() @ w.abs().t() * f
    far = x.double().abs().amax(1, keepdim=True) * w.abs().sum(1) * f
    bound = 2.0 ** -8 * want.abs() + (K / 16 + 16) * 2.0 ** -23 * size + 2.0 ** -33 * far
    assert ((d.double() - want).abs() <= bound).all(), float(((d.double() - want).abs() / bound.clamp(min=1e-300)).max())
    assert qfp4.poll_device_status() == 0
    return d


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16])
@pytest.mark.parametrize("N,K", [(1, 128), (16, 128), (127, 256), (128, 1024), (130, 1152), (300, 2176), (1000, 4096), (4096, 4096), (64, 16384)])
@pytest.mark.parametrize("fmt", [MX, NV])
def test_product(fmt, N, K, M):
    g = torch.Generator(device="cuda").manual_seed(N + K + M)
    x = (torch.randn(M, K, generator=g, device="cuda") * torch.exp(torch.randn(M, K, generator=g, device="cuda"))).bfloat16()
    check(fmt, x, *weights(fmt, N, K, g), torch.tensor([0.37], device="cuda") if fmt == NV else None)


@pytest.mark.parametrize("fmt", [MX, NV])
def test_large(fmt):
    g = torch.Generator(device="cuda").manual_seed(1)
    check(fmt, torch.randn(5, 7168, generator=g, device="cuda").bfloat16(), *weights(fmt, 20000, 7168, g), None)


def test_each_element_in_its_place():
    """One element of x and one weight at a time: any mix-up of rows, columns or scales shows."""
    for fmt in (MX, NV):
        N, K, block = 256, 512, qfp4.block_size(fmt)
        g = torch.Generator(device="cuda").manual_seed(2)
        code, mma, w = weights(fmt, N, K, g)
        for k0 in range(0, K, 16):
            x = torch.zeros(16, K, dtype=torch.bfloat16, device="cuda")
            x[torch.arange(16), k0 + torch.arange(16)] = 1.0
            d = torch.empty(16, N, dtype=torch.bfloat16, device="cuda")
            qfp4.gemv_nt(fmt, x, code, mma, None, d)
            assert torch.equal(d.double(), w[:, k0: k0 + 16].t())       # at most 6 significant bits: exact


def test_range_of_scales():
    """MXFP4 scales from 2^-126 to 2^100 side by side, and 255, which is NaN."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(3, 1024, generator=g, device="cuda").bfloat16()
    check(MX, x, *weights(MX, 200, 1024, g, 1, 228), None)
    check(MX, (x * 1e-3).bfloat16(), *weights(MX, 200, 1024, g, 60, 61), None)
    code, mma, w = weights(MX, 128, 128, g)
    sf = torch.full((128, 4), 127, dtype=torch.uint8, device="cuda")
    sf[5, 2] = 255
    qfp4.sf_interleave(sf, 128, 4, mma)
    d = torch.empty(3, 128, dtype=torch.bfloat16, device="cuda")
    qfp4.gemv_nt(MX, x[:, :128].contiguous(), code, mma, None, d)
    assert torch.isnan(d[:, 5]).all() and torch.isfinite(d[:, :5]).all() and torch.isfinite(d[:, 6:]).all()


@pytest.mark.parametrize("K", [128, 384])
def test_every_scale_byte(K):
    """Rows of weights 1 with one MXFP4 scale byte each, in order and spread over the rows' groups: powers of two, exact."""
    for order in (torch.arange(228), torch.randperm(228, generator=torch.Generator().manual_seed(K))):
        sf = order.to(torch.uint8).cuda()[:, None].expand(228, K // 32).contiguous()
        mma = torch.empty(qfp4.sf_mma_bytes(228, K // 32), dtype=torch.uint8, device="cuda")
        qfp4.sf_interleave(sf, 228, K // 32, mma)
        code = torch.full((228, K // 2), 0x22, dtype=torch.uint8, device="cuda")
        x = torch.zeros(9, K, dtype=torch.bfloat16, device="cuda")
        x[torch.arange(9), torch.arange(9) * 14 + K - 128] = 1.0
        d = torch.empty(9, 228, dtype=torch.bfloat16, device="cuda")
        qfp4.gemv_nt(MX, x, code, mma, None, d)
        want = torch.ldexp(torch.ones(228, dtype=torch.float64), order - 127)
        assert torch.equal(d.double().cpu(), want.expand(9, 228))


def test_range_of_activations():
    """Rows of any size, and elements far below the largest."""
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(10, 2048, generator=g, device="cuda")
    x *= torch.tensor([1e-38, 1e-30, 1e-10, 1.0, 1e10, 1e30, 0.0, 1.0, 1.0, 1.0], device="cuda")[:, None]
    x[7] *= torch.exp(8 * torch.randn(2048, generator=g, device="cuda"))
    x[8, 100] = 1e20
    x[9, 1500:] *= 1e-12
    check(NV, x.bfloat16(), *weights(NV, 257, 2048, g, 0x30, 0x40), None)


def test_nan_and_infinity():
    g = torch.Generator(device="cuda").manual_seed(5)
    code, mma, w = weights(NV, 100, 256, g, 0x30, 0x40)
    x = torch.randn(4, 256, generator=g, device="cuda").bfloat16()
    good = check(NV, x, code, mma, w, None)
    x[1, 7], x[2, 9] = float("nan"), float("inf")
    d = torch.empty_like(good)
    qfp4.gemv_nt(NV, x, code, mma, None, d)
    assert torch.equal(d[0], good[0]) and torch.equal(d[3], good[3])
    assert torch.isnan(d[1]).all()
    zero = w[:, 9] == 0
    assert torch.isnan(d[2][zero]).all() and torch.isinf(d[2][~zero]).all() and (d[2][~zero].sign() == w[:, 9][~zero].sign()).all()


def test_strides_and_rows_left_alone():
    g = torch.Generator(device="cuda").manual_seed(6)
    N, K, M = 301, 384, 5
    code, mma, w = weights(NV, N, K, g)
    wide = torch.full((M + 2, K + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:M, 8: K + 8] = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    out = torch.full((M + 2, N + 10), 5.0, dtype=torch.bfloat16, device="cuda")
    check(NV, wide[:M, 8: K + 8], code, mma, w, None, out[:M, 3: N + 3])
    assert (out[M:] == 5).all() and (out[:, :3] == 5).all() and (out[:, N + 3:] == 5).all()


def test_empty():
    d = torch.full((2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    qfp4.gemv_nt(NV, torch.empty(2, 0, dtype=torch.bfloat16, device="cuda"), none.view(128, 0), none, None, d)
    assert (d == 0).all()
    qfp4.gemv_nt(NV, torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"), torch.zeros(128, 128, dtype=torch.uint8, device="cuda"),
                 torch.zeros(2048, dtype=torch.uint8, device="cuda"), None, torch.empty(0, 128, dtype=torch.bfloat16, device="cuda"))


def test_same_as_the_quantised_product_on_exact_inputs():
    """x that four bits hold exactly: gemm_nt's accumulator and this one stand for the same sum."""
    g = torch.Generator(device="cuda").manual_seed(7)
    M, N, K = 4, 256, 512
    code, mma, w = weights(NV, N, K, g, 0x38, 0x39)         # scales of 1
    xc, xm, x = weights(NV, M, K, g, 0x38, 0x39)
    a, b = torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    qfp4.gemv_nt(NV, x.bfloat16(), code, mma, None, a)
    qfp4.gemm_nt(NV, M, N, K, xc, xm, code, mma, None, None, b)
    assert torch.equal(a, b)                                # sums of multiples of 1/4 below 2^22: exact in fp32


def test_repeats_graph_and_streams():
    g = torch.Generator(device="cuda").manual_seed(8)
    cases = [(torch.randn(m, 4096, generator=g, device="cuda").bfloat16(), weights(f, n, 4096, g), f) for m, n, f in ((1, 4096, NV), (16, 1000, MX))]
    want = [check(f, x, *w, None) for x, w, f in cases]
    out = [torch.empty_like(d) for d in want]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        for (x, w, f), d in zip(cases, out):
            qfp4.gemv_nt(f, x, w[0], w[1], None, d)
    for _ in range(3):
        for d in out:
            d.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(20):
        for s, (x, w, f), d in zip(streams, cases, want):
            with torch.cuda.stream(s):
                got.append((torch.empty_like(d), d))
                qfp4.gemv_nt(f, x, w[0], w[1], None, got[-1][0])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in got)
