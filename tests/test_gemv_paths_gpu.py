"""Few BF16 rows times 4-bit weights beyond the usual: infinite activations beside
large ones, and sizes that take several passes over K and several rounds of rows.
Bound as in test_gemv_gpu.py."""
import pytest
import torch

from block_scaled_fp4_tcgen05_gb300 import qfp4
from tests.test_gemv_gpu import GRID, MX, NV, check, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qfp4.load()
    assert qfp4.device_check() == 0


@pytest.mark.parametrize("large", [1e5, 1e20, 1e34])
@pytest.mark.parametrize("fmt", [MX, NV])
def test_infinity_beside_large_elements(fmt, large):
    """An infinity times a weight that is not zero is an infinity of its sign, whatever else is in the row."""
    g = torch.Generator(device="cuda").manual_seed(1)
    code, mma, w = weights(fmt, 300, 1024, g, *((60, 70) if fmt == MX else (0x30, 0x40)))
    for at in (9, 700):
        x = (torch.randn(3, 1024, generator=g, device="cuda").clamp(-1, 1) * large).bfloat16()
        x[0] = x[0].sign()
        x[1, at] = float("inf")
        x[2, at] = float("-inf")
        d = torch.empty(3, 300, dtype=torch.bfloat16, device="cuda")
        qfp4.gemv_nt(fmt, x, code, mma, torch.tensor([2.0 ** -20], device="cuda"), d)
        zero = w[:, at] == 0
        assert torch.isfinite(d[0]).all()
        for row, sign in ((1, 1), (2, -1)):
            assert torch.isnan(d[row][zero]).all()
            assert torch.equal(d[row][~zero].double(), sign * w[:, at][~zero].sign() * float("inf"))


@pytest.mark.parametrize("N,K", [(64, 32768 + 128), (300, 32768 + 128), (1, 65536)])
@pytest.mark.parametrize("fmt", [MX, NV])
def test_several_passes_over_k(fmt, N, K):
    """16 rows of which shared memory holds 2048 elements at a time: even an eighth of K takes three passes and more, the last one odd."""
    g = torch.Generator(device="cuda").manual_seed(K + N)
    x = (torch.randn(16, K, generator=g, device="cuda") * torch.exp(torch.randn(16, K, generator=g, device="cuda"))).bfloat16()
    check(fmt, x, *weights(fmt, N, K, g), torch.tensor([0.37], device="cuda") if fmt == NV else None)


@pytest.mark.parametrize("M,K", [(16, 16384 + 128), (16, 32768), (3, 16384)])
@pytest.mark.parametrize("fmt", [MX, NV])
def test_several_rounds_of_rows(fmt, M, K):
    """More groups of 16 rows for each cluster than have sums in shared memory at once, with one pass over K or more."""
    g = torch.Generator(device="cuda").manual_seed(K + M)
    N, block, step = 33001, qfp4.block_size(fmt), 4096
    code = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    sf = torch.randint(*((118, 136) if fmt == MX else (0, 0x7F)), (N, K // block), generator=g, device="cuda", dtype=torch.uint8)
    mma = torch.zeros(qfp4.sf_mma_bytes(N, K // block), dtype=torch.uint8, device="cuda")
    qfp4.sf_interleave(sf, N, K // block, mma)
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    d = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    qfp4.gemv_nt(fmt, x, code, mma, None, d)
    table = torch.cat([GRID, -GRID]).cuda()
    for lo in range(0, N, step):        # in pieces: the weights in 64 bits are sixteen times the codes
        c, f = code[lo: lo + step], sf[lo: lo + step]
        scale = ((f.long() - 127 + 1023) << 52).view(torch.float64) if fmt == MX else f.view(torch.float8_e4m3fn).double()
        w = torch.stack([table[(c & 15).int()], table[(c >> 4).int()]], -1).flatten(1)
        w = (w.view(c.shape[0], K // block, block) * scale[..., None]).flatten(1)
        want = x.double() @ w.t()
        size, far = x.double().abs() @ w.abs().t(), x.double().abs().amax(1, keepdim=True) * w.abs().sum(1)
        bound = 2.0 ** -8 * want.abs() + (K / 16 + 16) * 2.0 ** -23 * size + 2.0 ** -33 * far
        assert ((d[:, lo: lo + step].double() - want).abs() <= bound).all(), lo
    assert qfp4.poll_device_status() == 0


@pytest.mark.parametrize("fmt", [MX, NV])
def test_weights_beyond_32_bits(fmt):
    """4.6 GB of weights, all zero but the last rows."""
    g = torch.Generator(device="cuda").manual_seed(2)
    N, K, tail, block = 140000, 65536, 200, qfp4.block_size(fmt)
    code = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda")
    sf = torch.full((N, K // block), 127 if fmt == MX else 0x38, dtype=torch.uint8, device="cuda")
    mma = torch.zeros(qfp4.sf_mma_bytes(N, K // block), dtype=torch.uint8, device="cuda")
    qfp4.sf_interleave(sf, N, K // block, mma)
    code[-tail:] = torch.randint(0, 256, (tail, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    x = torch.randn(2, K, generator=g, device="cuda").bfloat16()
    d = torch.full((2, N), 7.0, dtype=torch.bfloat16, device="cuda")
    qfp4.gemv_nt(fmt, x, code, mma, None, d)
    table, c = torch.cat([GRID, -GRID]).cuda(), code[-tail:]
    w = torch.stack([table[(c & 15).int()], table[(c >> 4).int()]], -1).flatten(1)         # scales of 1
    want, size = x.double() @ w.t(), x.double().abs() @ w.abs().t()
    far = x.double().abs().amax(1, keepdim=True) * w.abs().sum(1)
    assert (d[:, :-tail] == 0).all()
    assert ((d[:, -tail:].double() - want).abs() <= 2.0 ** -8 * want.abs() + (K / 16 + 16) * 2.0 ** -23 * size + 2.0 ** -33 * far).all()
