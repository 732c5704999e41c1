"""Weight gradients of the head norms: sums over all tokens and heads whose every
term counts, and a norm without eps.

Bound of a sum of n terms: each term within 64 roundings of fp32 of its own, and the
sum's chain, all of 2^-24: a lane adds its warp's blocks four vectors each, the
warp's groups are joined by two exchanges, two kinds and eight warps one after the
other, then the CTAs in 32 chains and a tree of five.  Where all terms have one sign
that is less than one term of the sum."""
import pytest
import torch

from block_scaled_fp4_tcgen05_gb300 import qfp4
from tests import test_head_norm_rope_gpu as heads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qfp4.load()
    assert qfp4.device_check() == 0


@pytest.mark.parametrize("H,KV", [(2, 2), (12, 2), (1, 1), (16, 8)])
@pytest.mark.parametrize("D", [48, 64, 128, 192, 256])
@pytest.mark.parametrize("inter", [False, True])
def test_without_eps(monkeypatch, D, H, KV, inter):
    """eps = 0, heads that fill no block of a warp and some that do."""
    monkeypatch.setattr(heads, "EPS", 0.0)
    s = heads.inputs(9, H, KV, D, D, True, D + H)
    _, dqw, dkw = heads.check_backward(s, 9, H, KV, D, D, inter)
    assert torch.isfinite(dqw).all() and torch.isfinite(dkw).all()


def chain(T, H, KV, D):
    lanes = 8 if D <= 64 else 16 if D <= 128 else 32
    block = 32 // lanes * 4
    items = T * (-(-H // block) - (-KV // block))
    ctas = min(-(-items // 8), 2 * 152)
    return 4 * -(-items // (8 * ctas)) + 2 + 2 + 8 + -(-ctas // 32) + 5


SUMS = [(3001, 12, 4, 64), (2000, 9, 2, 128), (1500, 5, 3, 256), (5000, 1, 1, 64), (777, 16, 16, 64), (4100, 3, 1, 80), (2500, 8, 8, 128)]


@pytest.mark.parametrize("signs", [False, True])
@pytest.mark.parametrize("T,H,KV,D", SUMS)
def test_every_term_counts(T, H, KV, D, signs):
    """Vectors of 1 and -1 under gradients of 1 to 3, nothing turned: whole numbers, all of one sign or of both."""
    g = heads.generator(T + D)
    sign = torch.randint(0, 2, (T, H + KV, D), generator=g, device="cuda") * 2 - 1
    dy = torch.randint(1, 4, (T, H + KV, D), generator=g, device="cuda")
    if signs:
        dy *= torch.randint(0, 2, dy.shape, generator=g, device="cuda") * 2 - 1
    qkv = torch.cat([sign, torch.ones(T, KV, D, device="cuda")], 1).flatten(1).bfloat16()
    dy = dy * sign
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    dq, dk = dy[:, :H].bfloat16().contiguous(), dy[:, H:].bfloat16().contiguous()
    dqw, dkw = torch.full((D,), 3.0, device="cuda"), torch.full((D,), 3.0, device="cuda")
    ws = torch.empty(qfp4.qk_norm_rope_backward_workspace_bytes(T, H, KV, D), dtype=torch.uint8, device="cuda").fill_(0xFF)
    qfp4.qk_norm_rope_backward(qkv, H, KV, dq, dk, torch.empty_like(qkv), dqw, dkw, ws, w, w, eps=0.0)
    each = (dy * sign).double()
    for got, want, size in ((dqw, each[:, :H].sum((0, 1)), each[:, :H].abs().sum((0, 1))), (dkw, each[:, H:].sum((0, 1)), each[:, H:].abs().sum((0, 1)))):
        bound = (chain(T, H, KV, D) + 64) * 2.0 ** -24 * size
        assert (bound < 1.0).all()      # less than a term
        assert ((got.double() - want).abs() <= bound).all(), float(((got.double() - want).abs() / bound).max())
    assert qfp4.poll_device_status() == 0


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,H,KV,D", SUMS)
def test_sums_of_any_terms(T, H, KV, D, inter):
    s = heads.inputs(T, H, KV, D, D, True, T + 1)
    _, dqw, dkw = heads.check_backward(s, T, H, KV, D, D, inter)
    _, _, a, b, ma, mb = heads.backward64(s, H, KV, D, D, inter, s["dq"], s["dk"], 1.0)
    for got, want, size in ((dqw, a, ma), (dkw, b, mb)):
        assert ((got.double() - want).abs() <= (chain(T, H, KV, D) + 64) * 2.0 ** -24 * size).all()


def test_gradient_offsets_beyond_32_bits():
    """Rows of every tensor far apart: the last one's offset passes 2^31 elements."""
    T, H, KV, D, ld = 3, 2, 1, 64, 1 << 30
    s = heads.inputs(T, H, KV, D, D, True, 3)
    want, dqw, dkw = heads.check_backward(s, T, H, KV, D, D, False)
    flat = [torch.zeros(2 * ld + 4 * D, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    qkv, grads, out = (f.as_strided((T, (H + 2 * KV) * D), (ld, 1)) for f in flat)
    qkv.copy_(s["qkv"])
    dq, dk = grads[:, : H * D].unflatten(1, (H, D)), grads[:, H * D: (H + KV) * D].unflatten(1, (KV, D))
    dq.copy_(s["dq"])
    dk.copy_(s["dk"])
    a, b = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    ws = torch.empty(qfp4.qk_norm_rope_backward_workspace_bytes(T, H, KV, D), dtype=torch.uint8, device="cuda")
    qfp4.qk_norm_rope_backward(qkv, H, KV, dq, dk, out, a, b, ws, s["qw"], s["kw"], s["table"], s["pos"], eps=heads.EPS)
    assert torch.equal(out[:, : (H + KV) * D], want[:, : (H + KV) * D]) and torch.equal(a, dqw) and torch.equal(b, dkw)
    assert qfp4.poll_device_status() == 0
