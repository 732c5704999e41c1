"""The router and its gradient where the batches are large: more pairs than a
warp keeps in registers, every range of tokens in use, and more tokens than one
pass of the gradient's grid."""
import pytest
import torch

from block_scaled_fp4_tcgen05_gb300 import qfp4

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
RANGES = 152            # at most, of tokens


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qfp4.load()
    assert qfp4.device_check() == 0


def logits_of(T, E, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=g) + torch.randn(E, generator=g) * 0.5).to(dtype)


def softmax64(l):
    x = torch.exp(l - l.amax(1, keepdim=True))
    return x / x.sum(1, keepdim=True)


def expected(l, k, valid, renorm):
    """Every output of the router by its definition, on the CPU in 64 bits."""
    T, E = l.shape
    p = softmax64(l.double()) * valid[:, None]
    ids = torch.sort(l.double(), dim=1, descending=True, stable=True)[1][:, :k]
    here = (valid != 0)[:, None].expand(T, k)
    gates = p.gather(1, ids) * here
    if renorm:
        total = gates.sum(1, keepdim=True)
        gates = gates / torch.where(total == 0, torch.ones_like(total), total)
    flat = torch.where(here, ids, E).reshape(-1)
    counts = torch.bincount(flat, minlength=E + 1)[:E]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    order = torch.sort(flat, stable=True)[1][:int(offsets[-1])]
    dest = torch.full((T * k,), -1, dtype=torch.int64)
    dest[order] = torch.arange(len(order))
    src = torch.full((T * k,), -1, dtype=torch.int64)
    src[:len(order)] = order // k
    n = int(valid.sum())
    mean = p.sum(0) / max(n, 1)
    return {"ids": torch.where(here, ids, -1), "gates": gates, "counts": counts, "row_offsets": offsets, "dest": dest.view(T, k),
            "src": src, "n_valid": torch.tensor([n]), "mean_prob": mean,
            "loss": (E / (k * max(n, 1)) * (counts.double() * mean).sum()).view(1)}


def route(l, k, valid, renorm):
    T, E = l.shape
    i32 = dict(dtype=torch.int32, device="cuda")
    o = {"ids": torch.full((T, k), 99, **i32), "gates": torch.full((T, k), 9.0, device="cuda"), "counts": torch.full((E,), 99, **i32),
         "row_offsets": torch.full((E + 1,), 99, **i32), "dest": torch.full((T, k), 99, **i32), "src": torch.full((T * k,), 99, **i32),
         "n_valid": torch.full((1,), 99, **i32), "mean_prob": torch.full((E,), 9.0, device="cuda"),
         "loss": torch.full((1,), 9.0, device="cuda")}
    ws = torch.full((qfp4.moe_route_workspace_bytes(T, E, k),), 0xA5, dtype=torch.uint8, device="cuda")
    qfp4.moe_route(l.cuda(), k, *o.values(), ws, valid=valid.cuda(), renorm=renorm)
    torch.cuda.synchronize()
    assert qfp4.poll_device_status() == 0
    return {n: t.cpu() for n, t in o.items()}


def lanes(E):
    return 4 if E <= 64 else 8 if E <= 128 else 32


# (256, 64, 16): one CTA, 256 pairs per warp.  The others use all 152 ranges,
# with more than 128 pairs per warp from 45000 x 8 on, and 19 ranges per part of
# the totals where E > 128.
@pytest.mark.parametrize("T,E,k", [(256, 64, 16), (45000, 16, 8), (40000, 7, 7), (30000, 100, 16), (16384, 256, 8), (50001, 130, 9)])
@pytest.mark.parametrize("dtype,renorm", [(torch.float32, True), (torch.bfloat16, False)])
def test_route(T, E, k, dtype, renorm):
    l = logits_of(T, E, T + E, dtype)
    valid = (torch.rand(T, generator=torch.Generator().manual_seed(1)) < 0.9).to(torch.uint8)
    got, want = route(l, k, valid, renorm), expected(l, k, valid, renorm)
    for name in ("ids", "counts", "row_offsets", "dest", "src", "n_valid"):
        assert torch.equal(got[name].long(), want[name]), name
    # exp of an argument rounded at 2^-24 of the logits' span and 2^-22 itself, a
    # sum of E terms in a tree of at most 13 additions, a division, a product
    span = float(l.double().amax() - l.double().amin())
    rel = (span + 4 + 13 + 4) * U
    assert bool(((got["gates"].double() - want["gates"]).abs() <= 2 * rel * want["gates"]).all())
    # a warp's tokens one after the other, its lanes' side by side, the warps of
    # a CTA, then the ranges in up to 64 parts of at most 19
    G = lanes(E)
    warps = 32 if G == 32 else 16
    chunk = -(-T // RANGES)
    sums = (-(-chunk * G // (32 * warps)) + 3 + warps + 19 + 64) * U
    mean = want["mean_prob"]
    assert bool(((got["mean_prob"].double() - mean).abs() <= (rel + sums) * mean).all())
    loss = float(want["loss"])
    assert abs(float(got["loss"].double()) - loss) <= (rel + sums + (E + 6) * U) * loss


# one pass of the grid takes 1216 CTAs of 8 warps of 32 / G tokens: 9728 tokens
# at E > 128, 77824 at E <= 32
@pytest.mark.parametrize("T,E,k", [(12000, 256, 8), (30001, 130, 3), (80000, 8, 2), (90000, 32, 4), (41000, 63, 6), (20000, 128, 8)])
@pytest.mark.parametrize("dtype,renorm", [(torch.float32, True), (torch.bfloat16, False), (torch.bfloat16, True)])
def test_gradient(T, E, k, dtype, renorm):
    g = torch.Generator().manual_seed(T)
    l = logits_of(T, E, T + E, dtype)
    valid = (torch.rand(T, generator=g) < 0.9).to(torch.uint8)
    want = expected(l, k, valid, renorm)
    dgates, dloss = torch.randn(T, k, generator=g), torch.rand(1, generator=g) * 100
    out = torch.full((T, E), 9.0, dtype=dtype, device="cuda")
    qfp4.moe_route_backward(l.cuda(), want["ids"].int().cuda(), want["counts"].int().cuda(), want["n_valid"].int().cuda(),
                            dgates.cuda(), dloss.cuda(), out, valid=valid.cuda(), renorm=renorm)
    torch.cuda.synchronize()
    assert qfp4.poll_device_status() == 0
    # d/dl of the gates' part and of the balance part, each through its softmax, and the terms' magnitudes
    alive = valid.double()[:, None]
    p, n = softmax64(l.double()), int(valid.sum())
    s = float(dloss) * E / (k * n * n) * want["counts"].double()
    at = want["ids"].clamp(min=0)
    share = want["gates"]
    dg = dgates.double() * alive
    pull, pull_abs = (share * dg).sum(1, keepdim=True), (share * dg.abs()).sum(1, keepdim=True)
    chosen = torch.zeros_like(p).scatter_add_(1, at, share * (dg - pull) if renorm else share * dg)
    chosen_abs = torch.zeros_like(p).scatter_add_(1, at, share * (dg.abs() + pull_abs))
    ps = (p * s).sum(1, keepdim=True)
    d = (chosen + p * (s - ps - (0 if renorm else pull))) * alive
    terms = (chosen_abs + p * (s + ps + pull_abs)) * alive
    # p to 2 (span + 21) half steps as above, sums of at most 24 terms
    span = float(l.double().amax() - l.double().amin())
    tol = (2 * (span + 21) + 48) * U * terms + (2.0 ** -8 * d.abs() if dtype == torch.bfloat16 else 0) + 1e-38
    err = (out.cpu().double() - d).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
