"""Expert router and its gradient against 64-bit forms."""
import numpy as np
import pytest
import torch

from block_scaled_fp4_tcgen05_gb300 import qfp4

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qfp4.load()
    assert qfp4.device_check() == 0


def logits_of(T, E, seed, dtype=torch.float32, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=g) * spread + torch.randn(E, generator=g) * 0.5).to(dtype)


def choose(l, k):
    """The k largest, ties to the lowest index, NaN above all, -inf never."""
    l = l.double().numpy()
    rank = np.where(np.isnan(l), np.inf, l)
    T, E = l.shape
    ids = np.full((T, k), -1, np.int64)
    for t in range(T):
        order = sorted(range(E), key=lambda e: (not np.isnan(l[t, e]), -rank[t, e], e))
        order = [e for e in order if l[t, e] != -np.inf][:k]
        ids[t, :len(order)] = order
    return ids


def softmax64(l):
    l = l.double()
    top = l.amax(1, keepdim=True)
    x = torch.exp(l - torch.where(top == -float("inf"), torch.zeros_like(top), top))
    total = x.sum(1, keepdim=True)
    return x / torch.where(total == 0, torch.ones_like(total), total)


def forward64(l, ids, valid, renorm):
    """gates, counts, mean_prob, loss for given choices."""
    T, E = l.shape
    k = ids.shape[1]
    alive = torch.ones(T, dtype=torch.bool) if valid is None else valid != 0
    p = softmax64(l) * alive[:, None]
    here = torch.from_numpy(ids >= 0) & alive[:, None]
    at = torch.from_numpy(np.maximum(ids, 0))
    gates = p.gather(1, at) * here
    if renorm:
        total = gates.sum(1, keepdim=True)
        gates = gates / torch.where(total == 0, torch.ones_like(total), total)
    counts = torch.bincount(torch.where(here, at, E).view(-1), minlength=E + 1)[:E]
    n = max(1, int(alive.sum()))
    mean = p.sum(0) / n
    return gates, counts, int(alive.sum()), mean, E / (k * n) * (counts.double() * mean).sum()


def run_route(l, k, valid=None, renorm=True, ws=None, stream=None):
    T, E = l.shape
    i32 = dict(dtype=torch.int32, device="cuda")
    o = {"ids": torch.full((T, k), 99, **i32), "gates": torch.full((T, k), 9.0, device="cuda"),
         "counts": torch.full((E,), 99, **i32), "row_offsets": torch.full((E + 1,), 99, **i32),
         "dest": torch.full((T, k), 99, **i32), "src": torch.full((T * k,), 99, **i32),
         "n_valid": torch.full((1,), 99, **i32), "mean_prob": torch.full((E,), 9.0, device="cuda"),
         "loss": torch.full((1,), 9.0, device="cuda")}
    if ws is None:
        ws = torch.full((max(16, qfp4.moe_route_workspace_bytes(T, E, k)),), 0xA5, dtype=torch.uint8, device="cuda")
    qfp4.moe_route(l.cuda(), k, *(o[n] for n in ("ids", "gates", "counts", "row_offsets", "dest", "src", "n_valid",
                                                 "mean_prob", "loss")), ws,
                   valid=None if valid is None else valid.cuda(), renorm=renorm, stream=stream)
    torch.cuda.synchronize()
    assert qfp4.poll_device_status() == 0
    return {n: t.cpu() for n, t in o.items()}


def check_route(l, k, valid, renorm, o, finite=True):
    T, E = l.shape
    ids = choose(l, k)
    if valid is not None:
        ids[valid.numpy() == 0] = -1
    assert np.array_equal(o["ids"].numpy(), ids)
    gates, counts, n, mean, loss = forward64(l, ids, valid, renorm)
    assert torch.equal(o["counts"].long(), counts)
    offsets = np.concatenate([[0], np.cumsum(counts.numpy())])
    assert np.array_equal(o["row_offsets"].numpy(), offsets)
    assert int(o["n_valid"]) == n
    # rows: by expert, then token, then choice
    flat = ids.reshape(-1)
    order = np.argsort(np.where(flat >= 0, flat, E), kind="stable")[:offsets[-1]]
    dest = np.full(T * k, -1)
    dest[order] = np.arange(len(order))
    assert np.array_equal(o["dest"].numpy().reshape(-1), dest)
    src = np.full(T * k, -1)
    src[:len(order)] = order // k
    assert np.array_equal(o["src"].numpy(), src)
    if not finite:
        return
    # exp to 2 ulp of an argument rounded at 2^-24 of up to `span`, a sum of E
    # positive terms in a tree of at most 13 additions, a division, a product
    seen = torch.where(torch.isfinite(l.double()), l.double(), torch.zeros((), dtype=torch.float64))
    span = float((seen.amax() - seen.amin())) if l.numel() else 0.0
    rel = (span + 4 + 13 + 4) * U
    assert bool(((o["gates"].double() - gates).abs() <= 2 * rel * gates + 1e-37).all())
    # one addition per token of a warp, per warp and per range of tokens
    sums = (T / (16 * 304) + 1 + 16 + 304) * U
    assert bool(((o["mean_prob"].double() - mean).abs() <= (rel + sums) * mean + 1e-37).all())
    assert abs(float(o["loss"].double()) - float(loss)) <= (rel + sums + (E + 6) * U) * float(loss) + 1e-37


@pytest.mark.parametrize("T,E,k", [(0, 8, 2), (1, 1, 1), (1, 256, 16), (2, 2, 2), (15, 7, 3), (16, 8, 2), (17, 33, 8),
                                   (64, 8, 2), (100, 60, 4), (300, 64, 6), (511, 128, 8), (700, 200, 5), (1000, 256, 8),
                                   (9731, 16, 2)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [False, True])
def test_route(T, E, k, dtype, renorm):
    l = logits_of(T, E, T + E + k, dtype)
    check_route(l, k, None, renorm, run_route(l, k, None, renorm))
    if T:
        valid = (torch.rand(T, generator=torch.Generator().manual_seed(1)) < 0.8).to(torch.uint8) * 3
        check_route(l, k, valid, renorm, run_route(l, k, valid, renorm))


def test_no_valid_tokens():
    l = logits_of(50, 24, 1)
    o = run_route(l, 4, torch.zeros(50, dtype=torch.uint8))
    check_route(l, 4, torch.zeros(50, dtype=torch.uint8), True, o)
    assert float(o["loss"]) == 0.0 and not o["mean_prob"].any() and bool((o["ids"] == -1).all())


def test_closed_experts():
    """Rows with every expert closed, with fewer open than wanted, and with the
    lowest finite value as a mask (which stays selectable)."""
    l = logits_of(40, 20, 2)
    l[0] = -float("inf")
    l[1, 1:] = -float("inf")
    l[2, ::2] = -float("inf")
    l[3, 5:] = torch.finfo(torch.float32).min
    l[4] = torch.finfo(torch.float32).min
    l[5] = 0.0
    l[6, 3:] = -float("inf")
    for renorm in (False, True):
        o = run_route(l, 6, None, renorm)
        ids = choose(l, 6)
        gates, counts, n, mean, loss = forward64(l, ids, None, renorm)
        check_route(l, 6, None, renorm, o, finite=False)
        assert bool(((o["gates"].double() - gates).abs() <= 64 * U * gates + 1e-37).all())
        assert bool(((o["mean_prob"].double() - mean).abs() <= 400 * U * mean + 1e-37).all())


def test_ties_go_to_the_lowest_expert():
    g = torch.Generator().manual_seed(7)
    l = torch.randint(-1, 2, (400, 256), generator=g).float()
    l[:, ::3] *= -0.0                                       # zeros of either sign are equal
    for E in (5, 32, 70, 256):
        part = l[:, :E].contiguous()
        check_route(part, 5, None, True, run_route(part, 5))


def test_not_finite():
    """NaN ranks above +inf, which ranks above the rest; the token's gates and
    the statistics turn NaN, the other tokens' gates do not."""
    l = logits_of(30, 40, 3)
    l[3, 7] = float("nan")
    l[4, 9] = float("inf")
    l[4, 30] = float("nan")
    l[5, 11] = float("inf")
    o = run_route(l, 4)
    check_route(l, 4, None, True, o, finite=False)
    assert bool(o["gates"][3:6].isnan().all(1).all()) and bool(o["loss"].isnan().all())
    rest = torch.cat([o["gates"][:3], o["gates"][6:]])
    assert bool(torch.isfinite(rest).all())


def test_uniform_loss_is_one():
    T, E, k = 256, 16, 1
    l = torch.full((T, E), -40.0)
    l[torch.arange(T), torch.arange(T) % E] = 40.0
    o = run_route(l, k)
    assert abs(float(o["loss"]) - 1.0) <= 400 * U and bool((o["counts"] == T // E).all())


def test_route_repeats_and_runs_on_another_stream():
    l = logits_of(3000, 96, 4)
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    a = run_route(l, 7, ws=ws)
    b = run_route(l, 7, ws=ws, stream=None)
    side = torch.cuda.Stream()
    c = run_route(l, 7, ws=ws, stream=side)
    for n in a:
        assert torch.equal(a[n], b[n]) and torch.equal(a[n], c[n]), n


# -------------------------------------------------------------------- gradient

def gradient64(l, ids, valid, renorm, dgates, dloss):
    """The formula, and the magnitude of the terms that it adds up."""
    T, E = l.shape
    k = ids.shape[1]
    alive = (torch.ones(T, 1, dtype=torch.float64) if valid is None else (valid != 0).double()[:, None])
    p = softmax64(l)
    here = torch.from_numpy(ids >= 0).double()
    at = torch.from_numpy(np.maximum(ids, 0))
    _, counts, n, _, _ = forward64(l, ids, valid, renorm)
    n = max(1, n)
    s = (dloss * E / (k * n * n)) * counts.double()
    chosen = p.gather(1, at) * here
    dg = dgates.double() * here
    total = chosen.sum(1, keepdim=True)
    g = chosen / torch.where(total == 0, torch.ones_like(total), total) if renorm else chosen
    gd, gm = (g * dg).sum(1, keepdim=True), (g * dg.abs()).sum(1, keepdim=True)
    ps = (p * s).sum(1, keepdim=True)
    h = torch.zeros_like(p).scatter_add_(1, at, g * (dg - gd) if renorm else g * dg)
    hm = torch.zeros_like(p).scatter_add_(1, at, g * (dg.abs() + gm))
    d = h + p * (s - ps - (0 if renorm else gd))
    mag = hm + p * (s.abs() + ps.abs() + gm)
    return d * alive, mag * alive


def run_backward(l, ids, counts, n, dgates, dloss, valid, renorm, dtype):
    out = torch.full(l.shape, 9.0, dtype=dtype, device="cuda")
    qfp4.moe_route_backward(l.cuda(), ids.cuda(), counts.cuda(), n.cuda(), None if dgates is None else dgates.cuda(),
                            None if dloss is None else dloss.cuda(), out,
                            valid=None if valid is None else valid.cuda(), renorm=renorm)
    torch.cuda.synchronize()
    assert qfp4.poll_device_status() == 0
    return out.cpu()


def check_gradient(got, d, mag, dtype):
    # p to 44 half steps (see the forward check), sums of at most 24 terms
    tol = 100 * U * mag + (2.0 ** -8 * d.abs() if dtype == torch.bfloat16 else 0) + 1e-38
    err = (got.double() - d).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 16), (15, 7, 3), (64, 8, 2), (300, 64, 6), (200, 33, 4), (700, 200, 5),
                                   (1000, 256, 8)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient(T, E, k, dtype, renorm):
    g = torch.Generator().manual_seed(11)
    l = logits_of(T, E, T + E, dtype)
    valid = (torch.rand(T, generator=g) < 0.8).to(torch.uint8)
    dgates, dloss = torch.randn(T, k, generator=g), torch.rand(1, generator=g)
    for v in (None, valid):
        o = run_route(l, k, v, renorm)
        ids = o["ids"].numpy().astype(np.int64)
        for dg, dl in ((dgates, dloss), (None, dloss), (dgates, None), (None, None)):
            got = run_backward(l, o["ids"], o["counts"], o["n_valid"], dg, dl, v, renorm, dtype)
            d, mag = gradient64(l, ids, v, renorm, torch.zeros(T, k) if dg is None else dg, 0.0 if dl is None else float(dl))
            check_gradient(got, d, mag, dtype)


def test_gradient_of_closed_rows():
    l = logits_of(12, 20, 5)
    l[0] = -float("inf")
    l[1, 1:] = -float("inf")
    l[2, ::2] = -float("inf")
    for renorm in (False, True):
        o = run_route(l, 5, None, renorm)
        dg, dl = torch.randn(12, 5, generator=torch.Generator().manual_seed(2)), torch.tensor([0.5])
        got = run_backward(l, o["ids"], o["counts"], o["n_valid"], dg, dl, None, renorm, torch.float32)
        d, mag = gradient64(l, o["ids"].numpy().astype(np.int64), None, renorm, dg, 0.5)
        assert bool(torch.isfinite(got).all()) and not got[0].any()
        check_gradient(got, d, mag, torch.float32)


@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_against_differences(renorm):
    """Central differences of the 64-bit forward with the choices held fixed."""
    T, E, k, step = 6, 10, 3, 1e-5
    l = logits_of(T, E, 8)
    valid = torch.tensor([1, 1, 0, 1, 1, 1], dtype=torch.uint8)
    g = torch.Generator().manual_seed(3)
    dgates, dloss = torch.randn(T, k, generator=g), torch.tensor([0.7])
    o = run_route(l, k, valid, renorm)
    ids = o["ids"].numpy().astype(np.int64)

    def value(m):
        gates, _, _, _, loss = forward64(m, ids, valid, renorm)
        return float((gates * dgates.double()).sum() + float(dloss) * loss)

    d = torch.zeros(T, E, dtype=torch.float64)
    for t in range(T):
        for e in range(E):
            hi, lo = l.double().clone(), l.double().clone()
            hi[t, e] += step
            lo[t, e] -= step
            d[t, e] = (value(hi) - value(lo)) / (2 * step)
    got = run_backward(l, o["ids"], o["counts"], o["n_valid"], dgates, dloss, valid, renorm, torch.float32)
    # differences: 1e-10 of the third derivative, 1e-16 / step of the value; the kernel: 100 half steps of terms below 4
    assert float((got.double() - d).abs().max()) <= 1e-9 + 4 * 100 * U


def test_route_and_gradient_in_a_graph():
    T, E, k = 500, 64, 6
    l = logits_of(T, E, 1).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    ids, dest = torch.empty(T, k, **i32), torch.empty(T, k, **i32)
    gates, mean, loss = torch.empty(T, k, device="cuda"), torch.empty(E, device="cuda"), torch.empty(1, device="cuda")
    counts, offs, src, n = torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(T * k, **i32), torch.empty(1, **i32)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    dg, dl, out = torch.randn(T, k, device="cuda"), torch.rand(1, device="cuda"), torch.empty(T, E, device="cuda")

    def step():
        qfp4.moe_route(l, k, ids, gates, counts, offs, dest, src, n, mean, loss, ws)
        qfp4.moe_route_backward(l, ids, counts, n, dg, dl, out)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (2, 3):
        l.copy_(logits_of(T, E, seed))
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (ids, gates, counts, offs, dest, src, mean, loss, out)]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (ids, gates, counts, offs, dest, src, mean, loss, out)))
