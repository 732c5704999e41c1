"""Norms of query and key heads with the position rotation, and the gradient,
against the formulas in 64 bits.

Bounds.  Forward: one rounding to BF16 (half a step, 2^-8) and about 16 roundings
of fp32 on each of a pair's two terms: 2^-20 (|z_a| + |z_b|).  Gradient: the
roundings of the turned gradient, of the root (twice) and of the mean, 64 in all:
2^-18 of the terms' magnitudes.  Weight gradients: a sum of n terms in fp32, in
chains of at most L: (L + 64) 2^-24 sum |dz h|, L = terms per group of lanes + 16."""
import pytest
import torch

from block_scaled_fp4_tcgen05_gb300 import qfp4

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qfp4.load()
    assert qfp4.device_check() == 0


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def table(rows, r, g):
    a = torch.rand(rows, r // 2, generator=g, device="cuda", dtype=torch.float64) * 6.28
    return torch.cat([a.cos(), a.sin()], 1).float()


def inputs(T, H, KV, D, R, norm, seed, extra=0):
    g = generator(seed)
    s = {"qkv": (torch.randn(T, (H + 2 * KV) * D + extra, generator=g, device="cuda") * torch.exp(2 * torch.randn(T, 1, generator=g, device="cuda"))).bfloat16(),
         "table": table(50, R, g) if R else None,
         "pos": torch.randint(0, 50, (T,), generator=g, device="cuda", dtype=torch.int32) if R else None}
    for n in "qk":
        s[n + "w"] = (1 + 0.3 * torch.randn(D, generator=g, device="cuda")).bfloat16() if norm else None
    s["dq"] = torch.randn(T, H, D, generator=g, device="cuda").bfloat16()
    s["dk"] = torch.randn(T, KV, D, generator=g, device="cuda").bfloat16()
    return s


def pair(x, R, inter):
    """The other element of each pair and the sign of its sine."""
    y, sign = torch.zeros_like(x), torch.zeros(x.shape[-1], device=x.device, dtype=torch.float64)
    if inter:
        y[..., 0:R:2], y[..., 1:R:2] = x[..., 1:R:2], x[..., 0:R:2]
        sign[0:R:2], sign[1:R:2] = -1, 1
    else:
        y[..., : R // 2], y[..., R // 2: R] = x[..., R // 2: R], x[..., : R // 2]
        sign[: R // 2], sign[R // 2: R] = -1, 1
    return y, sign


def angles(s, D, R, inter):
    T = s["qkv"].shape[0]
    c, n = torch.ones(T, 1, D, dtype=torch.float64, device="cuda"), torch.zeros(T, 1, D, dtype=torch.float64, device="cuda")
    if R:
        rows = s["table"].double()[s["pos"].clamp(0, 49).long()][:, None]
        cos, sin = rows[..., : R // 2], rows[..., R // 2:]
        c[..., :R] = cos.repeat_interleave(2, -1) if inter else torch.cat([cos, cos], -1)
        n[..., :R] = sin.repeat_interleave(2, -1) if inter else torch.cat([sin, sin], -1)
    return c, n


def forward64(s, H, KV, D, R, inter):
    T = s["qkv"].shape[0]
    x = s["qkv"][:, : (H + KV) * D].reshape(T, H + KV, D).double()
    if s["qw"] is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
        x = x * torch.cat([s["qw"].double().expand(H, D), s["kw"].double().expand(KV, D)])
    c, n = angles(s, D, R, inter)
    o, sign = pair(x, R, inter)
    return x * c + o * n * sign, x.abs() + o.abs()


SHAPES = [  # T, H, KV, D, R
    (1, 1, 1, 64, 64), (3, 5, 1, 64, 32), (7, 9, 9, 128, 128), (64, 32, 8, 128, 128), (33, 3, 2, 96, 96), (9, 7, 1, 80, 16), (5, 4, 2, 192, 64),
    (17, 6, 2, 256, 256), (2, 16, 1, 256, 240), (40, 2, 1, 16, 16), (11, 9, 3, 112, 112), (6, 4, 4, 128, 0), (300, 12, 4, 48, 32),
]


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("T,H,KV,D,R", SHAPES)
def test_forward(T, H, KV, D, R, norm, inter):
    s = inputs(T, H, KV, D, R, norm, T + D, extra=8)
    q, k = (torch.full((T, n, D), 7.0, dtype=torch.bfloat16, device="cuda") for n in (H, KV))
    qfp4.qk_norm_rope(s["qkv"], H, KV, q, k, s["qw"], s["kw"], s["table"], s["pos"], eps=EPS, interleaved=inter)
    want, size = forward64(s, H, KV, D, R, inter)
    got = torch.cat([q, k], 1).double()
    bound = 2.0 ** -8 * want.abs() + 2.0 ** -20 * size * (1 if norm else 1) + 2.0 ** -134
    assert ((got - want).abs() <= bound).all(), float(((got - want).abs() / bound).max())
    assert qfp4.poll_device_status() == 0


def test_forward_in_place_and_strided():
    T, H, KV, D = 37, 8, 2, 128
    s = inputs(T, H, KV, D, D, True, 5)
    q, k = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda"), torch.empty(T, KV, D, dtype=torch.bfloat16, device="cuda")
    args = (s["qw"], s["kw"], s["table"], s["pos"])
    qfp4.qk_norm_rope(s["qkv"], H, KV, q, k, *args, eps=EPS)
    same = s["qkv"].clone()
    heads = same.view(T, -1, D)
    qfp4.qk_norm_rope(same, H, KV, heads[:, :H], heads[:, H: H + KV], *args, eps=EPS)
    assert torch.equal(heads[:, :H], q) and torch.equal(heads[:, H: H + KV], k)
    assert torch.equal(heads[:, H + KV:], s["qkv"].view(T, -1, D)[:, H + KV:])
    wide = torch.full((T, (H + 2 * KV) * D + 64), 3.0, dtype=torch.bfloat16, device="cuda")
    wide[:, : same.shape[1]] = s["qkv"]
    qfp4.qk_norm_rope(wide[:, : same.shape[1]], H, KV, same.view(T, -1, D)[:, :H], same.view(T, -1, D)[:, H: H + KV], *args, eps=EPS)
    assert torch.equal(heads[:, :H], q) and torch.equal(heads[:, H: H + KV], k)


def test_rows_without_position_stay_and_far_ones_report():
    T, H, KV, D = 20, 4, 2, 64
    s = inputs(T, H, KV, D, D, True, 6)
    s["pos"][3] = -1
    s["pos"][19] = -5
    q, k = torch.full((T, H, D), 9.0, dtype=torch.bfloat16, device="cuda"), torch.full((T, KV, D), 9.0, dtype=torch.bfloat16, device="cuda")
    qfp4.qk_norm_rope(s["qkv"], H, KV, q, k, s["qw"], s["kw"], s["table"], s["pos"], eps=EPS)
    for t in (3, 19):
        assert (q[t] == 9).all() and (k[t] == 9).all()
    assert not (q[4] == 9).any() and qfp4.poll_device_status() == 0
    s["pos"][4] = 50                # the table has rows 0..49
    q.fill_(9.0)
    qfp4.qk_norm_rope(s["qkv"], H, KV, q, k, s["qw"], s["kw"], s["table"], s["pos"], eps=EPS)
    assert qfp4.poll_device_status() == -1 and qfp4.poll_device_status() == 0
    assert (q[4] == 9).all() and not (q[5] == 9).any()


def test_infinities_pass_where_nothing_turns():
    s = inputs(2, 2, 1, 64, 16, False, 7)
    s["qkv"][0, 40] = float("inf")
    s["qkv"][1, 63] = float("-inf")
    q, k = torch.empty(2, 2, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 1, 64, dtype=torch.bfloat16, device="cuda")
    qfp4.qk_norm_rope(s["qkv"], 2, 1, q, k, None, None, s["table"], s["pos"])
    assert torch.equal(q[..., 16:], s["qkv"].view(2, -1, 64)[:, :2, 16:]) and torch.isfinite(q[..., :16]).all()


def backward64(s, H, KV, D, R, inter, dq, dk, alive):
    T = s["qkv"].shape[0]
    dy = torch.cat([dq, dk], 1).double() * alive
    c, n = angles(s, D, R, inter)
    o, sign = pair(dy, R, inter)
    dz = dy * c - o * n * sign
    big = (dy * c).abs() + (o * n * sign).abs()
    if s["qw"] is None:
        return dz, big, None, None, None, None
    x = s["qkv"][:, : (H + KV) * D].reshape(T, H + KV, D).double()
    w = torch.cat([s["qw"].double().expand(H, D), s["kw"].double().expand(KV, D)])
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    h = x * r
    dx = r * (dz * w - h * (dz * w * h).mean(-1, keepdim=True))
    size = r * (big * w.abs() + h.abs() * (big * w.abs() * h.abs()).mean(-1, keepdim=True))
    each, mag = dz * h, big * h.abs()
    return dx, size, each[:, :H].sum((0, 1)), each[:, H:].sum((0, 1)), mag[:, :H].sum((0, 1)), mag[:, H:].sum((0, 1))


def check_backward(s, T, H, KV, D, R, inter, alive=1.0, dqkv=None):
    norm = s["qw"] is not None
    dqkv = torch.full_like(s["qkv"], 5.0) if dqkv is None else dqkv
    dqw, dkw = (torch.full((D,), 3.0, device="cuda") if norm else None for _ in range(2))
    ws = torch.empty(qfp4.qk_norm_rope_backward_workspace_bytes(T, H, KV, D), dtype=torch.uint8, device="cuda").fill_(0xFF)
    qfp4.qk_norm_rope_backward(s["qkv"], H, KV, s["dq"], s["dk"], dqkv, dqw, dkw, ws, s["qw"], s["kw"], s["table"], s["pos"], eps=EPS, interleaved=inter)
    dx, size, a, b, ma, mb = backward64(s, H, KV, D, R, inter, s["dq"], s["dk"], alive)
    got = dqkv[:, : (H + KV) * D].reshape(T, H + KV, D).double()
    bound = 2.0 ** -8 * dx.abs() + 2.0 ** -18 * size + 2.0 ** -134
    assert ((got - dx).abs() <= bound).all(), float(((got - dx).abs() / bound).max())
    if norm:
        chain = -(-T * (H + KV + 16) // 8) + 16 + 64        # at least a warp's groups share the terms, eight warps a CTA
        for g, w, m in ((dqw, a, ma), (dkw, b, mb)):
            assert ((g.double() - w).abs() <= chain * 2.0 ** -24 * m + 1e-30).all()
    assert qfp4.poll_device_status() == 0
    return dqkv, dqw, dkw


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("T,H,KV,D,R", SHAPES)
def test_backward(T, H, KV, D, R, norm, inter):
    s = inputs(T, H, KV, D, R, norm, T + D + 1)
    dqkv, *_ = check_backward(s, T, H, KV, D, R, inter)
    assert (dqkv[:, (H + KV) * D:] == 5).all()       # the value heads' places


def test_backward_more_items_than_the_grid_holds():
    T, H, KV, D = 3001, 12, 4, 64
    s = inputs(T, H, KV, D, D, True, 8)
    _, a, b = check_backward(s, T, H, KV, D, D, False)
    _, a2, b2 = check_backward(s, T, H, KV, D, D, False)
    assert torch.equal(a, a2) and torch.equal(b, b2)


def test_backward_padding_gets_zeros():
    T, H, KV, D = 21, 4, 1, 128
    s = inputs(T, H, KV, D, D, True, 9)
    s["pos"][::4] = -1
    s["dq"][::4] = float("nan")     # what lies in rows of no sequence does not count
    s["qkv"][::4] = float("inf")
    clean = dict(s, dq=torch.nan_to_num(s["dq"]), qkv=torch.where(torch.isinf(s["qkv"]), torch.ones_like(s["qkv"]), s["qkv"]))
    alive = (s["pos"] >= 0).double()[:, None, None]
    dqkv = torch.full_like(s["qkv"], 5.0)
    dqw, dkw = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    qfp4.qk_norm_rope_backward(s["qkv"], H, KV, s["dq"], s["dk"], dqkv, dqw, dkw, ws, s["qw"], s["kw"], s["table"], s["pos"], eps=EPS)
    want, wq, wk = check_backward(clean, T, H, KV, D, D, False, alive)
    assert torch.equal(dqkv, want) and torch.equal(dqw, wq) and torch.equal(dkw, wk)
    assert (dqkv[::4, : (H + KV) * D] == 0).all()


def test_backward_in_place():
    """The gradient in the input's place, and the heads' gradients in its own."""
    T, H, KV, D = 19, 4, 2, 128
    s = inputs(T, H, KV, D, D, True, 10)
    want, wq, wk = check_backward(s, T, H, KV, D, D, True)
    check_backward(dict(s, qkv=s["qkv"].clone()), T, H, KV, D, D, True)
    buf = s["qkv"].clone()
    dq, dk, ws = torch.empty(D, device="cuda"), torch.empty(D, device="cuda"), torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    qfp4.qk_norm_rope_backward(buf, H, KV, s["dq"], s["dk"], buf, dq, dk, ws, s["qw"], s["kw"], s["table"], s["pos"], eps=EPS, interleaved=True)
    assert torch.equal(buf[:, : (H + KV) * D], want[:, : (H + KV) * D]) and torch.equal(dq, wq)
    buf = torch.zeros_like(s["qkv"])
    heads = buf.view(T, -1, D)
    heads[:, :H], heads[:, H: H + KV] = s["dq"], s["dk"]
    qfp4.qk_norm_rope_backward(s["qkv"], H, KV, heads[:, :H], heads[:, H: H + KV], buf, dq, dk, ws, s["qw"], s["kw"], s["table"], s["pos"], eps=EPS,
                               interleaved=True)
    assert torch.equal(buf[:, : (H + KV) * D], want[:, : (H + KV) * D]) and torch.equal(dk, wk)


def test_backward_without_tokens_is_zero():
    D = 64
    dq, dk = torch.ones(D, device="cuda"), torch.ones(D, device="cuda")
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    none = torch.empty(0, 4 * D, dtype=torch.bfloat16, device="cuda")
    qfp4.qk_norm_rope_backward(none, 2, 1, none.view(0, 4, D)[:, :2], none.view(0, 4, D)[:, :1], none, dq, dk, torch.empty(16, dtype=torch.uint8, device="cuda"), w, w)
    assert (dq == 0).all() and (dk == 0).all()


def test_gradient_against_differences():
    """sum(dy y) by central differences in 64 bits along random directions of x and of the weights."""
    T, H, KV, D, R = 3, 2, 1, 64, 32
    s = inputs(T, H, KV, D, R, True, 11)
    dqkv, dqw, dkw = check_backward(s, T, H, KV, D, R, False)
    g = generator(12)
    dy = torch.cat([s["dq"], s["dk"]], 1).double()

    def value(x, qw, kw):
        return (forward64(dict(s, qkv=x, qw=qw, kw=kw), H, KV, D, R, False)[0] * dy).sum()

    x, qw, kw = s["qkv"].double(), s["qw"].double(), s["kw"].double()
    for _ in range(4):
        vx, vq, vk = (torch.randn(v.shape, generator=g, device="cuda", dtype=torch.float64) * 1e-5 for v in (x, qw, kw))
        vx[:, (H + KV) * D:] = 0
        by_difference = (value(x + vx, qw + vq, kw + vk) - value(x - vx, qw - vq, kw - vk)) / 2
        terms = torch.cat([(dqkv.double() * vx)[:, : (H + KV) * D].flatten(), dqw.double() * vq, dkw.double() * vk])
        # each BF16 gradient is off by 2^-8 of itself at most; the differences' own error is third order
        assert abs(by_difference - terms.sum()) <= 2.0 ** -7.5 * terms.abs().sum()


def test_graph_and_stream():
    T, H, KV, D = 50, 8, 2, 128
    s = inputs(T, H, KV, D, D, True, 13)
    want, wq, wk = check_backward(s, T, H, KV, D, D, False)
    q, k = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda"), torch.empty(T, KV, D, dtype=torch.bfloat16, device="cuda")
    dqkv, dq, dk, ws = torch.zeros_like(s["qkv"]), torch.empty(D, device="cuda"), torch.empty(D, device="cuda"), torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qfp4.qk_norm_rope(s["qkv"], H, KV, q, k, s["qw"], s["kw"], s["table"], s["pos"], eps=EPS)
        qfp4.qk_norm_rope_backward(s["qkv"], H, KV, s["dq"], s["dk"], dqkv, dq, dk, ws, s["qw"], s["kw"], s["table"], s["pos"], eps=EPS)
    for _ in range(3):
        q.zero_(), dqkv.zero_(), dq.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dqkv[:, : (H + KV) * D], want[:, : (H + KV) * D]) and torch.equal(dq, wq) and torch.equal(dk, wk)
        want_y, size = forward64(s, H, KV, D, D, False)
        assert ((torch.cat([q, k], 1).double() - want_y).abs() <= 2.0 ** -8 * want_y.abs() + 2.0 ** -20 * size).all()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        q2 = torch.empty_like(q)
        qfp4.qk_norm_rope(s["qkv"], H, KV, q2, k, s["qw"], s["kw"], s["table"], s["pos"], eps=EPS)
    side.synchronize()
    assert torch.equal(q2, q)


def test_offsets_beyond_32_bits():
    """Rows far apart: the last row of a view whose offsets pass 2^31 elements."""
    T, H, KV, D = 3, 1, 1, 64
    ld = 1 << 30
    flat = torch.zeros(2 * ld + 3 * D, dtype=torch.bfloat16, device="cuda")
    qkv = flat.as_strided((T, 3 * D), (ld, 1))
    s = inputs(T, H, KV, D, D, True, 14)
    qkv.copy_(s["qkv"])
    q, k = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda"), torch.empty(T, KV, D, dtype=torch.bfloat16, device="cuda")
    qfp4.qk_norm_rope(qkv, H, KV, q, k, s["qw"], s["kw"], s["table"], s["pos"], eps=EPS)
    want, size = forward64(s, H, KV, D, D, False)
    assert ((torch.cat([q, k], 1).double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20 * size).all()
