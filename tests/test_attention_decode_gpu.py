"""Attention of one new token over the paged cache against softmax(q K^T) V in 64
bits over the cache's own values.

Bounds, with x_j the logits, p_j = exp(x_j - max x), S = sum p_j, T the largest
sum |scale q_k k_jk| of a logit's terms:
  lse  an fp32 sum of D terms in the tensor cores, 16 steps of at most 2^-22 of
       the terms each: 2^-18 T; the logarithm and its product with ln 2: 2^-20 + 2^-22 |lse|
  o    half a step of BF16, 2^-8 |o|; the same error of each logit, twice over
       (weights and their sum), and the rounding of each weight to FP16, 2^-11:
       (2^-11 + 2^-17 (1 + T)) sum p|v| / S; weights below 2^-14 of the largest
       lose 2^-25 of it: n 2^-25 max(p max|v|) / S"""
import math

import pytest
import torch

from block_scaled_fp4_tcgen05_gb300 import qfp4
from tests import _cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qfp4.load()
    assert qfp4.device_check() == 0


class Case:
    """A cache with garbage wherever no sequence has a token, filled by the library's write."""

    def __init__(self, type, lens, H, KV, D, page_size, seed=0, spread=1.0, max_pages=None, garbage=0xFF):
        g = self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.type, self.lens, self.H, self.KV, self.D, self.page_size = type, lens, H, KV, D, page_size
        each = [-(-n // page_size) for n in lens]
        pages = max(1, sum(each)) + 2
        order = torch.randperm(pages, generator=g, device="cuda").int()
        self.table = torch.full((len(lens), max_pages or max(1, max(each))), -7, dtype=torch.int32, device="cuda")      # entries of no token are not read
        at = 0
        for i, n in enumerate(each):
            self.table[i, :n] = order[at: at + n]
            at += n
        self.gs = [torch.tensor([v], device="cuda") if type == qfp4.CACHE_NVFP4 else None for v in (0.009, 0.0041)]
        self.cache = _cache.empty(type, pages, KV, D, page_size, garbage)
        self.k, self.v = [], []
        for i, n in enumerate(lens):
            k = torch.randn(n, KV, D, generator=g, device="cuda") * (1 + 4 * (torch.rand(KV, D, generator=g, device="cuda") < 0.05))
            v = torch.randn(n, KV, D, generator=g, device="cuda") * torch.exp(spread * torch.randn(n, KV, 1, generator=g, device="cuda"))
            self.put(i, k.bfloat16(), v.bfloat16())
        self.q = torch.randn(len(lens), H, D, generator=g, device="cuda").bfloat16()
        self.scale = 1 / math.sqrt(D)
        self.ws = torch.zeros(qfp4.attention_decode_workspace_bytes(len(lens), H, KV, D), dtype=torch.uint8, device="cuda")

    def slots(self, i):
        n = torch.arange(self.lens[i], device="cuda")
        return (self.table[i].long()[n // self.page_size] * self.page_size + n % self.page_size).int()

    def put(self, i, k, v):
        if self.lens[i]:
            qfp4.kv_cache_write(self.type, k, v, self.slots(i), self.cache, self.page_size, *self.gs)
        self.k.append(_cache.encode(self.type, k.float(), self.gs[0])[2].double() if self.lens[i] else k.double())
        self.v.append(_cache.encode(self.type, v.float(), self.gs[1])[2].double() if self.lens[i] else v.double())

    def run(self, window=0, lengths=None, q=None):
        B = len(self.lens)
        o = torch.full((B, self.H, self.D), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((B, self.H), 7.0, device="cuda")
        lengths = torch.tensor(self.lens, dtype=torch.int32, device="cuda") if lengths is None else lengths
        qfp4.attention_decode(self.type, self.q if q is None else q, self.cache, self.page_size, self.table, lengths, self.scale, o, self.ws, *self.gs,
                              lse=lse, window=window)
        return o, lse

    def want(self, window=0):
        """(o, lse, bounds of both)"""
        B, G = len(self.lens), self.H // self.KV
        o, lse = torch.zeros(B, self.H, self.D, dtype=torch.float64, device="cuda"), torch.full((B, self.H), -math.inf, dtype=torch.float64, device="cuda")
        bo, bl = torch.zeros_like(o), torch.zeros_like(lse)
        for i, n in enumerate(self.lens):
            if n == 0:
                continue
            lo = max(0, n - window) if window else 0
            k, v = self.k[i][lo:], self.v[i][lo:]
            q = self.q[i].double().view(self.KV, G, self.D)
            x = torch.einsum("hgd,nhd->hgn", q, k) * self.scale
            T = (torch.einsum("hgd,nhd->hgn", q.abs(), k.abs()) * self.scale).amax(-1, keepdim=True)
            p = torch.exp(x - x.amax(-1, keepdim=True))
            S = p.sum(-1, keepdim=True)
            out = torch.einsum("hgn,nhd->hgd", p, v) / S
            size = torch.einsum("hgn,nhd->hgd", p, v.abs()) / S
            small = (p * v.abs().amax(-1).t()[:, None]).amax(-1, keepdim=True) / S * (n - lo) * 2.0 ** -25
            o[i] = out.reshape(self.H, self.D)
            bo[i] = (2.0 ** -8 * out.abs() + (2.0 ** -11 + 2.0 ** -17 * (1 + T)) * size + small).reshape(self.H, self.D)
            lse[i] = torch.logsumexp(x, -1).flatten()
            bl[i] = (2.0 ** -18 * T[..., 0] + 2.0 ** -20).flatten() + 2.0 ** -22 * lse[i].abs()
        return o, lse, bo, bl

    def check(self, window=0):
        got, glse = self.run(window)
        o, lse, bo, bl = self.want(window)
        assert qfp4.poll_device_status() == 0
        full = torch.tensor([n > 0 for n in self.lens], device="cuda")
        assert ((got.double() - o).abs() <= bo).all(), float(((got.double() - o).abs() / bo.clamp(min=1e-30)).max())
        assert ((glse.double() - lse)[full].abs() <= bl[full]).all() and (glse[~full] == -math.inf).all()
        assert not self.ws[:4096].any()
        return got, glse


LENS = [  # lengths of the sequences
    [1], [16], [17], [15, 0, 33], [64, 128, 256], [0], [0, 0, 5, 0], [127, 129, 1, 500], [2000], [31] * 40, list(range(0, 70, 3)),
]


@pytest.mark.parametrize("lens", LENS, ids=lambda v: "-".join(map(str, v[:4])))
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("type", _cache.TYPES)
def test_lengths(type, D, lens):
    Case(type, lens, 8, 2, D, 16, seed=len(lens)).check()


@pytest.mark.parametrize("H,KV", [(1, 1), (2, 2), (7, 1), (8, 1), (9, 1), (16, 1), (17, 1), (40, 1), (64, 4), (12, 4), (30, 2), (96, 3), (33, 11)])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("type", _cache.TYPES)
def test_heads(type, D, H, KV):
    Case(type, [75, 300], H, KV, D, 32, seed=H).check()


@pytest.mark.parametrize("page_size", [16, 48, 64, 128, 400])
@pytest.mark.parametrize("type", _cache.TYPES)
def test_pages(type, page_size):
    Case(type, [401, 3, 399, 1000], 16, 4, 128, page_size, seed=page_size).check()


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 399, 5000])
@pytest.mark.parametrize("type", _cache.TYPES)
def test_window(type, window):
    Case(type, [401, 0, 7, 16, 1000], 8, 4, 128, 16, seed=window).check(window)


@pytest.mark.parametrize("type", _cache.TYPES)
def test_many_sequences(type):
    """More sequences than a CTA has threads, more tiles than the grid has CTAs."""
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 900, (300,), generator=g).tolist()
    Case(type, lens, 8, 2, 64, 16, seed=4).check()


@pytest.mark.parametrize("KV,window", [(1, 0), (2, 9)])
def test_thousands_of_sequences(KV, window):
    """Many sequences for each thread that looks for a CTA's first tile, long runs of empty ones among them."""
    g = torch.Generator().manual_seed(KV)
    lens = torch.randint(0, 40, (1501,), generator=g)
    lens[100:700] = 0
    lens[-3:] = torch.tensor([700, 0, 333])
    Case(qfp4.CACHE_E4M3, lens.tolist(), 4, KV, 64, 16, seed=KV).check(window)


@pytest.mark.parametrize("type", _cache.TYPES)
def test_long(type):
    """Few sequences, each split over many CTAs."""
    Case(type, [33000, 5, 20011], 16, 2, 128, 64, seed=5).check()


@pytest.mark.parametrize("H,KV,D,lens", [(8, 1, 128, [131072]), (16, 1, 128, [50000, 3, 0, 70001]), (3, 1, 256, [60000, 20000]), (8, 2, 64, [40000, 40000, 17]),
                                         (12, 1, 64, [1] * 700 + [30000, 9000])])
@pytest.mark.parametrize("type", _cache.TYPES)
def test_many_pieces(type, H, KV, D, lens):
    """Heads that hundreds of CTAs share, whose pieces are joined in groups; the same bits every time, and every counter at zero again."""
    c = Case(type, lens, H, KV, D, 16, seed=len(lens) + H)
    o, lse = c.check()
    for _ in range(3):
        o2, lse2 = c.run()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert not c.ws[:16384].any()


@pytest.mark.parametrize("garbage", [0x00, 0x7F, 0x7E, 0xFF])
@pytest.mark.parametrize("type", _cache.TYPES)
def test_what_lies_beyond_the_length_does_not_count(type, garbage):
    """Bytes that are NaN, infinities or huge in every type, beyond the last token and before the window."""
    c = Case(type, [5, 21, 130], 4, 1, 128, 16, seed=6, garbage=garbage)
    c.check()
    d = Case(type, [5, 21, 130], 4, 1, 128, 16, seed=6, garbage=garbage)
    bad = torch.full((1, 1, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    for i, n in enumerate(d.lens):       # the first tokens, out of the window
        qfp4.kv_cache_write(type, bad, bad, d.slots(i)[:1], d.cache, 16, *d.gs)
    d.check(window=4)


@pytest.mark.parametrize("type", _cache.TYPES)
def test_extreme_logits_and_scales(type):
    """Logits from -10^4 to 10^4, values of very different size."""
    c = Case(type, [700], 8, 2, 64, 16, seed=7, spread=4.0)
    c.q = (c.q.float() * torch.tensor([1e-4, 1.0, 1e2, 1e4, 1e-30, 1e30, 0.0, 3.0], device="cuda")[None, :, None]).bfloat16()
    c.scale = 1.0
    got, lse = c.run()
    o, want_lse, bo, bl = c.want()
    for h in (0, 1, 4, 6, 7):
        assert ((got[:, h].double() - o[:, h]).abs() <= bo[:, h]).all(), h
        assert ((lse[:, h].double() - want_lse[:, h]).abs() <= bl[:, h]).all(), h
    # one token has all the weight, or the bound on the logits says nothing
    assert torch.isfinite(got).all() and torch.isfinite(lse[:, :5]).all()


@pytest.mark.parametrize("type", _cache.TYPES)
def test_nan_query_gives_nan(type):
    c = Case(type, [40, 40], 4, 2, 128, 16, seed=8)
    c.q[0, 1, 3] = float("nan")
    got, lse = c.run()
    o, want_lse, bo, bl = c.want()
    assert torch.isnan(got[0, 1]).all() and torch.isnan(lse[0, 1])
    keep = [0, 2, 3, 4, 5, 6, 7]
    assert ((got.double() - o).abs() <= bo).flatten(0, 1)[keep].all()


def test_nan_key_gives_nan():
    c = Case(qfp4.CACHE_BF16, [40], 2, 1, 64, 16, seed=9)
    bad = torch.full((1, 1, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    qfp4.kv_cache_write(c.type, bad, bad, c.slots(0)[20:21], c.cache, 16)
    got, lse = c.run()
    assert torch.isnan(got).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("type", _cache.TYPES)
def test_same_page_for_several_sequences(type):
    """A shared prefix: two sequences' tables name the same pages."""
    c = Case(type, [64, 64], 4, 2, 64, 16, seed=10)
    c.table[1] = c.table[0]
    c.k[1], c.v[1] = c.k[0], c.v[0]
    c.check()


def test_pages_and_lengths_out_of_range_report():
    c = Case(qfp4.CACHE_E4M3, [40, 40, 40], 4, 2, 64, 16, seed=11)
    good, _ = c.run()
    for bad in (c.cache.shape[0], -1, 2 ** 31 - 1):
        keep = c.table[1, 0].clone()
        c.table[1, 0] = bad
        got, _ = c.run()
        assert qfp4.poll_device_status() == -1 and qfp4.poll_device_status() == 0
        assert torch.equal(got[0], good[0]) and torch.equal(got[2], good[2])
        c.table[1, 0] = keep
    for bad, n in ((-3, 0), (49, 48), (2 ** 31 - 1, 48)):     # three pages of 16 each
        got, lse = c.run(lengths=torch.tensor([40, bad, 40], dtype=torch.int32, device="cuda"))
        assert qfp4.poll_device_status() == -1
        assert torch.equal(got[0], good[0]) and torch.equal(got[2], good[2])
        if n == 0:
            assert (got[1] == 0).all() and (lse[1] == -math.inf).all()
    c.check()


@pytest.mark.parametrize("type", _cache.TYPES)
def test_repeats_and_workspace_of_other_shapes(type):
    """The same workspace for calls of different shapes, one after the other; the same bits every time."""
    a, b = Case(type, [5000, 3, 700], 16, 2, 128, 16, seed=12), Case(type, [900] * 5, 4, 4, 64, 32, seed=13)
    need = max(a.ws.numel(), b.ws.numel())
    a.ws = b.ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    first, second = a.run(), b.run()
    for _ in range(5):
        for c, (o, lse) in ((a, first), (b, second)):
            o2, lse2 = c.run()
            assert torch.equal(o, o2) and torch.equal(lse, lse2)
    a.check(), b.check()


def test_graph_with_growing_lengths_and_streams():
    """A captured step whose lengths grow from replay to replay, and calls side by side on two streams."""
    c = Case(qfp4.CACHE_NVFP4, [300, 40], 8, 2, 128, 16, seed=14)
    lengths = torch.tensor([1, 1], dtype=torch.int32, device="cuda")
    o, lse = torch.empty(2, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 8, device="cuda")
    args = (c.type, c.q, c.cache, c.page_size, c.table, lengths, c.scale, o, c.ws, *c.gs)
    qfp4.attention_decode(*args, lse=lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qfp4.attention_decode(*args, lse=lse)
    full, (k, v) = c.lens, (c.k, c.v)
    for n in ([7, 0], [299, 33], [300, 40]):
        lengths.copy_(torch.tensor(n, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        c.lens, c.k, c.v = n, [a[:m] for a, m in zip(k, n)], [a[:m] for a, m in zip(v, n)]
        want, _, bo, _ = c.want()
        assert ((o.double() - want).abs() <= bo).all(), n
    c.lens, c.k, c.v = full, k, v
    d = Case(qfp4.CACHE_NVFP4, [3000, 4000], 8, 2, 128, 16, seed=15)
    one, two = c.run(), d.run()
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(20):
        for s, x in zip(streams, (c, d)):
            with torch.cuda.stream(s):
                got.append((x, x.run(lengths=None)))
    torch.cuda.synchronize()
    for x, (o1, l1) in got:
        assert torch.equal(o1, (one if x is c else two)[0]) and torch.equal(l1, (one if x is c else two)[1])


@pytest.mark.parametrize("type", _cache.TYPES)
def test_queries_in_a_projection(type):
    """Rows of queries that lie apart; no lse."""
    c = Case(type, [90, 5], 4, 2, 128, 16, seed=16)
    want, _ = c.run()
    wide = torch.full((2, 8, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :4] = c.q
    o = torch.empty_like(want)
    qfp4.attention_decode(type, wide[:, :4], c.cache, 16, c.table, torch.tensor(c.lens, dtype=torch.int32, device="cuda"), c.scale, o, c.ws, *c.gs)
    assert torch.equal(o, want)


def test_offsets_beyond_32_bits():
    """Pages whose bytes lie beyond 2^32 of the cache."""
    type, KV, D, page_size = qfp4.CACHE_BF16, 8, 128, 64
    page = qfp4.kv_cache_page_bytes(type, KV, D, page_size)
    pages = (5 << 30) // page
    c = Case(type, [130], 16, KV, D, page_size, seed=17)
    small, c.cache = c.cache, torch.zeros(pages, KV, page // KV, dtype=torch.uint8, device="cuda")
    for i in range(3):
        c.cache[pages - 1 - i] = small[c.table[0, i]]
        c.table[0, i] = pages - 1 - i
    c.check()
