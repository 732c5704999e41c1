"""The paged cache: written bytes against the stated rules and layout bit for bit,
what is read back, and the writes behind norm and rotation."""
import pytest
import torch

from block_scaled_fp4_tcgen05_gb300 import qfp4
from tests import _cache
from tests.test_head_norm_rope_gpu import EPS, forward64, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qfp4.load()
    assert qfp4.device_check() == 0


def vectors(g, T, H, D):
    """Rows of very different size, zeros, equal magnitudes and lone elements among them."""
    x = torch.randn(T, H, D, generator=g, device="cuda") * torch.exp(3 * torch.randn(T, H, 1, generator=g, device="cuda"))
    x[::7] = 0
    x[1::7, :, : D // 2] = 0
    x[2::7] = x[2::7].sign()
    return x.bfloat16()


def scales(type):
    return [torch.tensor([v], device="cuda") if type == qfp4.CACHE_NVFP4 else None for v in (0.013, 0.0071)]


def slots_of(g, T, pages, page_size):
    return torch.randperm(pages * page_size, generator=g, device="cuda")[:T].int()


@pytest.mark.parametrize("page_size", [16, 48, 128])
@pytest.mark.parametrize("H,D", [(1, 64), (8, 64), (3, 128), (8, 128), (2, 256), (5, 256)])
@pytest.mark.parametrize("type", _cache.TYPES)
def test_write_and_read(type, H, D, page_size):
    g = torch.Generator(device="cuda").manual_seed(D + H)
    T, pages = 41, 5
    k, v = vectors(g, T, H, D), vectors(g, T, H, D)
    gs = scales(type)
    slots = slots_of(g, T, pages, page_size)
    want, got = (_cache.empty(type, pages, H, D, page_size, 0xA5) for _ in range(2))
    kv, vv = _cache.put(type, want, page_size, slots, k.float(), v.float(), *gs)
    qfp4.kv_cache_write(type, k, v, slots, got, page_size, *gs)
    assert torch.equal(got, want)
    ko, vo = (torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qfp4.kv_cache_read(type, got, page_size, slots, ko, vo, *gs)
    assert torch.equal(ko, kv.bfloat16()) and torch.equal(vo, vv.bfloat16())
    # one of the two alone, and into heads of a wider row
    wide = torch.full((T, 3 * H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    qfp4.kv_cache_read(type, got, page_size, slots, None, wide[:, H: 2 * H], *gs)
    assert torch.equal(wide[:, H: 2 * H], vo) and (wide[:, :H] == 7).all() and (wide[:, 2 * H:] == 7).all()
    assert qfp4.poll_device_status() == 0


@pytest.mark.parametrize("type", _cache.TYPES)
@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 64, 333])
def test_lengths_and_skipped_slots(type, T):
    g = torch.Generator(device="cuda").manual_seed(T)
    H, D, page_size, pages = 2, 128, 32, 12
    qkv = torch.randn(T, 4 * H * D, generator=g, device="cuda").bfloat16().view(T, 4 * H, D)
    k, v = qkv[:, H: 2 * H], qkv[:, 3 * H:]         # strided
    gs = scales(type)
    slots = slots_of(g, T, pages, page_size)
    keep = torch.rand(T, generator=g, device="cuda") < 0.7
    masked = torch.where(keep, slots, -1)
    want, got = (_cache.empty(type, pages, H, D, page_size, 0x5A) for _ in range(2))
    kv, vv = _cache.put(type, want, page_size, slots[keep], k[keep].float(), v[keep].float(), *gs)
    qfp4.kv_cache_write(type, k, v, masked, got, page_size, *gs)
    assert torch.equal(got, want)
    ko, vo = (torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qfp4.kv_cache_read(type, got, page_size, masked, ko, vo, *gs)
    assert torch.equal(ko[keep], kv.bfloat16()) and torch.equal(vo[keep], vv.bfloat16())
    assert (ko[~keep] == 0).all() and (vo[~keep] == 0).all()
    assert qfp4.poll_device_status() == 0


@pytest.mark.parametrize("type", _cache.TYPES)
def test_slots_beyond_the_cache_report(type):
    H, D, page_size, pages = 2, 64, 16, 3
    gs = scales(type)
    k = torch.ones(3, H, D, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([5, pages * page_size, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    want, got = (_cache.empty(type, pages, H, D, page_size) for _ in range(2))
    _cache.put(type, want, page_size, slots[:1], k[:1].float(), k[:1].float(), *gs)
    qfp4.kv_cache_write(type, k, k, slots, got, page_size, *gs)
    assert qfp4.poll_device_status() == -1 and torch.equal(got, want)
    ko, vo = torch.empty_like(k), torch.empty_like(k)
    qfp4.kv_cache_read(type, got, page_size, slots, ko, vo, *gs)
    assert qfp4.poll_device_status() == -1 and qfp4.poll_device_status() == 0
    assert (ko[1:] == 0).all() and (vo[1:] == 0).all() and (ko[0] != 0).all()


@pytest.mark.parametrize("type", _cache.TYPES)
def test_nan_and_infinity(type):
    """A NaN stays one; an infinity gives no finite value in its place."""
    D, gs = 64, scales(type)
    k = torch.ones(2, 1, D, dtype=torch.bfloat16, device="cuda")
    k[0, 0, 5], k[1, 0, 9] = float("nan"), float("inf")
    cache = _cache.empty(type, 1, 1, D, 16)
    slots = torch.arange(2, dtype=torch.int32, device="cuda")
    qfp4.kv_cache_write(type, k, k, slots, cache, 16, *gs)
    ko, vo = torch.empty_like(k), torch.empty_like(k)
    qfp4.kv_cache_read(type, cache, 16, slots, ko, vo, *gs)
    if type == qfp4.CACHE_NVFP4:        # E2M1 has neither: both saturate, as in the quantiser
        assert torch.isfinite(ko).all() and torch.isfinite(vo).all()
    else:
        assert torch.isnan(ko[0, 0, 5]) and not torch.isfinite(ko[1, 0, 9])
        assert torch.equal(ko.view(torch.int16), vo.view(torch.int16))      # no global scale tells them apart


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm,R", [(True, 1.0), (True, 0.5), (False, 1.0), (False, 0.0), (True, 0.0)])
@pytest.mark.parametrize("T,H,KV,D", [(1, 4, 1, 128), (19, 8, 8, 64), (37, 6, 2, 256), (70, 32, 8, 128)])
@pytest.mark.parametrize("type", _cache.TYPES)
def test_norm_rope_cache(type, T, H, KV, D, norm, R, inter):
    R = int(D * R)
    s = inputs(T, H, KV, D, R, norm, T + D)
    g = torch.Generator(device="cuda").manual_seed(T)
    page_size, pages, gs = 32, 4, scales(type)
    slots = slots_of(g, T, pages, page_size)
    cache = _cache.empty(type, pages, KV, D, page_size)
    q, q2, k2 = (torch.empty(T, n, D, dtype=torch.bfloat16, device="cuda") for n in (H, H, KV))
    args = (s["qw"], s["kw"], s["table"], s["pos"])
    qfp4.qk_norm_rope_cache(s["qkv"], H, KV, q, type, cache, page_size, slots, *args, *gs, eps=EPS, interleaved=inter)
    qfp4.qk_norm_rope(s["qkv"], H, KV, q2, k2, *args, eps=EPS, interleaved=inter)
    assert torch.equal(q, q2)
    ko, vo = (torch.empty(T, KV, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qfp4.kv_cache_read(type, cache, page_size, slots, ko, vo, *gs)
    v = s["qkv"][:, (H + KV) * D: (H + 2 * KV) * D].reshape(T, KV, D)
    assert torch.equal(vo, _cache.encode(type, v.float(), gs[1])[2].bfloat16())
    want, size = forward64(s, H, KV, D, R, inter)
    want, size = want[:, H:], size[:, H:]
    if type == qfp4.CACHE_BF16:
        assert torch.equal(ko, k2)
        return
    # half a code's step for the value itself, one more where the last bits of fp32 move it over a border; and the read's rounding
    if type == qfp4.CACHE_E4M3:
        top = want.abs().amax(-1, keepdim=True)
        step = torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** -10 / 448 * top)        # half a step
    else:
        blocks = want.unflatten(-1, (-1, 16))
        t = blocks.abs().amax(-1, keepdim=True) / 6 / gs[0].double()
        # the block's scale, off by half a step of UE4M3 (or 2^-10), and saturating at 448; half a step of E2M1 is a
        # quarter of the scale below 2, a fifth of the value above; what passes 6 scales is cut
        sc = torch.clamp(t * (1 + 2.0 ** -4) + 2.0 ** -10, max=448.0) * gs[0].double()
        least = torch.clamp(torch.clamp(t * (1 - 2.0 ** -4) - 2.0 ** -10, min=0.0), max=448.0) * gs[0].double()
        step = (torch.maximum(0.25 * sc.expand_as(blocks), blocks.abs() / 5) + (blocks.abs() - 6 * least).clamp(min=0)).flatten(-2)
    bound = step * (1 + 2.0 ** -10) + 2.0 ** -8 * (want.abs() + step) + 2.0 ** -19 * size
    assert ((ko.double() - want).abs() <= bound).all(), float(((ko.double() - want).abs() / bound).max())
    assert qfp4.poll_device_status() == 0


def test_norm_rope_cache_padding():
    """No position: nothing is written; a position without slot: the queries alone."""
    T, H, KV, D, type = 6, 2, 1, 64, qfp4.CACHE_E4M3
    s = inputs(T, H, KV, D, D, True, 3)
    s["pos"][1] = -1
    slots = torch.tensor([0, 1, -1, 3, 99, 5], dtype=torch.int32, device="cuda")
    cache = _cache.empty(type, 1, KV, D, 16, 0x77)
    before = cache.clone()
    q = torch.full((T, H, D), 9.0, dtype=torch.bfloat16, device="cuda")
    qfp4.qk_norm_rope_cache(s["qkv"], H, KV, q, type, cache, 16, slots, s["qw"], s["kw"], s["table"], s["pos"])
    assert qfp4.poll_device_status() == -1          # slot 99
    assert (q[1] == 9).all() and not (q[2] == 9).any() and not (q[4] == 9).any()
    written = _cache.empty(type, 1, KV, D, 16)
    _cache.put(type, written, 16, torch.tensor([0, 3, 5], device="cuda"), torch.full((3, KV, D), -1.0, device="cuda"), torch.full((3, KV, D), -1.0, device="cuda"), None, None)
    touched = written != 0
    assert torch.equal(cache[~touched], before[~touched])


@pytest.mark.parametrize("H,D", [(5, 64), (8, 128), (3, 256)])
@pytest.mark.parametrize("type", _cache.TYPES)
def test_read_of_many_tokens(type, H, D):
    """More tokens than the GPU has warps for each head: a warp takes several heads.
    The same slots many times, skipped and far ones among them, against small calls."""
    page_size, pages, T = 48, 7, 20011
    g = torch.Generator(device="cuda").manual_seed(H)
    gs, cache = scales(type), _cache.empty(type, pages, H, D, page_size)
    n = pages * page_size
    qfp4.kv_cache_write(type, vectors(g, n, H, D), vectors(g, n, H, D), torch.arange(n, dtype=torch.int32, device="cuda"), cache, page_size, *gs)
    k, v = (torch.empty(n, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for at in range(0, n, 42):
        qfp4.kv_cache_read(type, cache, page_size, torch.arange(at, at + 42, dtype=torch.int32, device="cuda"), k[at: at + 42], v[at: at + 42], *gs)
    assert qfp4.poll_device_status() == 0
    slots = torch.randint(-20, n, (T,), generator=g, device="cuda").int()
    slots[11::1000] = n
    slots[12::1000] = 2**31 - 1
    known = (slots >= 0) & (slots < n)
    at = torch.where(known, slots, 0).long()
    ko, vo = (torch.full((T + 1, H, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qfp4.kv_cache_read(type, cache, page_size, slots, ko[:T], vo[:T], *gs)
    assert qfp4.poll_device_status() == -1
    for got, want in ((ko, k), (vo, v)):
        assert torch.equal(got[:T], torch.where(known[:, None, None], want[at], 0)) and (got[T] == 7).all()


def test_offsets_beyond_32_bits():
    """A cache of more than 2^32 bytes: its last page."""
    type, H, D, page_size = qfp4.CACHE_BF16, 8, 128, 64
    page = qfp4.kv_cache_page_bytes(type, H, D, page_size)
    pages = (5 << 30) // page
    cache = torch.zeros(pages, H, page // H, dtype=torch.uint8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = vectors(g, 9, H, D), vectors(g, 9, H, D)
    slots = (pages * page_size - 1 - torch.arange(9, device="cuda")).int()
    qfp4.kv_cache_write(type, k, v, slots, cache, page_size)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    qfp4.kv_cache_read(type, cache, page_size, slots, ko, vo)
    assert torch.equal(ko, k) and torch.equal(vo, v)
    assert not cache[: pages - 1].any()


def test_graph_replays_with_new_contents():
    type, T, H, D, page_size = qfp4.CACHE_NVFP4, 5, 4, 128, 16
    g = torch.Generator(device="cuda").manual_seed(2)
    gs, cache = scales(type), _cache.empty(type, 2, H, D, page_size)
    k, v = vectors(g, T, H, D), vectors(g, T, H, D)
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    qfp4.kv_cache_write(type, k, v, slots, cache, page_size, *gs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qfp4.kv_cache_write(type, k, v, slots, cache, page_size, *gs)
        qfp4.kv_cache_read(type, cache, page_size, slots, ko, vo, *gs)
    for shift in (3, 11):
        k.copy_(vectors(g, T, H, D))
        slots.copy_(torch.arange(T, device="cuda") + shift)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ko, _cache.encode(type, k.float(), gs[0])[2].bfloat16()) and torch.equal(vo, _cache.encode(type, v.float(), gs[1])[2].bfloat16())
