"""The bounded waits of the attention and of the head norms' gradient, made to run
out by bulk copies that are left out (test build: 5 ms limit; nothing traps, faults
or hangs): the call ends, the status word says so, and the next call is right."""
import time

import pytest
import torch

from block_scaled_fp4_tcgen05_gb300 import qfp4
from tests import _cache

pytestmark = pytest.mark.gpu
TIMEOUT = -5


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qfp4.load()
    assert qfp4.device_check() == 0
    from block_scaled_fp4_tcgen05_gb300 import build
    build.build(variant="faultinj")          # no-op when already built
    return qfp4.load_fault_injection()


def runs_out(lib, call, outputs):
    """call() with copies left out, then without."""
    lib.qfp4_test_inject_skip_copy(0)
    assert call() == 0
    torch.cuda.synchronize()
    assert lib.qfp4_poll_device_status(None) == 0
    want = [o.clone() for o in outputs]
    lib.qfp4_test_inject_skip_copy(1)
    began = time.perf_counter()
    assert call() == 0
    torch.cuda.synchronize()
    assert time.perf_counter() - began < 1.0
    assert lib.qfp4_poll_device_status(None) == TIMEOUT and lib.qfp4_poll_device_status(None) == 0
    lib.qfp4_test_inject_skip_copy(0)
    return want


@pytest.mark.parametrize("B", [2, 400])
@pytest.mark.parametrize("type", _cache.TYPES)
def test_attention(lib, type, B):
    H, KV, D, page_size, n = 8, 2, 128, 16, 300
    g = torch.Generator(device="cuda").manual_seed(B)
    pages = -(-n // page_size)
    cache = _cache.empty(type, pages, KV, D, page_size)
    gs = torch.tensor([0.01], device="cuda")
    k = torch.randn(n, KV, D, generator=g, device="cuda").bfloat16()
    qfp4.kv_cache_write(type, k, k, torch.arange(n, dtype=torch.int32, device="cuda"), cache, page_size, gs, gs)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(B, 1)
    lengths = torch.full((B,), n, dtype=torch.int32, device="cuda")
    q, o = torch.randn(B, H, D, generator=g, device="cuda").bfloat16(), torch.empty(B, H, D, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(qfp4.attention_decode_workspace_bytes(B, H, KV, D), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()

    def call():
        return lib.qfp4_attention_decode(type, q.data_ptr(), H * D, B, H, KV, D, cache.data_ptr(), pages, page_size, table.data_ptr(), pages, lengths.data_ptr(), 0, 0.09,
                                         gs.data_ptr(), gs.data_ptr(), o.data_ptr(), None, ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)

    want, = runs_out(lib, call, [o])
    ws.zero_()
    assert call() == 0
    torch.cuda.synchronize()
    assert lib.qfp4_poll_device_status(None) == 0 and torch.equal(o, want)


@pytest.mark.parametrize("T", [8, 4000])
def test_gradient(lib, T):
    H, KV, D = 8, 2, 128
    g = torch.Generator(device="cuda").manual_seed(T)
    qkv, dq, dk = (torch.randn(T, n * D, generator=g, device="cuda").bfloat16() for n in (H + 2 * KV, H, KV))
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    dqkv, dqw, dkw = torch.zeros_like(qkv), torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    ws = torch.empty(qfp4.qk_norm_rope_backward_workspace_bytes(T, H, KV, D), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()

    def call():
        return lib.qfp4_qk_norm_rope_backward(qkv.data_ptr(), (H + 2 * KV) * D, T, H, KV, D, w.data_ptr(), w.data_ptr(), 1e-6, None, 0, 0, 0, None, dq.data_ptr(), H * D,
                                              dk.data_ptr(), KV * D, dqkv.data_ptr(), (H + 2 * KV) * D, dqw.data_ptr(), dkw.data_ptr(), ws.data_ptr(), ws.numel(),
                                              torch.cuda.current_stream().cuda_stream)

    want = runs_out(lib, call, [dqkv, dqw, dkw])
    assert call() == 0
    torch.cuda.synchronize()
    assert lib.qfp4_poll_device_status(None) == 0
    assert all(torch.equal(a, b) for a, b in zip((dqkv, dqw, dkw), want))
