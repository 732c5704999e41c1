"""The bounded waits of the 8-bit products, made to run out by a release that
never comes (test build: 5 ms limit; nothing traps, faults or hangs): the call
ends, the status word says so, and the next call is right."""
import time

import pytest
import torch

from block_scaled_fp4_tcgen05_gb300 import qfp4

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


@pytest.mark.parametrize("M,N,K", [(2048, 4096, 1024), (64, 512, 4096), (8, 256, 4096), (100, 4096, 2048)])
def test_wait_runs_out_and_the_context_stays_usable(lib, M, N, K):
    """CTA pairs; single CTAs on a split K, in both orientations, every CTA with
    more K blocks than the two slots take."""
    g = torch.Generator().manual_seed(M)
    a = torch.randn(M, K, generator=g).to(torch.float8_e4m3fn).cuda()
    b = torch.randn(N, K, generator=g).to(torch.float8_e4m3fn).cuda()
    sa, sb = torch.ones(K // 128, M, device="cuda"), torch.ones(N // 128, K // 128, device="cuda")
    want = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    qfp4.gemm_nt_fp8(qfp4.E4M3, qfp4.E4M3, M, N, K, a, sa, b, sb, want)
    torch.cuda.synchronize()
    assert qfp4.poll_device_status() == 0 and lib.qfp4_poll_device_status(None) == 0

    def call(d):
        return lib.qfp4_gemm_nt_fp8(0, 0, M, N, K, a.data_ptr(), sa.data_ptr(), b.data_ptr(), sb.data_ptr(), 128, 0, 0,
                                    d.data_ptr(), torch.cuda.current_stream().cuda_stream)

    assert lib.qfp4_test_inject_fp8_skip_release(1) == 0
    d = torch.empty_like(want)
    began = time.perf_counter()
    assert call(d) == 0
    torch.cuda.synchronize()
    assert time.perf_counter() - began < 1.0
    assert lib.qfp4_poll_device_status(None) == TIMEOUT
    assert lib.qfp4_poll_device_status(None) == 0
    assert lib.qfp4_test_inject_fp8_skip_release(0) == 0
    assert call(d) == 0
    torch.cuda.synchronize()
    assert lib.qfp4_poll_device_status(None) == 0
    assert torch.equal(d, want)
