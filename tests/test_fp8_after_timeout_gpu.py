"""What is queued right behind an 8-bit product that gives up on a wait (test
build: a release that never comes, 5 ms limit) is right: the kernel frees its
tensor memory only after what it had in flight has landed."""
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


@pytest.mark.parametrize("M,N,K", [(8, 256, 4096), (24, 512, 4096), (100, 4096, 2048), (2048, 4096, 1024)])
def test_calls_behind_one_that_gives_up(lib, M, N, K):
    """The released library's products, whose waits are not tampered with, on
    the same stream: they start while the first one ends."""
    g = torch.Generator().manual_seed(M)
    a = torch.randn(M, K, generator=g).to(torch.float8_e4m3fn).cuda()
    b = torch.randn(N, K, generator=g).to(torch.float8_e4m3fn).cuda()
    sa, sb = torch.ones(K // 128, M, device="cuda"), torch.ones(N // 128, K // 128, device="cuda")
    want = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    qfp4.gemm_nt_fp8(qfp4.E4M3, qfp4.E4M3, M, N, K, a, sa, b, sb, want)
    torch.cuda.synchronize()
    assert qfp4.poll_device_status() == 0 and lib.qfp4_poll_device_status(None) == 0
    lost, after = torch.empty_like(want), [torch.zeros_like(want) for _ in range(3)]
    assert lib.qfp4_test_inject_fp8_skip_release(1) == 0
    try:
        assert lib.qfp4_gemm_nt_fp8(0, 0, M, N, K, a.data_ptr(), sa.data_ptr(), b.data_ptr(), sb.data_ptr(), 128, 0, 0,
                                    lost.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
        for d in after:
            qfp4.gemm_nt_fp8(qfp4.E4M3, qfp4.E4M3, M, N, K, a, sa, b, sb, d)
        torch.cuda.synchronize()
    finally:
        assert lib.qfp4_test_inject_fp8_skip_release(0) == 0
    assert lib.qfp4_poll_device_status(None) == TIMEOUT and lib.qfp4_poll_device_status(None) == 0
    assert qfp4.poll_device_status() == 0
    assert all(torch.equal(d, want) for d in after)
