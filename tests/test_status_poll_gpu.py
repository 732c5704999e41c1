"""The status poll: one reading gathers and clears the words of every kernel,
and costs no more than a launch and one copy back."""
import statistics
import threading
import time

import pytest
import torch

from block_scaled_fp4_tcgen05_gb300 import qfp4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qfp4.load()
    assert qfp4.device_check() == 0


def bad_quantize(stream=None):
    """An index beyond X: recorded, nothing read."""
    x = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")
    q, sf = torch.empty(2, 128, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(1, 2, device="cuda")
    index = torch.tensor([0, 9], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    qfp4.fp8_quantize(qfp4.E4M3, x, q, sf, row_index=index, stream=stream)


def bad_product():
    offs = torch.tensor([0, 6, 4], dtype=torch.int32, device="cuda")
    z, s = torch.zeros(256, 128, dtype=torch.uint8, device="cuda"), torch.ones(2, 8, device="cuda")
    d = torch.empty(8, 128, dtype=torch.bfloat16, device="cuda")
    qfp4.gemm_nt_fp8_grouped(qfp4.E4M3, qfp4.E4M3, offs, 8, 0, 128, 128, z[:8], s[:1], z, s[:, :1].contiguous(), d)


def test_one_poll_gathers_and_clears_every_word():
    assert qfp4.poll_device_status() == 0
    bad_quantize()
    bad_product()
    assert qfp4.poll_device_status() == -1
    assert qfp4.poll_device_status() == 0


def test_poll_is_ordered_behind_its_stream():
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)
        bad_quantize(side)
        assert qfp4.poll_device_status(side) == -1
    assert qfp4.poll_device_status() == 0


def test_polls_of_many_threads():
    """A word set once is reported exactly once, whichever thread's poll meets it."""
    seen, errors = [], []
    gate = threading.Barrier(8)

    def work():
        try:
            stream = torch.cuda.Stream()
            for _ in range(20):
                gate.wait()
                seen.append(qfp4.poll_device_status(stream))
                gate.wait()
        except Exception as e:      # a thread's failure must fail the test
            errors.append(e)
            gate.abort()

    threads = [threading.Thread(target=work) for _ in range(8)]
    bad_quantize()
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert sorted(set(seen)) == [-1, 0] and seen.count(-1) == 1


def test_poll_costs_one_round_trip():
    """A launch, a copy and a wait: within five reads of four bytes by torch
    (each of them a copy and a wait), where a copy and a wait to read and as much
    to clear each kernel's word would take more than ten."""
    word = torch.zeros(1, dtype=torch.int32, device="cuda")

    def median_us(call):
        times = []
        for _ in range(300):
            began = time.perf_counter()
            call()
            times.append(time.perf_counter() - began)
        return statistics.median(times) * 1e6

    for call in (word.item, qfp4.poll_device_status):
        median_us(call)
    read, poll = median_us(word.item), median_us(qfp4.poll_device_status)
    assert poll <= 5 * read, (poll, read)
