"""Read from the sources (no GPU): a kernel that gave up on a wait lets what is
still in flight land before it frees its tensor memory.  Columns freed earlier
could go to another CTA, which the MMAs in flight would then write into."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_scaled_fp4_tcgen05_gb300", "csrc")


def frees():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"\btmem_dealloc(_pair)?\(", text):
            yield pytest.param(text[:m.start()], id=f"{os.path.basename(path)}:{text[:m.start()].count(chr(10)) + 1}")


@pytest.mark.parametrize("before", list(frees()))
def test_delay_comes_before_tensor_memory_is_freed(before):
    barrier = max(before.rfind("cluster_sync_all()"), before.rfind("__syncthreads()"))
    delay = re.search(r"if \(\*abort_flag\) \{\s*const uint64_t t0 = globaltimer_ns\(\);\s*while \(globaltimer_ns\(\) - t0 <",
                      before[barrier:])
    assert barrier > 0 and delay, "no delay between the CTA's last barrier and the release"


def test_there_is_something_to_read():
    assert len(list(frees())) >= 5
