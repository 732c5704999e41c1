"""A process whose first call of each operator of the decoding layer is made under
stream capture: nothing that a first call sets up (attributes, occupancy queries,
addresses of status words) may need an eager call before it."""
import subprocess
import sys
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import torch
from block_scaled_fp4_tcgen05_gb300 import qfp4
T, H, KV, D, page = 9, 4, 2, 128, 16
g = torch.Generator(device="cuda").manual_seed(1)
bf16 = dict(dtype=torch.bfloat16, device="cuda")
qkv = torch.randn(T, (H + 2 * KV) * D, generator=g, device="cuda").bfloat16()
w = torch.ones(D, **bf16)
gs = torch.tensor([0.01], device="cuda")
cache = torch.zeros(2, KV, qfp4.kv_cache_page_bytes(qfp4.CACHE_NVFP4, 1, D, page), dtype=torch.uint8, device="cuda")
slots = torch.arange(T, dtype=torch.int32, device="cuda")
q, k, v, o = (torch.zeros(T, n, D, **bf16) for n in (H, KV, KV, H))
dqkv, dw = torch.zeros_like(qkv), [torch.zeros(D, device="cuda") for _ in range(2)]
ws, ws2 = (torch.zeros(n, dtype=torch.uint8, device="cuda") for n in
           (qfp4.qk_norm_rope_backward_workspace_bytes(T, H, KV, D), qfp4.attention_decode_workspace_bytes(T, H, KV, D)))
table, lengths = torch.zeros(T, 1, dtype=torch.int32, device="cuda"), torch.full((T,), 9, dtype=torch.int32, device="cuda")
code, sf = torch.randint(0, 256, (256, 64), generator=g, device="cuda", dtype=torch.uint8), torch.full((256 * 8,), 0x38, dtype=torch.uint8, device="cuda")
x, d = torch.randn(2, 128, generator=g, device="cuda").bfloat16(), torch.zeros(2, 256, **bf16)

def step():
    qfp4.qk_norm_rope_cache(qkv, H, KV, q, qfp4.CACHE_NVFP4, cache, page, slots, w, w, gs_k=gs, gs_v=gs)
    qfp4.kv_cache_read(qfp4.CACHE_NVFP4, cache, page, slots, k, v, gs, gs)
    qfp4.attention_decode(qfp4.CACHE_NVFP4, q, cache, page, table, lengths, 0.09, o, ws2, gs, gs)
    qfp4.qk_norm_rope_backward(qkv, H, KV, q, k, dqkv, *dw, ws, w, w)
    qfp4.gemv_nt(qfp4.NVFP4, x, code, sf, None, d)

out = (q, k, v, o, dqkv, *dw, d)
graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    step()
graph.replay()
torch.cuda.synchronize()
assert qfp4.poll_device_status() == 0
first = [t.clone() for t in out]
for t in out:
    t.zero_()
step()
torch.cuda.synchronize()
assert qfp4.poll_device_status() == 0 and all(t.any() and torch.equal(t, f) for t, f in zip(out, first))
print("the same")
"""


def test_first_calls_under_capture():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "the same" in r.stdout, r.stdout + r.stderr[-3000:]
