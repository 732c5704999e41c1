"""The example layer (router, gathered quantiser, experts' products, gradients)
against the same layer in fp32 torch with autograd."""
import importlib.util
import os

import pytest
import torch

from block_scaled_fp4_tcgen05_gb300 import qfp4

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_fp8_layer.py")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    assert qfp4.device_check() == 0
    spec = importlib.util.spec_from_file_location("moe_fp8_layer", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("T,E,k,D,H", [(300, 8, 2, 256, 128), (513, 16, 3, 144, 208), (40, 4, 1, 128, 64)])
def test_layer(example, T, E, k, D, H):
    x, logits, w_up, w_down, dy = example.inputs(T, E, D, H, seed=T)
    y, loss, grads = example.layer(x, logits, example.Experts(w_up), example.Experts(w_down), k, dy)
    assert qfp4.poll_device_status() == 0
    want_y, want_loss, want = example.plain(x, logits, w_up, w_down, k, dy, 0.01)
    assert abs(float(loss) - float(want_loss)) <= 1e-4 * float(want_loss)
    # An E4M3 code is off by 2^-4 of its value at most (0.027 rms over a uniform
    # mantissa), an E5M2 code by 2^-3 (0.05): three quantised factors in a row on
    # the way out, up to five on the way back, each product's own errors averaging
    # out; 0.1 and 0.2 are twice what that adds up to.
    assert float((y - want_y).norm() / want_y.norm()) <= 0.1
    for name in want:
        rel = float((grads[name].float() - want[name]).norm() / want[name].norm())
        assert rel <= 0.2, (name, rel)


def test_layer_with_padding(example):
    """Tokens that are not valid get no output and no gradient, and leave the
    others as they are without them."""
    T, E, k, D, H = 200, 8, 2, 256, 128
    x, logits, w_up, w_down, dy = example.inputs(T, E, D, H)
    up, down = example.Experts(w_up), example.Experts(w_down)
    valid = torch.ones(T, dtype=torch.uint8, device="cuda")
    valid[150:] = 0
    logits[160:170] = float("nan")
    y, loss, grads = example.layer(x, logits, up, down, k, dy, valid=valid)
    z, loss2, grads2 = example.layer(x[:150].contiguous(), logits[:150].contiguous(), up, down, k, dy[:150])
    assert qfp4.poll_device_status() == 0
    assert not y[150:].any() and not grads["x"][150:].any() and not grads["logits"][150:].any()
    assert torch.equal(y[:150], z) and torch.equal(grads["x"][:150], grads2["x"])
    for name in ("up", "down"):
        assert torch.equal(grads[name], grads2[name])
    assert torch.allclose(loss, loss2, rtol=1e-5) and torch.allclose(grads["logits"][:150], grads2["logits"], rtol=1e-4, atol=1e-9)
