"""Refusals of the decoding attention layer beside those of test_decode_layer_abi.py (no
GPU needed): tensors of the right size and the wrong order of axes, scales of no use."""
import pytest
import torch

from block_scaled_fp4_tcgen05_gb300 import qfp4
from tests.test_decode_layer_abi import BF16, CASES, Tensor, calls  # noqa: F401

ROWS = ("D", "Q_out", "K_out", "dQ", "dK", "dQKV", "K", "V", "V_out")       # the others' shapes say the sizes


@pytest.mark.parametrize("fn,args", CASES, ids=lambda v: getattr(v, "__name__", ""))
def test_other_orders_of_axes(calls, fn, args):  # noqa: F811
    fn(**args)
    n = 1
    for name in args:
        t = args[name]
        if name not in ROWS or (name == "K_out" and fn is qfp4.kv_cache_read) or (name == "K" and fn is qfp4.kv_cache_write):
            continue
        s = tuple(t.shape)
        orders = [(s[1], s[0])] if len(s) == 2 else [(s[1], s[0], s[2]), (s[0], s[2], s[1]), (s[2], s[1], s[0]), (s[1], s[0] * s[2])]
        if fn in (qfp4.qk_norm_rope, qfp4.qk_norm_rope_cache) and name == "Q_out" or name == "dQ":
            orders = [o for o in orders if len(o) == 3 and o[2] == s[2]]    # its last axis says how long a head is
        for shape in [*orders, (1, *s)]:
            with pytest.raises((ValueError, IndexError)):
                fn(**{**args, name: Tensor(BF16, *shape)})
                raise AssertionError((name, shape))
        if len(s) == 3 and name not in ("Q_out", "dQ"):         # heads as one row
            fn(**{**args, name: Tensor(BF16, s[0], s[1] * s[2])})
            n += 1
    assert len(calls) == n
    assert all(c == calls[0] for c in calls)


def test_queries_of_the_attention(calls):  # noqa: F811
    fn, args = next(c for c in CASES if c[0] is qfp4.attention_decode)
    fn(**args)
    B, H, D = args["Q"].shape
    for shape in ((H, B, D), (B, D, H)):
        with pytest.raises(ValueError):
            fn(**{**args, "Q": Tensor(BF16, *shape)})
    assert len(calls) == 1


def test_scale_of_the_attention():
    """The kernel works in units of log 2: a scale that is infinite there gives NaN for logits of 0."""
    lib = qfp4.load()
    need = lib.qfp4_attention_decode_workspace_bytes(0, 8, 2, 128)

    def call(scale):
        return lib.qfp4_attention_decode(2, 1 << 40, 1024, 0, 8, 2, 128, 1 << 40, 4, 16, 1 << 40, 2, 1 << 40, 0, scale, 1 << 40, 1 << 40, 1 << 40, None, 1 << 40,
                                         need, None)

    for scale in (0.0, -1.0, 2.3e38, -2.3e38):
        assert call(scale) == 0, scale
    for scale in (2.4e38, -2.9e38, 3.3e38, float("inf"), float("nan")):
        assert call(scale) == -1, scale
