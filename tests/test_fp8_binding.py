"""Sizes of the tensors given to the 8-bit and router calls (no GPU: stand-ins
for tensors and for the library).  The C ABI sees addresses only, so the binding
refuses a tensor shorter than what the kernels read or write."""
import inspect

import pytest
import torch

from block_scaled_fp4_tcgen05_gb300 import qfp4

F32, BF16, I32, U8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8


class Tensor:
    """What the binding asks of a contiguous tensor on the GPU."""
    is_cuda = True

    def __init__(self, dtype, *shape):
        self.dtype, self.shape = dtype, torch.Size(shape)

    def numel(self):
        return self.shape.numel()

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    @property
    def nbytes(self):
        return self.numel() * self.dtype.itemsize

    def data_ptr(self):
        return 1 << 40

    def shorter(self):
        return Tensor(self.dtype, self.numel() - 1)


@pytest.fixture
def calls(monkeypatch):
    """Names of the library calls that the binding lets through."""
    made = []

    class Library:
        def qfp4_fp8_grouped_cols(self, rows, groups):
            return 128 * (-(-rows // 128) + groups)

    monkeypatch.setattr(qfp4, "load", lambda: Library())
    monkeypatch.setattr(qfp4, "_call", lambda name, *a: made.append(name))
    monkeypatch.setattr(qfp4, "_stream", lambda s: None)
    return made


# function, its arguments by name, and those whose sizes it has to look at
M, N, K, G, T, E, TOPK = 200, 300, 272, 4, 50, 8, 2
COLS = 128 * (2 + G)
CASES = [
    (qfp4.fp8_quantize, dict(type=qfp4.E4M3, X=Tensor(BF16, M, K), Q=Tensor(U8, M, K), SF=Tensor(F32, 3, M), Q_t=Tensor(U8, K, 208),
                             SF_t=Tensor(F32, 2, K)), ("Q", "SF", "Q_t", "SF_t")),
    (qfp4.fp8_quantize, dict(type=qfp4.E5M2, X=Tensor(BF16, 7, K), Q=Tensor(U8, M, K), SF=Tensor(F32, 3, M), Q_t=Tensor(U8, K, 208),
                             SF_t=Tensor(F32, 2, K), row_index=Tensor(I32, M)), ("Q", "SF", "Q_t", "SF_t")),
    (qfp4.fp8_quantize_grouped, dict(type=qfp4.E4M3, X=Tensor(BF16, M, K), row_offsets=Tensor(I32, G + 1), Q_t=Tensor(U8, K, COLS),
                                     SF_t=Tensor(F32, COLS // 128, K), Q=Tensor(U8, M, K), SF=Tensor(F32, 3, M)),
     ("Q", "SF", "Q_t", "SF_t")),
    (qfp4.fp8_quantize_weight, dict(type=qfp4.E4M3, W=Tensor(BF16, G, N, K), Q=Tensor(U8, G, N, K), SF=Tensor(F32, G, 3, 3),
                                    Q_t=Tensor(U8, G, K, 304), SF_t=Tensor(F32, G, 3, 3)), ("Q", "SF", "Q_t", "SF_t")),
    (qfp4.gemm_nt_fp8, dict(a_type=qfp4.E4M3, b_type=qfp4.E5M2, M=M, N=N, K=K, A=Tensor(U8, M, K), A_sf=Tensor(F32, 3, M),
                            B=Tensor(U8, N, K), B_sf=Tensor(F32, 3, 3), D=Tensor(BF16, M, N)), ("A", "A_sf", "B", "B_sf", "D")),
    (qfp4.gemm_nt_fp8, dict(a_type=qfp4.E4M3, b_type=qfp4.E4M3, M=M, N=N, K=K, A=Tensor(U8, M, K), A_sf=Tensor(F32, 3, M),
                            B=Tensor(U8, N, K), B_sf=Tensor(F32, 3, N), D=Tensor(F32, M, N), b_rows=1, out=qfp4.OUT_FP32),
     ("A", "A_sf", "B", "B_sf", "D")),
    (qfp4.gemm_nt_fp8_grouped, dict(a_type=qfp4.E4M3, b_type=qfp4.E4M3, row_offsets=Tensor(I32, G + 1), total_rows=M, max_group_rows=0,
                                    N=N, K=K, A=Tensor(U8, M, K), A_sf=Tensor(F32, 3, M), B=Tensor(U8, G, N, K),
                                    B_sf=Tensor(F32, G, 3, 3), D=Tensor(BF16, M, N)), ("A", "A_sf", "B", "B_sf", "D")),
    (qfp4.gemm_nt_fp8_kgrouped, dict(a_type=qfp4.E5M2, b_type=qfp4.E4M3, row_offsets=Tensor(I32, G + 1), total_rows=M, M=48, N=80,
                                     A=Tensor(U8, 48, COLS), A_sf=Tensor(F32, COLS // 128, 48), B=Tensor(U8, 80, COLS),
                                     B_sf=Tensor(F32, COLS // 128, 80), D=Tensor(F32, G, 48, 80)), ("A", "A_sf", "B", "B_sf", "D")),
    (qfp4.moe_route, dict(logits=Tensor(F32, T, E), topk=TOPK, ids=Tensor(I32, T, TOPK), gates=Tensor(F32, T, TOPK), counts=Tensor(I32, E),
                          row_offsets=Tensor(I32, E + 1), dest=Tensor(I32, T, TOPK), src=Tensor(I32, T * TOPK), n_valid=Tensor(I32, 1),
                          mean_prob=Tensor(F32, E), loss=Tensor(F32, 1), workspace=Tensor(U8, 1 << 20), valid=Tensor(U8, T)),
     ("ids", "gates", "counts", "row_offsets", "dest", "src", "n_valid", "mean_prob", "loss", "valid")),
    (qfp4.moe_route_backward, dict(logits=Tensor(BF16, T, E), ids=Tensor(I32, T, TOPK), counts=Tensor(I32, E), n_valid=Tensor(I32, 1),
                                   dgates=Tensor(F32, T, TOPK), dloss=Tensor(F32, 1), dlogits=Tensor(BF16, T, E), valid=Tensor(U8, T)),
     ("counts", "n_valid", "dgates", "dloss", "dlogits", "valid")),
]


@pytest.mark.parametrize("function,arguments,sized", CASES, ids=[f"{c[0].__name__}-{i}" for i, c in enumerate(CASES)])
def test_a_tensor_that_is_too_short_is_refused(calls, function, arguments, sized):
    function(**arguments)
    assert calls == ["qfp4_" + function.__name__]       # as long as it has to be
    function(**{k: Tensor(v.dtype, v.numel() + 5) if k in sized else v for k, v in arguments.items()})      # or longer
    for name in sized:
        del calls[:]
        with pytest.raises(ValueError, match="at least"):
            function(**{**arguments, name: arguments[name].shorter()})
        assert not calls
    # nothing that has a size is left out: the others are what the sizes are taken from
    rest = {n for n, v in arguments.items() if isinstance(v, Tensor)} - set(sized)
    assert rest <= {"X", "W", "logits", "row_index", "row_offsets", "workspace", "ids"}, rest
    assert set(arguments) <= set(inspect.signature(function).parameters)


def test_choices_of_fewer_tokens_than_logits_are_refused(calls):
    a = {**CASES[-1][1], "ids": Tensor(I32, T - 1, TOPK)}
    with pytest.raises(ValueError, match="at least"):
        qfp4.moe_route_backward(**a)
    assert not calls


def test_other_refusals_say_what_they_are(calls):
    a = CASES[4][1]
    with pytest.raises(ValueError, match="float32"):
        qfp4.gemm_nt_fp8(**{**a, "A_sf": Tensor(BF16, 3, M)})
    strided = Tensor(BF16, M, N)
    strided.is_contiguous = lambda: False
    with pytest.raises(ValueError, match="contiguous"):
        qfp4.gemm_nt_fp8(**{**a, "D": strided})
    qfp4.gemm_nt_fp8(**{**a, "A": 1 << 40, "D": 1 << 40})       # addresses stand as they are
    assert calls == ["qfp4_gemm_nt_fp8"]


def test_arguments_reach_the_library_as_they_are():
    """Every call that takes its arguments as packed words, against the C entry
    itself: each argument is made bad in turn, and both refuse it alike."""
    if torch.cuda.is_available():
        pytest.skip("a call that is not refused would be launched with these addresses")
    lib = qfp4.load()
    fake = 1 << 40
    values = {
        "qfp4_fp8_quantize": (0, 0, fake, 16, None, 16, 256, fake, fake, fake, fake, None),
        "qfp4_fp8_quantize_grouped": (0, 0, fake, 16, None, 4, fake, 16, 256, fake, fake, fake, fake, None),
        "qfp4_fp8_quantize_weight": (0, 0, 1, fake, 128, 256, fake, fake, fake, fake, None),
        "qfp4_gemm_nt_fp8": (0, 1, 16, 128, 256, fake, fake, fake, fake, 128, 0, 0, fake, None),
        "qfp4_gemm_nt_fp8_grouped": (0, 0, 4, fake, 64, 0, 128, 256, fake, fake, fake, fake, 0, fake, None),
        "qfp4_gemm_nt_fp8_kgrouped": (1, 0, 4, fake, 64, 128, 256, fake, fake, fake, fake, 0, fake, None),
        "qfp4_moe_route": (1, fake, 64, 8, 2, None, 1, *[fake] * 9, fake, 1 << 20, None),
        "qfp4_moe_route_backward": (0, fake, 64, 8, 2, None, 0, fake, fake, fake, fake, fake, fake, None),
    }
    assert set(values) == set(qfp4._WORDS)
    for name, good in values.items():
        function, pack = qfp4._words[name]
        assert len(good) == len(qfp4.SIGNATURES[name][1])
        refused = 0
        for i, v in enumerate(good):
            for bad in (-(1 << 40) - 7, -1, 0, fake + 1):
                args = (*good[:i], bad, *good[i + 1:])
                want = getattr(lib, name)(*[None if a is None else a for a in args])
                if want in (0, -4):     # not refused (there is no GPU to launch it on)
                    continue
                refused += 1
                assert function(pack(*(0 if a is None else a for a in args))) == want, (name, i, bad)
        assert refused >= len(good), name
