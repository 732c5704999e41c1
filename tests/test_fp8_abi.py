"""Refusals of the 8-bit floating point and router entry points: bad arguments
are answered on the host, before anything is launched (no GPU needed)."""
import os

import pytest
import torch

from block_scaled_fp4_tcgen05_gb300 import qfp4

OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, -1, -2, -3, -7
FAKE = 1 << 40          # a 16-byte aligned address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(qfp4.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return qfp4.load()


def caller(fn, **defaults):
    def call(**kw):
        assert set(kw) <= set(defaults), kw
        return fn(*{**defaults, **kw}.values())
    return call


def test_quantize(lib):
    call = caller(lib.qfp4_fp8_quantize, type=0, scale=0, X=FAKE, X_rows=16, row_index=None, M=16, K=256, Q=FAKE, SF=FAKE,
                  Q_t=FAKE, SF_t=FAKE, stream=None)
    for bad in (dict(type=2), dict(type=-1), dict(scale=2), dict(M=-1), dict(K=-16), dict(X=None), dict(X_rows=15),
                dict(X_rows=-1), dict(Q=None), dict(SF=None), dict(Q_t=None), dict(SF_t=None),
                dict(Q=None, SF=None, Q_t=None, SF_t=None)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(K=8), dict(K=250), dict(K=1 << 31), dict(M=1 << 31, X_rows=1 << 31)):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(X=FAKE + 8), dict(Q=FAKE + 4), dict(Q_t=FAKE + 8), dict(SF=FAKE + 2), dict(SF_t=FAKE + 1),
                dict(row_index=FAKE + 2)):
        assert call(**bad) == MISALIGNED, bad
    assert call(M=0, X_rows=0) == OK and call(K=0) == OK


def test_quantize_weight(lib):
    call = caller(lib.qfp4_fp8_quantize_weight, type=0, scale=0, groups=1, W=FAKE, N=128, K=256, Q=FAKE, SF=FAKE,
                  Q_t=FAKE, SF_t=FAKE, stream=None)
    for bad in (dict(type=7), dict(scale=-1), dict(groups=0), dict(N=-1), dict(W=None), dict(Q=None), dict(SF=None),
                dict(Q_t=None), dict(SF_t=None)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(K=24), dict(groups=65536), dict(N=1 << 31)):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(W=FAKE + 2), dict(Q=FAKE + 8), dict(Q_t=FAKE + 1), dict(SF=FAKE + 3), dict(SF_t=FAKE + 2)):
        assert call(**bad) == MISALIGNED, bad
    assert call(N=0) == OK


def test_quantize_grouped(lib):
    call = caller(lib.qfp4_fp8_quantize_grouped, type=0, scale=0, X=FAKE, X_rows=16, row_index=None, groups=4, offs=FAKE,
                  rows=16, K=256, Q=FAKE, SF=FAKE, Q_t=FAKE, SF_t=FAKE, stream=None)
    for bad in (dict(type=2), dict(scale=5), dict(groups=0), dict(offs=None), dict(rows=-1, X_rows=-1), dict(K=-16),
                dict(X=None), dict(X_rows=15), dict(Q=None), dict(SF=None), dict(Q_t=None), dict(SF_t=None)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(K=40), dict(groups=257), dict(rows=1 << 31, X_rows=1 << 31)):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(X=FAKE + 8), dict(Q_t=FAKE + 4), dict(offs=FAKE + 2), dict(row_index=FAKE + 1), dict(SF_t=FAKE + 2)):
        assert call(**bad) == MISALIGNED, bad
    assert call(rows=0, X_rows=0) == OK
    assert qfp4.fp8_grouped_cols(0, 3) == 384 and qfp4.fp8_grouped_cols(129, 2) == 512
    assert qfp4.fp8_grouped_cols(-1, 2) == 0 and qfp4.fp8_grouped_cols(5, 0) == 0


def test_kgrouped(lib):
    call = caller(lib.qfp4_gemm_nt_fp8_kgrouped, ta=1, tb=0, groups=4, offs=FAKE, rows=64, M=128, N=256, A=FAKE, A_sf=FAKE,
                  B=FAKE, B_sf=FAKE, accumulate=0, D=FAKE, stream=None)
    for bad in (dict(ta=2), dict(tb=9), dict(groups=0), dict(offs=None), dict(rows=-1), dict(M=-1), dict(N=-1),
                dict(A=None), dict(A_sf=None), dict(B=None), dict(B_sf=None), dict(D=None)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(groups=257), dict(M=1 << 29), dict(N=1 << 31), dict(rows=1 << 31)):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(offs=FAKE + 2), dict(A=FAKE + 4), dict(B=FAKE + 8), dict(D=FAKE + 8), dict(A_sf=FAKE + 1),
                dict(B_sf=FAKE + 3)):
        assert call(**bad) == MISALIGNED, bad
    assert call(M=0) == OK and call(N=0) == OK


def test_gemm(lib):
    call = caller(lib.qfp4_gemm_nt_fp8, ta=0, tb=1, M=16, N=128, K=256, A=FAKE, A_sf=FAKE, B=FAKE, B_sf=FAKE, b_rows=128,
                  out=0, accumulate=0, D=FAKE, stream=None)
    for bad in (dict(ta=2), dict(tb=-1), dict(out=2), dict(b_rows=64), dict(b_rows=0), dict(M=-1), dict(N=-1), dict(K=-1),
                dict(A=None), dict(A_sf=None), dict(B=None), dict(B_sf=None), dict(D=None), dict(accumulate=1)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(K=8), dict(K=100), dict(M=1 << 31), dict(N=1 << 31), dict(K=1 << 31)):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(A=FAKE + 8), dict(B=FAKE + 1), dict(D=FAKE + 2), dict(A_sf=FAKE + 2), dict(B_sf=FAKE + 1)):
        assert call(**bad) == MISALIGNED, bad
    assert call(M=0) == OK and call(N=0) == OK
    assert call(K=0, out=1, accumulate=1) == OK          # an empty sum is added


def test_grouped(lib):
    call = caller(lib.qfp4_gemm_nt_fp8_grouped, ta=0, tb=0, groups=4, offs=FAKE, rows=64, most=0, N=128, K=256, A=FAKE,
                  A_sf=FAKE, B=FAKE, B_sf=FAKE, out=0, D=FAKE, stream=None)
    for bad in (dict(ta=3), dict(out=-1), dict(groups=0), dict(offs=None), dict(rows=-1), dict(most=-1), dict(N=0),
                dict(K=0), dict(A=None), dict(A_sf=None), dict(B=None), dict(B_sf=None), dict(D=None)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(groups=257), dict(K=24), dict(N=1 << 29), dict(rows=1 << 31)):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(offs=FAKE + 2), dict(A=FAKE + 4), dict(B=FAKE + 8), dict(D=FAKE + 8), dict(A_sf=FAKE + 1),
                dict(B_sf=FAKE + 3)):
        assert call(**bad) == MISALIGNED, bad
    assert call(rows=0) == OK


def test_route(lib):
    names = ("ids", "gates", "counts", "row_offsets", "dest", "src", "n_valid", "mean_prob", "loss", "workspace")
    call = caller(lib.qfp4_moe_route, kind=1, logits=FAKE, T=64, E=8, topk=2, valid=None, renorm=1,
                  **{n: FAKE for n in names}, ws_bytes=1 << 20, stream=None)
    for bad in (dict(kind=2), dict(T=-1), dict(E=0), dict(topk=0), dict(logits=None), *({n: None} for n in names)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(E=257), dict(topk=9), dict(E=64, topk=17), dict(T=1 << 31)):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(logits=FAKE + 4), dict(workspace=FAKE + 8), *({n: FAKE + 2} for n in names[:-1])):
        assert call(**bad) == MISALIGNED, bad
    assert call(ws_bytes=16) == WORKSPACE
    assert call(ws_bytes=0) == WORKSPACE


def test_route_workspace(lib):
    most = 0
    for T in (0, 1, 16, 17, 4096, 1 << 20, 1 << 26):
        for E, k in ((1, 1), (8, 2), (64, 6), (256, 8), (256, 16)):
            need = qfp4.moe_route_workspace_bytes(T, E, k)
            assert need > 0
            most = max(most, need)
    assert most <= 1 << 20
    for T, E, k in ((-1, 8, 2), (4, 0, 1), (4, 8, 0), (4, 257, 1), (4, 4, 5)):
        assert qfp4.moe_route_workspace_bytes(T, E, k) == 0


def test_route_backward(lib):
    names = ("ids", "counts", "n_valid", "dgates", "dloss", "dlogits")
    call = caller(lib.qfp4_moe_route_backward, kind=0, logits=FAKE, T=64, E=8, topk=2, valid=None, renorm=0,
                  **{n: FAKE for n in names}, stream=None)
    for bad in (dict(kind=-1), dict(T=-1), dict(E=0), dict(topk=0), dict(logits=None),
                *({n: None} for n in ("ids", "counts", "n_valid", "dlogits"))):
        assert call(**bad) == INVALID, bad
    for bad in (dict(E=300), dict(topk=9)):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(logits=FAKE + 8), dict(dlogits=FAKE + 4), *({n: FAKE + 1} for n in names[:-1])):
        assert call(**bad) == MISALIGNED, bad
    assert call(T=0) == OK


def test_binding_refuses_what_the_abi_cannot_see(lib):
    x = torch.zeros(32, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        qfp4.fp8_quantize(qfp4.E4M3, x, x, x)                       # on the host
    with pytest.raises(ValueError):
        qfp4.moe_route_backward(x.t(), x, x, x, None, None, x)      # strided


def test_binding_refuses_codes_of_another_type(lib):
    x = torch.zeros(32, 64, dtype=torch.bfloat16)
    e4m3, e5m2 = (torch.zeros(32, 64, dtype=t) for t in (torch.float8_e4m3fn, torch.float8_e5m2))
    for a_type, a in ((qfp4.E4M3, e5m2), (qfp4.E5M2, e4m3), (qfp4.E4M3, x)):
        with pytest.raises(ValueError, match="codes"):      # the other arguments are addresses
            qfp4.gemm_nt_fp8(a_type, qfp4.E4M3, 32, 32, 64, a, 16, 16, 16, 16)
