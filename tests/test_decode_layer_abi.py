"""Refusals of the entry points of the decoding attention layer: bad arguments are
answered on the host, before anything is launched (no GPU needed); and tensors
that the binding refuses."""
import inspect
import os

import pytest
import torch

from block_scaled_fp4_tcgen05_gb300 import qfp4

OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, -1, -2, -3, -7
FAKE = 1 << 40          # a 16-byte aligned address that is never dereferenced
NAN, INF = float("nan"), float("inf")


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


HEADS = dict(QKV=FAKE, ld=10 * 128, T=4, q_heads=4, kv_heads=2, head_dim=128, q_weight=FAKE, k_weight=FAKE, eps=1e-6, cos_sin=FAKE,
             table_rows=64, rotary_dim=128, interleaved=0, positions=FAKE)


def refuses_heads(call):
    """What all calls on query and key heads refuse."""
    for bad in (dict(T=-1), dict(q_heads=0), dict(kv_heads=0), dict(head_dim=0), dict(rotary_dim=-16), dict(interleaved=2), dict(eps=-1.0), dict(eps=NAN),
                dict(eps=INF), dict(ld=128), dict(q_weight=None), dict(k_weight=None), dict(cos_sin=None), dict(positions=None), dict(table_rows=0),
                dict(table_rows=-1), dict(QKV=None)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(rotary_dim=144), dict(rotary_dim=24), dict(T=(1 << 30) + 1), dict(ld=10 * 128 + 4)):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(QKV=FAKE + 8), dict(q_weight=FAKE + 2), dict(k_weight=FAKE + 8), dict(cos_sin=FAKE + 4), dict(positions=FAKE + 2)):
        assert call(**bad) == MISALIGNED, bad
    assert call(T=0) == OK


def test_norm_rope(lib):
    call = caller(lib.qfp4_qk_norm_rope, **HEADS, Q=FAKE, ldq=512, K=FAKE, ldk=256, stream=None)
    refuses_heads(call)
    for bad in (dict(Q=None), dict(K=None), dict(ldq=504), dict(ldk=248)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(ldq=516), dict(ldk=260), dict(head_dim=272, rotary_dim=16, ld=10 * 272, ldq=4 * 272, ldk=2 * 272), dict(head_dim=40, rotary_dim=16),
                dict(q_heads=4097, ld=1 << 20, ldq=1 << 20)):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(Q=FAKE + 2), dict(K=FAKE + 8)):
        assert call(**bad) == MISALIGNED, bad


def test_norm_rope_cache(lib):
    call = caller(lib.qfp4_qk_norm_rope_cache, **HEADS, Q=FAKE, ldq=512, type=2, cache=FAKE, pages=4, page_size=16, slots=FAKE, gs_k=FAKE, gs_v=FAKE,
                  stream=None)
    refuses_heads(call)
    for bad in (dict(Q=None), dict(ldq=504), dict(type=3), dict(type=-1), dict(cache=None), dict(pages=-1), dict(page_size=0), dict(slots=None),
                dict(gs_k=None), dict(gs_v=None), dict(ld=7 * 128)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(head_dim=96, rotary_dim=96), dict(page_size=24), dict(page_size=1 << 17), dict(pages=1 << 28), dict(ldq=514)):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(cache=FAKE + 8), dict(slots=FAKE + 2), dict(gs_k=FAKE + 1), dict(gs_v=FAKE + 2), dict(Q=FAKE + 4)):
        assert call(**bad) == MISALIGNED, bad


def test_norm_rope_backward(lib):
    need = lib.qfp4_qk_norm_rope_backward_workspace_bytes(4, 4, 2, 128)
    assert need > 0
    call = caller(lib.qfp4_qk_norm_rope_backward, **HEADS, dQ=FAKE, lddq=512, dK=FAKE, lddk=256, dQKV=FAKE, lddqkv=1280, dq_weight=FAKE, dk_weight=FAKE,
                  workspace=FAKE, ws_bytes=need, stream=None)
    for bad in (dict(dQ=None), dict(dK=None), dict(dQKV=None), dict(lddq=504), dict(lddk=248), dict(lddqkv=760), dict(dq_weight=None), dict(dk_weight=None),
                dict(eps=NAN), dict(T=-1)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(lddq=516), dict(lddk=258), dict(lddqkv=1284)):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(dQ=FAKE + 8), dict(dK=FAKE + 2), dict(dQKV=FAKE + 8), dict(dq_weight=FAKE + 2), dict(dk_weight=FAKE + 1), dict(workspace=FAKE + 8)):
        assert call(**bad) == MISALIGNED, bad
    assert call(workspace=None) == WORKSPACE and call(ws_bytes=need - 1) == WORKSPACE
    assert call(T=0, q_weight=None, k_weight=None, dq_weight=None, dk_weight=None, workspace=None, ws_bytes=0) == OK
    for bad in ((-1, 4, 2, 128), (4, 0, 2, 128), (4, 4, 0, 128), (4, 4, 2, 100), (4, 4, 2, 512)):
        assert lib.qfp4_qk_norm_rope_backward_workspace_bytes(*bad) == 0, bad


def test_page_bytes():
    assert qfp4.kv_cache_page_bytes(qfp4.CACHE_BF16, 8, 128, 16) == 8 * 16 * 2 * 256
    assert qfp4.kv_cache_page_bytes(qfp4.CACHE_E4M3, 2, 64, 32) == 2 * 32 * 2 * (64 + 4)
    assert qfp4.kv_cache_page_bytes(qfp4.CACHE_NVFP4, 1, 256, 48) == 48 * 2 * (128 + 16)
    for bad in ((3, 8, 128, 16), (0, 0, 128, 16), (0, 8, 96, 16), (0, 8, 128, 8), (0, 8, 128, 0), (0, 8, 128, 1 << 17)):
        assert qfp4.kv_cache_page_bytes(*bad) == 0, bad


def test_cache_write_and_read(lib):
    write = caller(lib.qfp4_kv_cache_write, type=2, K=FAKE, ldk=256, V=FAKE, ldv=256, T=4, kv_heads=2, head_dim=128, slots=FAKE, gs_k=FAKE, gs_v=FAKE,
                   cache=FAKE, pages=4, page_size=16, stream=None)
    read = caller(lib.qfp4_kv_cache_read, type=2, cache=FAKE, pages=4, page_size=16, kv_heads=2, head_dim=128, slots=FAKE, T=4, gs_k=FAKE, gs_v=FAKE, K=FAKE,
                  ldk=256, V=FAKE, ldv=256, stream=None)
    for call in (write, read):
        for bad in (dict(type=3), dict(T=-1), dict(kv_heads=0), dict(head_dim=0), dict(slots=None), dict(gs_k=None), dict(gs_v=None), dict(cache=None),
                    dict(pages=-1), dict(page_size=0), dict(ldk=248), dict(ldv=128)):
            assert call(**bad) == INVALID, bad
        for bad in (dict(head_dim=32), dict(head_dim=192, ldk=384, ldv=384), dict(page_size=20), dict(T=(1 << 30) + 1), dict(ldk=260), dict(ldv=258)):
            assert call(**bad) == UNSUPPORTED, bad
        for bad in (dict(K=FAKE + 8), dict(V=FAKE + 2), dict(cache=FAKE + 4), dict(slots=FAKE + 1), dict(gs_k=FAKE + 2)):
            assert call(**bad) == MISALIGNED, bad
        assert call(T=0) == OK
    assert write(K=None) == INVALID and write(V=None) == INVALID and read(K=None, V=None) == INVALID


def test_more_heads_than_32_bits_count(lib):
    wide = dict(T=1 << 30, q_heads=2048, kv_heads=2048, ld=1 << 19)
    forward = caller(lib.qfp4_qk_norm_rope, **HEADS, Q=FAKE, ldq=1 << 18, K=FAKE, ldk=1 << 18, stream=None)
    assert forward(**wide) == UNSUPPORTED
    fused = caller(lib.qfp4_qk_norm_rope_cache, **HEADS, Q=FAKE, ldq=1 << 18, type=2, cache=FAKE, pages=4, page_size=16, slots=FAKE, gs_k=FAKE, gs_v=FAKE,
                   stream=None)
    assert fused(**{**wide, "ld": 3 << 18}) == UNSUPPORTED
    backward = caller(lib.qfp4_qk_norm_rope_backward, **HEADS, dQ=FAKE, lddq=1 << 18, dK=FAKE, lddk=1 << 18, dQKV=FAKE, lddqkv=1 << 19, dq_weight=FAKE,
                      dk_weight=FAKE, workspace=FAKE, ws_bytes=1 << 40, stream=None)
    assert backward(**wide) == UNSUPPORTED
    assert lib.qfp4_qk_norm_rope_backward_workspace_bytes(1 << 30, 2048, 2048, 128) == 0
    write = caller(lib.qfp4_kv_cache_write, type=2, K=FAKE, ldk=512, V=FAKE, ldv=512, T=1 << 29, kv_heads=4, head_dim=128, slots=FAKE, gs_k=FAKE, gs_v=FAKE,
                   cache=FAKE, pages=4, page_size=16, stream=None)
    read = caller(lib.qfp4_kv_cache_read, type=2, cache=FAKE, pages=4, page_size=16, kv_heads=4, head_dim=128, slots=FAKE, T=1 << 29, gs_k=FAKE, gs_v=FAKE,
                  K=FAKE, ldk=512, V=FAKE, ldv=512, stream=None)
    assert write() == UNSUPPORTED and read() == UNSUPPORTED


def test_attention(lib):
    need = lib.qfp4_attention_decode_workspace_bytes(2, 8, 2, 128)
    assert need > 0
    call = caller(lib.qfp4_attention_decode, type=2, Q=FAKE, ldq=1024, B=2, q_heads=8, kv_heads=2, head_dim=128, cache=FAKE, pages=4, page_size=16,
                  page_table=FAKE, max_pages=2, lengths=FAKE, window=0, scale=0.1, gs_k=FAKE, gs_v=FAKE, O=FAKE, lse=FAKE, workspace=FAKE, ws_bytes=need,
                  stream=None)
    for bad in (dict(type=3), dict(type=-1), dict(Q=None), dict(ldq=1016), dict(B=-1), dict(q_heads=0), dict(kv_heads=0), dict(head_dim=0), dict(cache=None),
                dict(pages=-1), dict(pages=0), dict(page_size=0), dict(page_table=None), dict(max_pages=-1), dict(lengths=None), dict(window=-1),
                dict(scale=NAN), dict(scale=INF), dict(gs_k=None), dict(gs_v=None), dict(O=None)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(q_heads=7), dict(head_dim=32), dict(head_dim=96), dict(page_size=8), dict(max_pages=1 << 27), dict(ldq=1028), dict(q_heads=8192, ldq=1 << 20),
                dict(B=(1 << 20) + 1)):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(Q=FAKE + 8), dict(cache=FAKE + 2), dict(O=FAKE + 8), dict(workspace=FAKE + 4), dict(page_table=FAKE + 2), dict(lengths=FAKE + 1),
                dict(lse=FAKE + 2), dict(gs_v=FAKE + 3)):
        assert call(**bad) == MISALIGNED, bad
    assert call(workspace=None) == WORKSPACE and call(ws_bytes=need - 1) == WORKSPACE
    assert call(B=0) == OK
    for bad in ((-1, 8, 2, 128), (2, 0, 2, 128), (2, 8, 0, 128), (2, 8, 3, 128), (2, 8, 2, 80)):
        assert lib.qfp4_attention_decode_workspace_bytes(*bad) == 0, bad


def test_gemv(lib):
    call = caller(lib.qfp4_gemv_nt, fmt=1, M=2, N=100, K=256, X=FAKE, ldx=256, W=FAKE, W_sf=FAKE, gs=FAKE, D=FAKE, ldd=100, stream=None)
    for bad in (dict(fmt=2), dict(fmt=-1), dict(M=-1), dict(N=-1), dict(K=-128), dict(ldx=128), dict(ldd=99), dict(X=None), dict(W=None), dict(W_sf=None),
                dict(D=None)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(M=17), dict(K=192, ldx=256), dict(ldx=260), dict(N=(1 << 30) + 1, ldd=1 << 31), dict(K=1 << 31, ldx=1 << 31)):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(X=FAKE + 8), dict(W=FAKE + 4), dict(W_sf=FAKE + 8), dict(gs=FAKE + 2), dict(D=FAKE + 1)):
        assert call(**bad) == MISALIGNED, bad
    assert call(M=0) == OK and call(N=0, ldd=0) == OK


# ------------------------------------------------------- the binding's checks

BF16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


class Tensor:
    """What the binding asks of a tensor on the GPU."""
    is_cuda, device = True, "cuda"

    def __init__(self, dtype, *shape, stride=None):
        self.dtype, self.shape = dtype, torch.Size(shape)
        whole = [1] * len(shape)
        for i in range(len(shape) - 2, -1, -1):
            whole[i] = whole[i + 1] * shape[i + 1]
        self._stride = tuple(whole) if stride is None else stride

    def numel(self):
        return self.shape.numel()

    def stride(self):
        return self._stride

    def is_contiguous(self):
        return self._stride == Tensor(self.dtype, *self.shape)._stride

    @property
    def nbytes(self):
        return self.numel() * self.dtype.itemsize

    def data_ptr(self):
        return 1 << 40


@pytest.fixture
def calls(monkeypatch):
    made = []
    monkeypatch.setattr(qfp4, "_call", lambda name, *a: made.append((name, a)))
    monkeypatch.setattr(qfp4, "_stream", lambda s: None)
    return made


T, H, KV, D, PAGES, PAGE = 6, 4, 2, 128, 5, 16
NV_PAGE = 16 * 2 * (64 + 8) * KV
COMMON = dict(q_weight=Tensor(BF16, D), k_weight=Tensor(BF16, D), cos_sin=Tensor(F32, 32, D), positions=Tensor(I32, T))
QKV = Tensor(BF16, T, (H + 2 * KV) * D)
CASES = [
    (qfp4.gemv_nt, dict(fmt=qfp4.NVFP4, X=Tensor(BF16, 3, 256), W=Tensor(U8, 130, 128), W_sf=Tensor(U8, 256 * 16), gs_w=Tensor(F32, 1), D=Tensor(BF16, 3, 130))),
    (qfp4.qk_norm_rope, dict(QKV=QKV, q_heads=H, kv_heads=KV, Q_out=Tensor(BF16, T, H, D), K_out=Tensor(BF16, T, KV, D), **COMMON)),
    (qfp4.qk_norm_rope_backward, dict(QKV=QKV, q_heads=H, kv_heads=KV, dQ=Tensor(BF16, T, H, D), dK=Tensor(BF16, T, KV, D), dQKV=QKV, dq_weight=Tensor(F32, D),
                                      dk_weight=Tensor(F32, D), workspace=Tensor(U8, 1 << 20), **COMMON)),
    (qfp4.qk_norm_rope_cache, dict(QKV=QKV, q_heads=H, kv_heads=KV, Q_out=Tensor(BF16, T, H, D), type=qfp4.CACHE_NVFP4, cache=Tensor(U8, PAGES, NV_PAGE),
                                   page_size=PAGE, slots=Tensor(I32, T), gs_k=Tensor(F32, 1), gs_v=Tensor(F32, 1), **COMMON)),
    (qfp4.kv_cache_write, dict(type=qfp4.CACHE_NVFP4, K=Tensor(BF16, T, KV, D), V=Tensor(BF16, T, KV, D), slots=Tensor(I32, T), cache=Tensor(U8, PAGES, NV_PAGE),
                               page_size=PAGE, gs_k=Tensor(F32, 1), gs_v=Tensor(F32, 1))),
    (qfp4.kv_cache_read, dict(type=qfp4.CACHE_NVFP4, cache=Tensor(U8, PAGES, NV_PAGE), page_size=PAGE, slots=Tensor(I32, T), K_out=Tensor(BF16, T, KV, D),
                              V_out=Tensor(BF16, T, KV, D), gs_k=Tensor(F32, 1), gs_v=Tensor(F32, 1))),
    (qfp4.attention_decode, dict(type=qfp4.CACHE_NVFP4, Q=Tensor(BF16, 3, H, D), cache=Tensor(U8, PAGES, KV, NV_PAGE // KV), page_size=PAGE,
                                 page_table=Tensor(I32, 3, 2), lengths=Tensor(I32, 3), scale=0.1, O=Tensor(BF16, 3, H, D), workspace=Tensor(U8, 1 << 20),
                                 gs_k=Tensor(F32, 1), gs_v=Tensor(F32, 1), lse=Tensor(F32, 3, H))),
]


@pytest.mark.parametrize("fn,args", CASES, ids=lambda v: getattr(v, "__name__", ""))
def test_binding_refuses_what_does_not_fit(calls, fn, args):
    fn(**args)
    assert len(calls) == 1 and len(calls[0][1]) == len(qfp4.SIGNATURES[calls[0][0]][1])
    assert set(args) <= set(inspect.signature(fn).parameters)
    for name, t in args.items():
        if not isinstance(t, Tensor) or name == "workspace":
            continue
        wrong = [Tensor(torch.float64, *t.shape)]
        if name not in ("QKV", "cos_sin", "X", "Q", "K", "page_table"):     # the others' sizes go by these
            wrong.append(Tensor(t.dtype, *t.shape[:-1], t.shape[-1] - 1))
        if t.dtype is BF16 and len(t.shape) > 1:        # rows whose elements do not lie together
            wrong.append(Tensor(t.dtype, *t.shape, stride=tuple(reversed(t.stride()))))
        for w in wrong:
            with pytest.raises(ValueError):
                fn(**{**args, name: w})
    assert len(calls) == 1


def test_binding_takes_heads_of_a_projection(calls):
    """Rows that lie apart: strides are passed on."""
    ld = (H + 2 * KV) * D
    k, v = (Tensor(BF16, T, KV, D, stride=(ld, D, 1)) for _ in range(2))
    qfp4.kv_cache_write(qfp4.CACHE_NVFP4, k, v, Tensor(I32, T), Tensor(U8, PAGES, NV_PAGE), PAGE, Tensor(F32, 1), Tensor(F32, 1))
    assert calls[0][1][2] == ld and calls[0][1][4] == ld
    q = Tensor(BF16, T, H, D, stride=(ld, D, 1))
    qfp4.qk_norm_rope(QKV, H, KV, q, k)
    assert calls[1][1][15] == ld and calls[1][1][17] == ld
    with pytest.raises(ValueError):
        qfp4.qk_norm_rope(Tensor(BF16, T, (H + KV) * D - 16), H, KV, q, k)
    with pytest.raises(ValueError):
        qfp4.attention_decode(qfp4.CACHE_NVFP4, Tensor(BF16, 3, H, D), Tensor(U8, PAGES, KV, NV_PAGE // KV), PAGE, Tensor(I32, 2, 2), Tensor(I32, 3), 0.1,
                              Tensor(BF16, 3, H, D), Tensor(U8, 1 << 20), Tensor(F32, 1), Tensor(F32, 1))


def test_arguments_reach_the_library_as_they_are():
    """The packed form of a call says what the call itself says: float arguments
    among them, which travel as their bits."""
    if torch.cuda.is_available():
        pytest.skip("a call that is not refused would be launched with these addresses")
    lib = qfp4.load()
    heads = tuple(HEADS.values())
    values = {
        "qfp4_gemv_nt": (1, 2, 100, 256, FAKE, 256, FAKE, FAKE, FAKE, FAKE, 100, None),
        "qfp4_qk_norm_rope": (*heads, FAKE, 512, FAKE, 256, None),
        "qfp4_qk_norm_rope_cache": (*heads, FAKE, 512, 2, FAKE, 4, 16, FAKE, FAKE, FAKE, None),
        "qfp4_qk_norm_rope_backward": (*heads, FAKE, 512, FAKE, 256, FAKE, 1280, FAKE, FAKE, FAKE, 1 << 20, None),
        "qfp4_kv_cache_write": (2, FAKE, 256, FAKE, 256, 4, 2, 128, FAKE, FAKE, FAKE, FAKE, 4, 16, None),
        "qfp4_kv_cache_read": (2, FAKE, 4, 16, 2, 128, FAKE, 4, FAKE, FAKE, FAKE, 256, FAKE, 256, None),
        "qfp4_attention_decode": (2, FAKE, 1024, 2, 8, 2, 128, FAKE, 4, 16, FAKE, 2, FAKE, 0, 0.125, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 26, None),
    }
    assert set(values) == set(qfp4._LAYER_WORDS)
    for name, good in values.items():
        function, pack = qfp4._words[name]
        kinds = qfp4.SIGNATURES[name][1]
        assert len(kinds) == len(good)
        answers = set()
        for i, kind in enumerate(kinds):
            for wrong in ((NAN, -1.0, 1e39) if kind is qfp4._f32 else (-1, 0, 3, 7, FAKE + 2)):
                if kind is qfp4._f32 and wrong == 1e39:
                    wrong = INF
                args = list(good)
                args[i] = wrong
                plain = getattr(lib, name)(*args)
                packed = function(pack(*[0 if a is None else a for a in args]))
                assert plain == packed, (name, i, wrong)
                answers.add(plain)
        assert len(answers) > 2, name
