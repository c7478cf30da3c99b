"""Refusals of the INT8 cache's and the sampling entry points: arguments are validated on
the host before anything is enqueued.  No GPU needed (no call here reaches a launch)."""
import ctypes

import pytest

from test_layer_abi import ALIGN, INF, INVAL, NAN, OK, P, PO, PU, UNSUP, BAD_SEQS, seqs
from test_layer_abi import lib  # noqa: F401
from weight_only_quantized_dequant_gb300 import _lib


def cache8(**kw):
    a = dict(k=P, v=P, k_scale=P, v_scale=P, n_pages=4, page_size=16, n_kv_heads=2, head_dim=64,
             k_page=2048, k_head=1024, k_token=64, v_page=2048, v_head=1024, v_token=64,
             ks_page=32, ks_head=16, ks_token=1, vs_page=32, vs_head=16, vs_token=1)
    a.update(kw)
    return _lib.KvCacheInt8(**a)


BAD_CACHE8 = [(dict(k=None), INVAL), (dict(v=None), INVAL), (dict(k_scale=None), INVAL),
              (dict(v_scale=None), INVAL), (dict(n_pages=0), INVAL), (dict(n_kv_heads=0), INVAL),
              (dict(head_dim=0), INVAL), (dict(page_size=0), INVAL), (dict(k_page=-16), INVAL),
              (dict(vs_head=-1), INVAL), (dict(k_token=72), ALIGN), (dict(v_head=8), ALIGN),
              (dict(k=PU), ALIGN), (dict(v=PU), ALIGN), (dict(k_scale=0x10002), ALIGN),
              (dict(head_dim=80), UNSUP), (dict(head_dim=512), UNSUP), (dict(page_size=24), UNSUP),
              (dict(page_size=4), UNSUP), (dict(page_size=512), UNSUP),
              (dict(n_pages=1 << 31), UNSUP), (dict(n_kv_heads=4097), UNSUP)]


def test_struct_layouts():
    assert ctypes.sizeof(_lib.KvCacheInt8) == 20 * 8
    assert ctypes.sizeof(_lib.Sampling) == 48


def _append(lib, c=None, b=None, q=P, hq=4, qs=(256, 64), k=P, ks=(128, 64),  # noqa: F811
            v=P, vs=(128, 64), rope=P, rope_len=8, qo=P, qos=(256, 64)):
    return lib.qz_rope_append_int8(q, hq, *qs, k, *ks, v, *vs, rope, rope_len,
                                   ctypes.byref(c or cache8()), ctypes.byref(b or seqs()), qo,
                                   *qos, None)


def test_append(lib):  # noqa: F811
    for kw, want in BAD_CACHE8:
        assert _append(lib, c=cache8(**kw)) == want, kw
    for kw, want in BAD_SEQS:
        assert _append(lib, b=seqs(**kw)) == want, kw
    assert _append(lib, b=seqs(n_tokens=0)) == OK and _append(lib, b=seqs(n_seqs=0)) == OK
    assert _append(lib, k=None) == INVAL and _append(lib, v=None) == INVAL
    assert _append(lib, q=None) == INVAL and _append(lib, qo=None) == INVAL
    assert _append(lib, rope_len=-1) == INVAL and _append(lib, hq=0) == INVAL
    assert _append(lib, k=PU) == ALIGN and _append(lib, qs=(252, 64)) == ALIGN
    assert _append(lib, rope=PU) == ALIGN and _append(lib, qo=PU) == ALIGN


def test_read(lib):  # noqa: F811
    def f(c=None, b=None, k=P, ks=(128, 64), v=P, vs=(128, 64)):
        return lib.qz_cache_read_int8(ctypes.byref(c or cache8()), ctypes.byref(b or seqs()), k,
                                      *ks, v, *vs, None)
    for kw, want in BAD_CACHE8:
        assert f(c=cache8(**kw)) == want, kw
    for kw, want in BAD_SEQS:
        assert f(b=seqs(**kw)) == want, kw
    assert f(b=seqs(n_tokens=0)) == OK and f(b=seqs(n_seqs=0)) == OK
    assert f(k=None) == INVAL and f(v=None) == INVAL and f(ks=(-8, 64)) == INVAL
    assert f(k=PU) == ALIGN and f(vs=(128, 60)) == ALIGN


def _attention(lib, c=None, b=None, q=P, hq=4, qs=(256, 64), scale=0.125,  # noqa: F811
               cap=0.0, window=0, out=P, os_=(256, 64), ws=P, nbytes=1 << 40):
    return lib.qz_attention_paged_int8(q, hq, *qs, ctypes.byref(c or cache8()),
                                       ctypes.byref(b or seqs()), scale, cap, window, out, *os_,
                                       ws, nbytes, None)


def test_attention(lib):  # noqa: F811
    for kw, want in BAD_CACHE8:
        assert _attention(lib, c=cache8(**kw)) == want, kw
    for kw, want in BAD_SEQS:
        assert _attention(lib, b=seqs(**kw)) == want, kw
    assert _attention(lib, b=seqs(n_tokens=0)) == OK and _attention(lib, b=seqs(n_seqs=0)) == OK
    assert _attention(lib, hq=3) == INVAL and _attention(lib, hq=0) == INVAL
    assert _attention(lib, window=-1) == INVAL and _attention(lib, cap=-1.0) == INVAL
    for bad in (NAN, INF, -INF):
        assert _attention(lib, scale=bad) == INVAL and _attention(lib, cap=bad) == INVAL
    assert _attention(lib, q=None) == INVAL and _attention(lib, out=None) == INVAL
    assert _attention(lib, ws=None) == INVAL and _attention(lib, nbytes=15) == INVAL
    assert _attention(lib, q=PU) == ALIGN and _attention(lib, os_=(256, 60)) == ALIGN
    assert _attention(lib, ws=PU) == ALIGN


def test_sample(lib):  # noqa: F811
    def opts(**kw):
        return _lib.Sampling(**dict(dict(temperature_all=1.0, top_p_all=1.0), **kw))

    def f(x=P, kind=0, B=2, V=100, ld=100, u=P, o=None, tok=P, lp=P):
        return lib.qz_sample(x, kind, B, V, ld, u, ctypes.byref(o or opts()), tok, lp, None)

    assert f(B=0) == OK and f(B=0, x=None, u=None, tok=None) == OK
    assert f(B=-1) == INVAL and f(V=0) == INVAL and f(ld=99) == INVAL
    assert f(kind=3) == INVAL and f(kind=-1) == INVAL
    assert f(x=None) == INVAL and f(u=None) == INVAL and f(tok=None) == INVAL
    assert lib.qz_sample(P, 0, 2, 100, 100, P, None, P, P, None) == INVAL
    assert f(V=(1 << 18) + 1, ld=1 << 20) == UNSUP and f(B=(1 << 24) + 1) == UNSUP
    assert f(x=PO) == ALIGN and f(x=0x10002, kind=2) == ALIGN
    assert f(u=0x10002) == ALIGN and f(tok=0x10001) == ALIGN and f(lp=0x10002) == ALIGN
    for name in ("temperature", "top_k", "top_p", "min_p"):
        assert f(o=opts(**{name: 0x10002})) == ALIGN


@pytest.mark.parametrize("name", ["qz_rope_append_int8", "qz_cache_read_int8",
                                  "qz_attention_paged_int8"])
def test_missing_structs(lib, name):  # noqa: F811
    fn = getattr(lib, name)
    args = [None if t not in (ctypes.c_int64, ctypes.c_float, ctypes.c_size_t) else
            (0.0 if t is ctypes.c_float else 0) for t in fn.argtypes]
    assert fn(*args) == INVAL
