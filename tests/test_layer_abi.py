"""Refusals of the layer-glue entry points (norm, rotary append, paged
attention, adapters): arguments are validated on the host before anything is
enqueued.  No GPU needed (no call here reaches a launch)."""
import ctypes
import os

import pytest

from weight_only_quantized_dequant_gb300 import _lib

OK, INVAL, ALIGN, UNSUP = 0, 1, 2, 3
P, PU, PO = 0x10000, 0x10008, 0x10001  # 16-byte aligned, 8-byte aligned, odd
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from weight_only_quantized_dequant_gb300 import build
        build.build()
    return _lib.load()


def test_struct_layouts():
    assert ctypes.sizeof(_lib.KvCache) == 96
    assert ctypes.sizeof(_lib.SeqBatchArg) == 48
    assert ctypes.sizeof(_lib.LoraArg) == 96


def test_rmsnorm(lib):
    def f(x=P, ldx=64, r=None, ldr=0, w=P, bias=0.0, eps=1e-5, T=2, K=64, y=P, ldy=64, h=None,
          ldh=0):
        return lib.qz_rmsnorm(x, ldx, r, ldr, w, bias, eps, T, K, y, ldy, h, ldh, None)
    assert f(T=0) == OK and f(T=0, x=None, w=None, y=None) == OK
    assert f(x=None) == INVAL and f(w=None) == INVAL and f(y=None) == INVAL
    assert f(T=-1) == INVAL and f(K=0) == INVAL
    assert f(ldx=63) == INVAL and f(ldy=63) == INVAL
    assert f(r=P, ldr=63) == INVAL and f(h=P, ldh=63) == INVAL
    assert f(eps=-1.0) == INVAL and f(eps=NAN) == INVAL and f(bias=NAN) == INVAL
    assert f(x=PO) == ALIGN and f(y=PO) == ALIGN and f(r=PO, ldr=64) == ALIGN
    assert f(K=57345, ldx=57345, ldy=57345) == UNSUP
    assert f(T=(1 << 24) + 1) == UNSUP


def test_rmsnorm_int8(lib):
    def f(q=P, ldq=64, scale=P, T=2, K=64, x=P, ldx=64):
        return lib.qz_rmsnorm_int8(x, ldx, None, 0, P, 0.0, 1e-5, T, K, q, ldq, scale, None, 0,
                                   None)
    assert f(T=0) == OK
    assert f(q=None) == INVAL and f(scale=None) == INVAL and f(ldq=63) == INVAL
    assert f(x=None) == INVAL
    assert f(scale=0x10002) == ALIGN


def cache(**kw):
    a = dict(k=P, v=P, n_pages=4, page_size=16, n_kv_heads=2, head_dim=64, k_page=2048,
             k_head=1024, k_token=64, v_page=2048, v_head=1024, v_token=64)
    a.update(kw)
    return _lib.KvCache(**a)


def seqs(**kw):
    a = dict(n_seqs=1, n_tokens=1, cu_q=P, kv_len=P, page_table=P, ld_table=4)
    a.update(kw)
    return _lib.SeqBatchArg(**a)


BAD_CACHE = [(dict(k=None), INVAL), (dict(v=None), INVAL), (dict(n_pages=0), INVAL),
             (dict(n_kv_heads=0), INVAL), (dict(head_dim=0), INVAL), (dict(page_size=0), INVAL),
             (dict(k_page=-8), INVAL), (dict(k_token=60), ALIGN), (dict(v_head=4), ALIGN),
             (dict(k=PU), ALIGN), (dict(v=PU), ALIGN), (dict(head_dim=80), UNSUP),
             (dict(head_dim=512), UNSUP), (dict(page_size=24), UNSUP), (dict(page_size=4), UNSUP),
             (dict(page_size=512), UNSUP)]
BAD_SEQS = [(dict(n_seqs=-1), INVAL), (dict(n_tokens=-1), INVAL), (dict(ld_table=-1), INVAL),
            (dict(cu_q=None), INVAL), (dict(kv_len=None), INVAL), (dict(page_table=None), INVAL),
            (dict(cu_q=0x10002), ALIGN), (dict(page_table=0x10001), ALIGN),
            (dict(n_tokens=1 << 25), UNSUP), (dict(n_seqs=1 << 21), UNSUP)]


def _append(lib, c=None, b=None, q=P, hq=4, qs=(256, 64), k=P, ks=(128, 64), v=P, vs=(128, 64),
            rope=P, rope_len=8, qo=P, qos=(256, 64)):
    return lib.qz_rope_append(q, hq, *qs, k, *ks, v, *vs, rope, rope_len,
                              ctypes.byref(c or cache()), ctypes.byref(b or seqs()), qo, *qos,
                              None)


def test_rope_append(lib):
    for kw, want in BAD_CACHE:
        assert _append(lib, c=cache(**kw)) == want, kw
    for kw, want in BAD_SEQS:
        assert _append(lib, b=seqs(**kw)) == want, kw
    assert _append(lib, b=seqs(n_tokens=0)) == OK and _append(lib, b=seqs(n_seqs=0)) == OK
    assert _append(lib, k=None) == INVAL and _append(lib, v=None) == INVAL
    assert _append(lib, q=None) == INVAL                     # q_out without q
    assert _append(lib, qo=None) == INVAL                    # a rotation without q_out
    assert _append(lib, rope_len=-1) == INVAL and _append(lib, hq=0) == INVAL
    assert _append(lib, k=PU) == ALIGN and _append(lib, qs=(252, 64)) == ALIGN
    assert _append(lib, rope=PU) == ALIGN and _append(lib, qo=PU) == ALIGN


def _attention(lib, c=None, b=None, q=P, hq=4, qs=(256, 64), scale=0.125, cap=0.0, window=0,
               out=P, os_=(256, 64), ws=P, nbytes=1 << 40):
    return lib.qz_attention_paged(q, hq, *qs, ctypes.byref(c or cache()),
                                  ctypes.byref(b or seqs()), scale, cap, window, out, *os_, ws,
                                  nbytes, None)


def test_attention(lib):
    for kw, want in BAD_CACHE:
        assert _attention(lib, c=cache(**kw)) == want, kw
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


def test_attention_workspace_bytes(lib):
    f = lib.qz_attention_workspace_bytes
    assert f(1, 1, 8, 2, 128) > 0 and f(0, 0, 8, 2, 128) > 0
    assert f(1, 1, 8, 3, 128) == 0 and f(1, 1, 0, 1, 128) == 0 and f(1, 1, 8, 2, 96) == 0
    assert f(-1, 1, 8, 2, 128) == 0 and f(1, -1, 8, 2, 128) == 0


def lora(**kw):
    a = dict(a=P, b=P, scale=P, rank=None, n_adapters=3, R=16, K=64, N=32, a_adapter=1024,
             a_row=64, b_adapter=512, b_row=16)
    a.update(kw)
    return _lib.LoraArg(**a)


def test_lora(lib):
    def f(ad=None, index=P, T=2, x=P, ldx=64, y=P, ldy=32, out=P, ldo=32, ws=P, nbytes=1 << 40):
        return lib.qz_lora(ctypes.byref(ad or lora()), index, T, x, ldx, y, ldy, out, ldo, ws,
                           nbytes, None)
    assert f(T=0) == OK and f(T=-1) == INVAL
    for kw, want in [(dict(a=None), INVAL), (dict(b=None), INVAL), (dict(scale=None), INVAL),
                     (dict(R=0), INVAL), (dict(K=0), INVAL), (dict(N=0), INVAL),
                     (dict(n_adapters=-1), INVAL), (dict(a_row=63), INVAL), (dict(b_row=15), INVAL),
                     (dict(a_adapter=-1), INVAL), (dict(R=129), UNSUP), (dict(K=1 << 21), UNSUP),
                     (dict(N=1 << 21), UNSUP), (dict(a=PO), ALIGN), (dict(b=PO), ALIGN),
                     (dict(scale=0x10002), ALIGN), (dict(rank=0x10002), ALIGN)]:
        assert f(ad=lora(**kw)) == want, kw
    assert f(index=None) == INVAL and f(index=0x10002) == ALIGN
    assert f(x=None) == INVAL and f(y=None) == INVAL and f(out=None) == INVAL
    assert f(ldx=63) == INVAL and f(ldy=31) == INVAL and f(ldo=31) == INVAL
    assert f(x=PO) == ALIGN and f(out=PO) == ALIGN
    assert f(ws=None) == INVAL and f(nbytes=1) == INVAL and f(ws=PU) == ALIGN
    g = lib.qz_lora_workspace_bytes
    assert g(1, 1, 1) > 0 and g(0, 1, 1) > 0
    assert g(-1, 1, 1) == 0 and g(1, 0, 1) == 0 and g(1, 1, 0) == 0 and g(1, 1, 129) == 0
