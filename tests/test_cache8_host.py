"""The Python side of the INT8 cache and of sampling: handles, checks of arguments and what
a call hands to the library.  No GPU needed (see test_layer_host)."""
import dataclasses

import pytest
import torch

from test_layer_host import F16, F32, I32, OnGpu, Stream, gpu, handles, moved, strided
from test_layer_host import lib  # noqa: F401
from weight_only_quantized_dequant_gb300 import _lib, layer

I8 = torch.int8


def cache8(pages=4, hkv=2, page=16, D=64):
    return layer.PagedKVInt8(gpu(pages, hkv, page, D, dtype=I8), gpu(pages, hkv, page, D, dtype=I8),
                             gpu(pages, hkv, page, dtype=F32), gpu(pages, hkv, page, dtype=F32))


def append_args(**kw):
    return dict(dict(q=gpu(3, 4, 64), k=gpu(3, 2, 64), v=gpu(3, 2, 64), cache=cache8(),
                     seqs=handles()[1], rope=gpu(9, 64, dtype=F32), q_out=gpu(3, 4, 64),
                     stream=Stream), **kw)


def attention_args(**kw):
    return dict(dict(q=gpu(3, 4, 64), cache=cache8(), seqs=handles()[1], out=gpu(3, 4, 64),
                     workspace=gpu(64, dtype=torch.uint8), stream=Stream), **kw)


def read_args(**kw):
    return dict(dict(cache=cache8(), seqs=handles()[1], n_tokens=3, k=gpu(3, 2, 64),
                     v=gpu(3, 2, 64), stream=Stream), **kw)


def sample_args(**kw):
    return dict(dict(logits=gpu(3, 50), u=gpu(3, dtype=F32), out=gpu(3, dtype=I32),
                     logprob=gpu(3, dtype=F32), stream=Stream), **kw)


CALLS = [(layer.rope_append, append_args, "qz_rope_append_int8"),
         (layer.attention_paged, attention_args, "qz_attention_paged_int8"),
         (layer.cache_read, read_args, "qz_cache_read_int8"),
         (layer.sample, sample_args, "qz_sample")]
OPERANDS = [(f, make, n) for f, make, _ in CALLS for n, v in make().items()
            if isinstance(v, OnGpu)]


@pytest.mark.parametrize("f,make,name", CALLS)
def test_operands_of_the_current_device_are_taken(lib, f, make, name):  # noqa: F811
    f(**make())
    assert [c[0] for c in lib.calls] == [name] and lib.calls[0][1][-1] == Stream.cuda_stream


@pytest.mark.parametrize("f,make,name", OPERANDS)
def test_operands_elsewhere_are_refused(lib, f, make, name):  # noqa: F811
    args = make()
    for t in (moved(args[name], 1), args[name].t):
        with pytest.raises(ValueError):
            f(**dict(args, **{name: t}))
    assert not lib.calls


@pytest.mark.parametrize("f,make,name", CALLS)
def test_a_call_beside_the_current_device_is_refused(lib, monkeypatch, f, make, name):  # noqa: F811
    monkeypatch.setattr(layer, "_current_device", lambda: 1, raising=False)
    with pytest.raises(ValueError):
        f(**make())
    assert not lib.calls


def test_handles(lib):  # noqa: F811
    c = cache8()
    for name in ("k", "v", "k_scale", "v_scale"):
        with pytest.raises(AttributeError):
            setattr(c, name, getattr(c, name))
        with pytest.raises(ValueError):
            dataclasses.replace(c, **{name: moved(getattr(c, name), 1)})
    far = layer.PagedKVInt8(*(moved(getattr(c, n), 1) for n in ("k", "v", "k_scale", "v_scale")))
    for f, make, _ in CALLS[:3]:
        with pytest.raises(ValueError):
            f(**make(cache=far))
    with pytest.raises(ValueError):
        layer.cache_read(**read_args(cache=handles()[0]))  # fp16 rows need no reading back
    for bad in (dict(k=gpu(4, 2, 16, 64)), dict(v=gpu(4, 2, 8, 64, dtype=I8)),
                dict(k_scale=gpu(4, 2, 16)), dict(v_scale=gpu(4, 2, 8, dtype=F32)),
                dict(k=OnGpu(torch.zeros((4, 2, 64, 16), dtype=I8).transpose(2, 3)))):
        with pytest.raises(ValueError):
            dataclasses.replace(c, **bad)


def test_a_cache_decides_by_its_kind(lib):  # noqa: F811
    """Classes derived from a cache's are that kind of cache."""
    class Mine(layer.PagedKV):
        pass

    class Mine8(layer.PagedKVInt8):
        pass

    a, b = handles()[0], cache8()
    caches = (Mine(a.k, a.v), Mine8(b.k, b.v, b.k_scale, b.v_scale))
    for f, make, name in CALLS[:2]:
        for c in caches:
            f(**make(cache=c))
        assert [c[0] for c in lib.calls[-2:]] == [name[:-len("_int8")], name]


def test_strides_of_a_cache(lib):  # noqa: F811
    """Strides are handed on as they are, and a dimension of one has none of its own."""
    nhd = layer.PagedKVInt8(
        *(OnGpu(torch.zeros((4, 16, 2, 64), dtype=I8).transpose(1, 2)) for _ in range(2)),
        *(OnGpu(torch.zeros((4, 16, 2)).transpose(1, 2)) for _ in range(2)))
    a = nhd._arg
    assert (a.k_page, a.k_head, a.k_token) == (2048, 64, 128)
    assert (a.vs_page, a.vs_head, a.vs_token) == (32, 1, 2)
    one = layer.PagedKVInt8(*(strided((1, 1, 16, 64), (3, 5, 64, 1), I8) for _ in range(2)),
                            *(strided((1, 1, 16), (7, 9, 1), F32) for _ in range(2)))
    a = one._arg
    assert all(getattr(a, f"{t}_{n}") % 16 == 0 for t in "kv" for n in ("page", "head", "token"))
    assert a.ks_token == 1


def test_calls_that_share_sequences_keep_their_row_counts(lib):  # noqa: F811
    seqs = handles()[1]

    def read(n):
        layer.cache_read(**read_args(seqs=seqs, n_tokens=n, k=gpu(n, 2, 64), v=gpu(n, 2, 64)))

    lib.before = {"qz_cache_read_int8": lambda: read(4)}
    read(6)
    rows = [x._obj.n_tokens for _, args in lib.calls for x in args
            if isinstance(getattr(x, "_obj", None), _lib.SeqBatchArg)]
    assert rows == [4, 6]


def test_sampling_options(lib):  # noqa: F811
    layer.sample(**sample_args(temperature=0.5, top_k=7, top_p=0.25, min_p=0.125))
    o = lib.calls[-1][1][6]._obj
    assert (o.temperature, o.top_k, o.top_p, o.min_p) == (None,) * 4
    assert (o.temperature_all, o.top_k_all, o.top_p_all, o.min_p_all) == (0.5, 7, 0.25, 0.125)
    for kind, dtype in enumerate((F16, torch.bfloat16, F32)):
        layer.sample(**sample_args(logits=gpu(3, 50, dtype=dtype)))
        assert lib.calls[-1][1][1] == kind and lib.calls[-1][1][2:5] == (3, 50, 50)
    layer.sample(**sample_args(logits=strided((3, 50), (64, 1))))
    assert lib.calls[-1][1][4] == 64
    n = len(lib.calls)
    for bad in (dict(logits=gpu(3, 50, dtype=torch.float64)), dict(logits=gpu(3)),
                dict(logits=gpu(3, 0)), dict(logits=strided((3, 50), (1, 3))),
                dict(u=gpu(2, dtype=F32)), dict(u=gpu(3)), dict(out=gpu(3, dtype=F32)),
                dict(logprob=gpu(3)), dict(top_k=2 ** 31)):
        with pytest.raises(ValueError):
            layer.sample(**sample_args(**bad))
    assert len(lib.calls) == n
