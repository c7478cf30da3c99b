"""The Python side of the layer operators: handles, checks of arguments and what
a call hands to the library.  No GPU needed: tensors on the host stand for the
device's, and the library is a record of its calls."""
import dataclasses

import pytest
import torch

from weight_only_quantized_dequant_gb300 import _lib, layer

F16, F32, I32 = torch.float16, torch.float32, torch.int32


class Device:
    def __init__(self, index):
        self.index = index


class OnGpu:
    """A host tensor that says it lies on GPU `index`."""

    def __init__(self, t, index=0):
        self.t, self.device, self.is_cuda = t, Device(index), True

    def get_device(self):
        return self.device.index

    def __getattr__(self, name):
        return getattr(self.t, name)


class Stream:
    cuda_stream = 77


def gpu(*shape, dtype=F16, index=0):
    return OnGpu(torch.zeros(shape, dtype=dtype), index)


class Library:
    """Answers every call with status 0 and keeps its arguments."""

    def __init__(self):
        self.calls, self.before = [], {}

    def __getattr__(self, name):
        def call(*args):
            if name in self.before:
                self.before.pop(name)()
            self.calls.append((name, args))
            return 1 << 20 if name.endswith("_bytes") else 0
        return call


@pytest.fixture
def lib(monkeypatch):
    rec = Library()
    monkeypatch.setattr(_lib, "load", lambda: rec)
    monkeypatch.setattr(layer, "_current_device", lambda: 0, raising=False)
    return rec


def handles(S=2, pages=3, hkv=2, page=16, D=64):
    cache = layer.PagedKV(gpu(4, hkv, page, D), gpu(4, hkv, page, D))
    seqs = layer.SeqBatch(gpu(S + 1, dtype=I32), gpu(S, dtype=I32), gpu(S, pages, dtype=I32))
    return cache, seqs


def adapters(n=2, R=8, K=64, N=32):
    return layer.LoraAdapters(gpu(n, R, K), gpu(n, N, R), gpu(n, dtype=F32))


# ---------------------------------------------------------------- handles ---
@pytest.mark.parametrize("name", ["k", "v", "cu_q", "kv_len", "page_table", "a", "b", "scale",
                                  "rank"])
def test_a_handle_keeps_its_tensors(name):
    """The kernels get the addresses of the tensors that a handle was made of, so
    none of them can be exchanged (and freed) behind it."""
    for h in (*handles(), adapters()):
        if not hasattr(h, name):
            continue
        was = getattr(h, name)
        with pytest.raises(AttributeError):
            setattr(h, name, gpu(2, dtype=I32))
        assert getattr(h, name) is was


def test_a_handle_with_another_tensor_is_a_new_one():
    _, seqs = handles()
    n = gpu(2, dtype=I32)
    other = dataclasses.replace(seqs, kv_len=n)
    assert other.kv_len is n and other.cu_q is seqs.cu_q and seqs.kv_len is not n
    ad = adapters()
    assert dataclasses.replace(ad, rank=gpu(2, dtype=I32))._arg.rank is not None
    assert ad._arg.rank is None


def test_calls_that_share_sequences_keep_their_row_counts(lib):
    """The library runs without the interpreter's lock, so another thread may call
    with the same SeqBatch before it has read this call's arguments."""
    cache, seqs = handles()

    def append(T):
        q = gpu(T, 4, 64)
        layer.rope_append(q, gpu(T, 2, 64), gpu(T, 2, 64), cache, seqs, None, q_out=q,
                          stream=Stream)

    def attend(T):
        q = gpu(T, 4, 64)
        layer.attention_paged(q, cache, seqs, out=q, workspace=gpu(1 << 20, dtype=torch.uint8),
                              stream=Stream)

    lib.before = {"qz_rope_append": lambda: append(3), "qz_attention_paged": lambda: attend(4)}
    append(5)
    attend(6)
    append(2)
    rows = [a._obj.n_tokens for _, args in lib.calls for a in args
            if isinstance(getattr(a, "_obj", None), _lib.SeqBatchArg)]
    assert rows == [3, 5, 4, 6, 2]


# ---------------------------------------------------- devices, workspaces ---
def norm_args(**kw):
    return dict(dict(x=gpu(3, 64), weight=gpu(64), residual=gpu(3, 64), out=gpu(3, 64),
                     residual_out=gpu(3, 64), stream=Stream), **kw)


def int8_args(**kw):
    return norm_args(**dict(dict(out=gpu(3, 64, dtype=torch.int8), scale=gpu(3, dtype=F32)), **kw))


def append_args(**kw):
    cache, seqs = handles()
    return dict(dict(q=gpu(3, 4, 64), k=gpu(3, 2, 64), v=gpu(3, 2, 64), cache=cache, seqs=seqs,
                     rope=gpu(9, 64, dtype=F32), q_out=gpu(3, 4, 64), stream=Stream), **kw)


def attention_args(**kw):
    cache, seqs = handles()
    return dict(dict(q=gpu(3, 4, 64), cache=cache, seqs=seqs, out=gpu(3, 4, 64),
                     workspace=gpu(64, dtype=torch.uint8), stream=Stream), **kw)


def lora_args(**kw):
    return dict(dict(x=gpu(3, 64), y=gpu(3, 32), adapters=adapters(), index=gpu(3, dtype=I32),
                     out=gpu(3, 32), workspace=gpu(64, dtype=torch.uint8), stream=Stream), **kw)


CALLS = [(layer.rmsnorm, norm_args), (layer.rmsnorm_int8, int8_args),
         (layer.rope_append, append_args), (layer.attention_paged, attention_args),
         (layer.lora, lora_args)]
OPERANDS = [(f, make, n) for f, make in CALLS for n, v in make().items() if isinstance(v, OnGpu)]


def moved(t, index):
    return OnGpu(t.t, index)


@pytest.mark.parametrize("f,make", CALLS)
def test_operands_of_the_current_device_are_taken(lib, f, make):
    f(**make())
    assert len(lib.calls) == 1


@pytest.mark.parametrize("f,make,name", OPERANDS)
def test_operands_of_another_device_are_refused(lib, f, make, name):
    args = make()
    with pytest.raises(ValueError):
        f(**dict(args, **{name: moved(args[name], 1)}))
    assert not lib.calls


@pytest.mark.parametrize("f,make,name", OPERANDS)
def test_operands_on_the_host_are_refused(lib, f, make, name):
    args = make()
    with pytest.raises(ValueError):
        f(**dict(args, **{name: args[name].t}))
    assert not lib.calls


@pytest.mark.parametrize("f,make", CALLS)
def test_a_call_beside_the_current_device_is_refused(lib, monkeypatch, f, make):
    """The library launches on the current device, whatever the operands'."""
    monkeypatch.setattr(layer, "_current_device", lambda: 1, raising=False)
    with pytest.raises(ValueError):
        f(**make())
    assert not lib.calls


def test_handles_of_another_device_are_refused(lib):
    cache, seqs = handles()
    other = dataclasses.replace(cache, k=moved(cache.k, 1), v=moved(cache.v, 1))
    far = dataclasses.replace(seqs, cu_q=moved(seqs.cu_q, 1), kv_len=moved(seqs.kv_len, 1),
                              page_table=moved(seqs.page_table, 1))
    for f, make in CALLS[2:4]:
        for kw in (dict(cache=other), dict(seqs=far)):
            with pytest.raises(ValueError):
                f(**make(**kw))
    ad = adapters()
    away = layer.LoraAdapters(moved(ad.a, 1), moved(ad.b, 1), moved(ad.scale, 1))
    with pytest.raises(ValueError):
        layer.lora(**lora_args(adapters=away))
    assert not lib.calls
    # one handle, two devices
    for h in (cache, seqs, layer.LoraAdapters(ad.a, ad.b, ad.scale, gpu(2, dtype=I32))):
        for field in dataclasses.fields(h):
            t = getattr(h, field.name)
            if isinstance(t, OnGpu):
                with pytest.raises(ValueError):
                    dataclasses.replace(h, **{field.name: moved(t, 1)})


@pytest.mark.parametrize("f,make", CALLS[3:])
def test_workspaces(lib, f, make):
    f(**make(workspace=gpu(100, dtype=F32)))  # any type: its bytes count
    assert lib.calls[-1][1][-2] == 400
    for bad in (torch.zeros(64, dtype=torch.uint8), gpu(64, dtype=torch.uint8, index=1),
                OnGpu(torch.zeros(64, dtype=torch.uint8)[::2])):
        with pytest.raises(ValueError):
            f(**make(workspace=bad))
    assert len(lib.calls) == 1


# ---------------------------------------------------------------- strides ---
def strided(shape, stride, dtype=F16):
    n = 1 + sum((a - 1) * b for a, b in zip(shape, stride))
    return OnGpu(torch.zeros(n, dtype=dtype).as_strided(shape, stride))


def test_a_dimension_of_one_has_no_stride_of_its_own(lib):
    """torch reports any number there (a token's row out of a wider one); the kernels'
    rule of multiples of 8 is for strides that are used."""
    cache, seqs = handles(S=1)
    q, k = strided((1, 4, 64), (259, 64, 1)), strided((1, 2, 64), (131, 64, 1))
    layer.rope_append(q, k, k, cache, seqs, None, q_out=q, stream=Stream)
    layer.attention_paged(q, cache, seqs, out=q, workspace=gpu(64, dtype=torch.uint8),
                          stream=Stream)
    one = layer.PagedKV(*(strided((1, 1, 16, 64), (3, 5, 64, 1)) for _ in range(2)))
    q = strided((3, 1, 64), (64, 5, 1))
    layer.rope_append(q, q, q, one, seqs, None, q_out=q, stream=Stream)
    layer.attention_paged(q, one, seqs, out=q, workspace=gpu(64, dtype=torch.uint8),
                          stream=Stream)
    for name, a in lib.calls:
        a = [x for x in a if x is not Stream.cuda_stream]
        strides = [a[i] for i in ((2, 3, 5, 6, 8, 9, 15, 16) if name == "qz_rope_append"
                                  else (2, 3, 10, 11))]
        assert all(s % 8 == 0 and s >= 64 for s in strides), (name, strides)
        c = next(x._obj for x in a if isinstance(getattr(x, "_obj", None), _lib.KvCache))
        assert all(getattr(c, f"{t}_{n}") % 8 == 0 for t in "kv" for n in ("page", "head", "token"))
    # strides that are used are handed on as they are
    big = strided((3, 2, 64), (640, 320, 1))
    lib.calls.clear()
    layer.attention_paged(big, handles()[0], seqs, out=big, workspace=gpu(64, dtype=torch.uint8),
                          stream=Stream)
    assert lib.calls[0][1][2:4] == (640, 320)
