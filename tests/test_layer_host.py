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
