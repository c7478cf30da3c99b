"""The layer operators where their depth tells: calls of many rows and long contexts,
with bounds that a lost block of keys or a product in too few bits does not pass."""
import pytest
import torch

import layer_cases as C

pytestmark = pytest.mark.gpu

DEV = "cuda"
F16, F64 = torch.float16, torch.float64


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from weight_only_quantized_dequant_gb300 import build
    build.build()


@pytest.fixture(autouse=True)
def _no_error():
    qz().device_error()
    yield
    assert qz().device_error() == 0


def qz():
    import weight_only_quantized_dequant_gb300 as m
    return m


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(F16)


def within(got, want, tol):
    err = (got.to(F64) - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (f"{int(bad.sum())}/{bad.numel()} outside, worst "
                           f"{float((err - tol).max()):.3e} over")


# --------------------------------------------------------------- adapters ---
def shifted(t, offset):
    """t in a buffer that it starts `offset` elements into."""
    buf = torch.empty((t.numel() + offset,), dtype=t.dtype, device=t.device)
    return buf[offset:].view(t.shape).copy_(t)


@pytest.mark.parametrize("T,run,n,R,K,N,mixed,offset", C.ADAPTERS)
def test_lora_many_rows(T, run, n, R, K, N, mixed, offset):
    g = gen(60)
    x, y = randn(g, T, K), randn(g, T, N)
    a, b = randn(g, n, R, K, scale=K ** -0.5), randn(g, n, N, R, scale=0.5)
    scale = torch.rand((n,), generator=g, device=DEV) + 0.5
    rank = [max(1, R >> (i % 3)) for i in range(n)] if mixed else None
    index = C.adapter_index(T, run, n)
    x, y, a, b = (shifted(t, offset) for t in (x, y, a, b))
    ad = qz().LoraAdapters(a, b, scale, rank and torch.tensor(rank, dtype=torch.int32, device=DEV))
    idx = torch.tensor(index, dtype=torch.int32, device=DEV)
    got = qz().lora(x, y, ad, idx)
    within(got, *C.adapter_reference(x, y, a, b, scale, rank, index))
    assert torch.equal(qz().lora(x, y, ad, idx, out=y), got)  # in place, same bits


@pytest.mark.parametrize("K", [1024, 2048, 4096, 4104, 8192])
@pytest.mark.parametrize("T,R,N", [(1, 2, 64), (19, 16, 200), (64, 100, 136), (500, 16, 4096),
                                   (1500, 64, 4096)])
def test_lora_inner_vector_keeps_its_bits(T, R, N, K):
    x, y, a, b, index, want = C.cancelling_adapters(T, 3, R, K, N, DEV)
    assert torch.equal(want.to(F16).to(F64), want)
    ad = qz().LoraAdapters(a, b, torch.ones(3, device=DEV))
    assert torch.equal(qz().lora(x, y, ad, index), want.to(F16))
