"""The INT8 key/value cache where one query, key or value is unlike its neighbours: what is
not finite stays where it is seen.  Tolerances are those of test_cache8_gpu."""
import pytest
import torch

from test_cache8_gpu import F32, I8, Paged8, tolerance
from test_layer_gpu import DEV, F64, attention_ref, gen, randn, within

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


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


def set_keys(p, i, codes, scale):
    """Sequence i's keys: codes [held, kv heads, D] and scales [held, kv heads]."""
    p.kc[i] = codes.to(F64) * scale.to(F64)[..., None]
    for j in range(-(-p.kvs[i] // p.page)):
        a, b = j * p.page, min(p.kvs[i], (j + 1) * p.page)
        p.cache.k[p.rows[i][j], :, :b - a] = codes[a:b].to(I8).transpose(0, 1)
        p.cache.k_scale[p.rows[i][j], :, :b - a] = scale[a:b].to(F32).transpose(0, 1)


# ------------------------------------------------------------- not finite ---
# Contexts of one block, of several, and cut between many CTAs.
LENGTHS = [100, 600, 40000]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", LENGTHS)
@pytest.mark.parametrize("new", [1, 5, 40])
def test_a_query_that_is_not_finite(new, n, D):
    """Its own row is NaN, however its keys are split; the others have their answers."""
    p = Paged8([new, 1], [n, 300], 2, 32, D, 1)
    q = randn(gen(2), p.T, 8, D)
    want, mag, dot = attention_ref(p, q, 8, D ** -0.5, 0.0, 0)
    tol = tolerance(p, want, mag, dot, n)
    t = new // 2
    q[t, 5, 3] = NAN
    q[new, 0] = INF
    out = qz().attention_paged(q, p.cache, p.seqs)
    bad = torch.zeros((p.T, 8), dtype=torch.bool, device=DEV)
    bad[t, 5] = bad[new, 0] = True
    assert bool(out[bad].isnan().all())
    within(out[~bad], want[~bad], tol[~bad], "out")


@pytest.mark.parametrize("scale", [NAN, INF])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", LENGTHS)
@pytest.mark.parametrize("new", [1, 5, 40])
def test_no_key_is_finite(new, n, D, scale):
    """Every key's row says that it was not finite: outputs of its sequence are NaN."""
    p = Paged8([new, 1], [n, 300], 2, 32, D, 3)
    q = randn(gen(4), p.T, 8, D)
    good = qz().attention_paged(q, p.cache, p.seqs)
    set_keys(p, 0, torch.zeros((n, 2, D), device=DEV), torch.full((n, 2), scale, device=DEV))
    out = qz().attention_paged(q, p.cache, p.seqs)
    assert bool(out[:new].isnan().all())
    assert torch.equal(out[new], good[new])
