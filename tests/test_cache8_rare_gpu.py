"""The INT8 key/value cache where one query, key or value is unlike its neighbours: what is
not finite stays where it is seen, and what is very large or very small leaves the others
their own precision.  Tolerances are those of test_cache8_gpu."""
import pytest
import torch

from test_cache8_gpu import F32, I8, Paged8, new_tokens, quantised, tolerance
from test_layer_gpu import DEV, F16, F64, Paged, attention_ref, gen, randn, within

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


def codes_like(p, i, seed):
    return torch.randint(-127, 128, (p.kvs[i], p.hkv, p.D), generator=gen(seed), device=DEV)


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


# --------------------------------------------------------- large and small ---
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("softcap", [0.0, 50.0])
@pytest.mark.parametrize("new,n", [(3, 70), (64, 64), (64, 700), (150, 150)])
def test_a_key_far_above_its_neighbours(new, n, softcap, D):
    """The last token's key is 2^25 times the others'.  Queries before it do not see it, and
    attend over small keys (their own queries are large)."""
    p = Paged8([new], [n], 2, 32, D, 5, spread=0.0)
    scale = torch.full((n, 2), 1.5e-5, device=DEV)
    scale *= 1 + torch.rand((n, 2), generator=gen(6), device=DEV)
    scale[-1] = 500.0
    set_keys(p, 0, codes_like(p, 0, 7), scale)
    q = randn(gen(8), p.T, 8, D, scale=1500.0)
    out = qz().attention_paged(q, p.cache, p.seqs, softcap=softcap)
    want, mag, dot = attention_ref(p, q, 8, D ** -0.5, softcap, 0)
    tol = tolerance(p, want, mag, dot, n)
    assert float(want[:-1].abs().median()) > 20 * float(tol[:-1].median())
    within(out, want, tol, "out")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("first", [25.0, 40.0, 60.0])
@pytest.mark.parametrize("new", [3, 64, 150])
def test_small_keys_beside_a_large_one_that_repels(new, first, D):
    """All logits are below zero.  Keys of logits near -first, then blocks with a large key,
    whose weight is zero, and small keys, whose logits are the largest of all."""
    n = 400
    p = Paged8([new], [n], 1, 32, D, 9, spread=0.0)
    codes = torch.randint(40, 128, (n, 1, D), generator=gen(10), device=DEV)
    q = (torch.rand((p.T, 4, D), generator=gen(11), device=DEV) * 256 + 256).to(F16)
    one = float(q[0, 0].double().sum()) * 84 * D ** -0.5  # the logit of a key of scale 1
    scale = torch.full((n, 1), first / one, device=DEV)
    scale[200:] = 2.0 / one
    scale[[210, 300, 350]] = 500.0
    set_keys(p, 0, codes, scale)
    out = qz().attention_paged(-q, p.cache, p.seqs)
    want, mag, _ = attention_ref(p, -q, 4, D ** -0.5, 0.0, 0)
    # (a large key's weight is 0, and its products enter no other logit: the small ones' bound)
    p.kc[0] = torch.where(scale[..., None] < 1, p.kc[0], 0.0)
    _, _, dot = attention_ref(p, -q, 4, D ** -0.5, 0.0, 0)
    within(out, want, tolerance(p, want, mag, dot, n), "out")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("scale", [1e-16, -1e-25, 1e-37, 1e-44])
@pytest.mark.parametrize("new", [2, 64, 150])
def test_logits_that_vanish(new, scale, D):
    """A tiny scale, over keys that are ordinary, zero or tiny: every seen key has the same
    weight, and the masked ones none."""
    n = 200
    p = Paged8([new, new, new], [n, n, n], 2, 32, D, 12)
    set_keys(p, 1, torch.zeros((n, 2, D), device=DEV), torch.zeros((n, 2), device=DEV))
    set_keys(p, 2, codes_like(p, 2, 13), torch.full((n, 2), 2.0 ** -60, device=DEV))
    q = randn(gen(14), p.T, 8, D)
    out = qz().attention_paged(q, p.cache, p.seqs, scale=scale)
    want, mag, dot = attention_ref(p, q, 8, scale, 0.0, 0)
    within(out, want, tolerance(p, want, mag, dot, n), "out")


# -------------------------------------------------------------- workspaces ---
@pytest.mark.parametrize("D", [64, 128, 256])
def test_both_caches_share_a_workspace(D):
    """Calls over fp16 and INT8 rows, of single tokens, drafts and chunks, one after the other
    with one workspace, whose contexts are cut between CTAs."""
    hq, hkv, page = 8, 2, 64
    ws = qz().attention_workspace(200, 3, hq, hkv, D)
    calls = []
    shapes = [([1], [30000]), ([3, 1], [9000, 20000]), ([70, 1], [9000, 5000])]
    for i, (qs, kvs) in enumerate(shapes):
        for kind in (Paged, Paged8):
            p = kind(qs, kvs, hkv, page, D, 20 + i)
            q = randn(gen(30 + i), p.T, hq, D)
            calls.append((p, q, qz().attention_paged(q, p.cache, p.seqs)))
    for order in (calls, calls[::-1], calls[::2] + calls[1::2]):
        got = [qz().attention_paged(q, p.cache, p.seqs, workspace=ws) for p, q, _ in order]
        for o, (_, _, want) in zip(got, order):
            assert torch.equal(o, want)
    assert not bool(ws[:8192].any())


# ------------------------------------------------------------------ append ---
@pytest.mark.parametrize("D", [64, 128, 256])
def test_rotated_keys_are_rounded_once(D):
    """Rows of two values that rotate into one another, by any two fp32 factors: the larger
    result decides the scale, to the last bit.  (Products are exact in 64 bits, and so are
    sums of products of about one size: one rounding to fp32 is left.)"""
    T, page = 4096, 64
    p, q, k, v = new_tokens([T], [T], 1, 2, page, D, 40)
    g = gen(41)
    half = D // 2
    rope = torch.rand((T, D), generator=g, device=DEV) + 0.5
    rope[::2] *= torch.sign(torch.randn((T // 2, D), generator=g, device=DEV))
    t = torch.arange(T, device=DEV)
    at = t % half
    k.zero_()
    for h in range(2):
        for j in (at, at + half):
            k[t, h, j] = (torch.rand((T,), generator=g, device=DEV) + 0.5).to(F16)
    qz().rope_append(q, k, v, p.cache, p.seqs, rope)
    x = k.to(F64)
    c, s = rope[:, None, :half].to(F64), rope[:, None, half:].to(F64)
    a, b = x[..., :half], x[..., half:]
    x = torch.cat([a * c - b * s, b * c + a * s], -1)
    codes, scale = quantised(x.float())
    pages = p.seqs.page_table[0, :T // page].long()
    assert torch.equal(p.cache.k_scale[pages].transpose(1, 2).reshape(T, 2).cpu(), scale)
    got = p.cache.k[pages].transpose(1, 2).reshape(T, 2, D)
    assert torch.equal(got.cpu(), codes)
