"""The layer-glue kernels against their definitions in 64 bits (plain torch
float64): norm with residual and INT8 rows, rotary append, paged attention,
low-rank adapters, at the sizes, masks and layouts where they can go wrong.

Tolerances.  U16 = 2^-11 is the relative error of one rounding to fp16 and S16
= 2^-24 its absolute error below the normal range; fp32 sums of n products
are within n * 2^-24 of the sum of magnitudes, fp32 functions (exp, rsqrt,
tanh) within a few 2^-22.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
U16, S16, U32 = 2.0 ** -11, 2.0 ** -24, 2.0 ** -24
F64, F16 = torch.float64, torch.float16


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
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(F16)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def within(got, want, tol, what=""):
    err = (got.to(F64) - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())}/{bad.numel()} outside, worst "
                           f"{float((err - tol).max()):.3e} over")


# ------------------------------------------------------------------ norm ---
def strided(t, pad, offset=0):
    """A copy of t whose rows are `pad` elements apart beyond their length,
    starting `offset` elements into its buffer."""
    T, K = t.shape
    buf = torch.full((T * (K + pad) + offset,), float("nan"), dtype=t.dtype, device=t.device) \
        if t.dtype == F16 else torch.zeros((T * (K + pad) + offset,), dtype=t.dtype, device=DEV)
    v = buf[offset:].view(T, K + pad)[:, :K]
    v.copy_(t)
    return v


def norm_ref(x, r, w, eps, bias):
    h = x.to(F64) + (0 if r is None else r.to(F64))
    return h, h / (h.square().mean(1, keepdim=True) + eps).sqrt() * (bias + w.to(F64))


NORM_SIZES = [(1, 1), (3, 7), (1, 8), (5, 64), (17, 1000), (2, 1024), (3, 1032), (130, 4096),
              (7, 4104), (2, 8192), (3, 8200), (2, 16384), (2, 16392), (1, 57344), (2, 57343)]


@pytest.mark.parametrize("T,K", NORM_SIZES)
@pytest.mark.parametrize("residual,bias", [(True, 0.0), (False, 1.0)])
def test_rmsnorm(T, K, residual, bias):
    g = gen(100 + K)
    x, w = randn(g, T, K, scale=3.0), randn(g, K) * 0.2 + 1
    r = randn(g, T, K, scale=5.0) if residual else None
    y, h = qz().rmsnorm(x, w, 1e-5, residual=r, w_bias=bias)
    hr, yr = norm_ref(x, r, w, 1e-5, bias)
    rel = U16 + (K + 64) * U32
    within(y, yr, rel * yr.abs() + S16, "y")
    if residual:
        within(h, hr, U16 * hr.abs() + S16, "h")
    else:
        assert h is x


@pytest.mark.parametrize("T,K", [(5, 64), (3, 1000), (2, 4096), (2, 20000)])
@pytest.mark.parametrize("pad,offset", [(8, 0), (1, 0), (8, 1), (24, 8)])
def test_rmsnorm_strides_and_alignment(T, K, pad, offset):
    g = gen(7)
    x, r, w = randn(g, T, K), randn(g, T, K), randn(g, K)
    want, hw = qz().rmsnorm(x, w, 1e-6, residual=r)
    xs, rs, ws = strided(x, pad, offset), strided(r, pad, offset), strided(w[None], 0, offset)[0]
    y, h = strided(torch.zeros_like(x), pad, offset), strided(torch.zeros_like(x), pad, offset)
    qz().rmsnorm(xs, ws, 1e-6, residual=rs, out=y, residual_out=h)
    hr, yr = norm_ref(x, r, w, 1e-6, 0.0)
    within(y, yr, (U16 + (K + 64) * U32) * yr.abs() + S16)
    assert torch.equal(h, hw)
    for t in (y, h):  # the gaps between rows keep their contents
        gap = t.as_strided((T - 1, pad), (K + pad, 1), t.storage_offset() + K)
        assert bool(gap.isnan().all())


@pytest.mark.parametrize("K", [512, 1001, 20000])
def test_rmsnorm_in_place(K):
    g = gen(8)
    x, r, w = randn(g, 6, K), randn(g, 6, K), randn(g, K)
    y0, h0 = qz().rmsnorm(x, w, residual=r)
    y1, h1 = qz().rmsnorm(x.clone(), w, residual=(r2 := r.clone()), residual_out=r2)
    assert torch.equal(h1, h0) and torch.equal(r2, h0) and torch.equal(y1, y0)
    x2 = x.clone()
    qz().rmsnorm(x2, w, residual=r, out=x2)
    assert torch.equal(x2, y0)


@pytest.mark.parametrize("T,K", NORM_SIZES)
def test_rmsnorm_int8(T, K):
    g = gen(200 + K)
    x, r, w = randn(g, T, K, scale=3.0), randn(g, T, K), randn(g, K)
    x[0] = 0
    r[0] = 0  # a row of zeros: scale 0, codes 0
    q, s, h = qz().rmsnorm_int8(x, w, 1e-5, residual=r)
    hr, yr = norm_ref(x, r, w, 1e-5, 0.0)
    sr = yr.abs().amax(1) / 127
    rel = (K + 64) * U32
    within(s, sr, (rel + 2 * U32) * sr)
    assert float(s[0]) == 0 and not q[0].any()
    # a code is the nearest to y / s, ties and y's own error aside
    live = sr > 0
    c = (yr / torch.where(live, sr, 1.0)[:, None])
    within(q, c, 0.5 + 127 * 3 * rel + 1e-6, "codes")
    assert int(q.abs().max()) <= 127
    if T > 1 or K > 1:
        assert bool((q[live].abs().amax(1) == 127).all())
    within(h, hr, U16 * hr.abs() + S16)


def test_rmsnorm_large_values_and_eps():
    # squares of fp16's largest value stay finite in fp32
    x = torch.full((2, 4096), 65504.0, dtype=F16, device=DEV)
    y, _ = qz().rmsnorm(x, torch.ones(4096, dtype=F16, device=DEV), 0.0)
    within(y, torch.ones_like(x, dtype=F64), torch.tensor(2 * U16, device=DEV))
    z, _ = qz().rmsnorm(torch.zeros_like(x), torch.ones(4096, dtype=F16, device=DEV), 1e-6)
    assert not z.any()


def test_norm_refusals():
    g = gen(1)
    x, w = randn(g, 4, 64), randn(g, 64)
    for bad in [lambda: qz().rmsnorm(x.cpu(), w), lambda: qz().rmsnorm(x.float(), w),
                lambda: qz().rmsnorm(x, w[:32]), lambda: qz().rmsnorm(x, w, residual=x[:3]),
                lambda: qz().rmsnorm(x.t(), w), lambda: qz().rmsnorm(x, w, out=x[:2]),
                lambda: qz().rmsnorm_int8(x, w, out=torch.empty_like(x)),
                lambda: qz().rmsnorm_int8(x, w, scale=torch.empty(3, device=DEV))]:
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(qz().QzError):
        qz().rmsnorm(x, w, eps=-1.0)
    y, _ = qz().rmsnorm(x[:0], w)
    assert y.shape == (0, 64)


# ----------------------------------------------------------- paged cache ---
class Paged:
    """Sequences with new tokens `qs` and held tokens `kvs`, pages in random
    order, every slot that holds no token NaN."""

    def __init__(self, qs, kvs, hkv, page, D, seed, nhd=False, spare=2, before=0):
        g = gen(seed)
        self.qs, self.kvs, self.page, self.D, self.hkv = qs, kvs, page, D, hkv
        need = [-(-n // page) for n in kvs]
        n = sum(need) + spare
        width = max(1, max(need, default=1)) + 1
        order = torch.randperm(n, generator=g, device=DEV).tolist()
        rows, at = [], 0
        for m in need:
            rows.append(order[at:at + m] + [-7] * (width - m))  # past the end: not read
            at += m
        shape = (n, page, hkv, D) if nhd else (n, hkv, page, D)
        k = torch.full(shape, float("nan"), dtype=F16, device=DEV)
        v = torch.full(shape, float("nan"), dtype=F16, device=DEV)
        if nhd:
            k, v = k.transpose(1, 2), v.transpose(1, 2)
        self.kc, self.vc = [], []
        for i, m in enumerate(kvs):
            kk, vv = randn(g, m, hkv, D), randn(g, m, hkv, D)
            self.kc.append(kk)
            self.vc.append(vv)
            for j in range(need[i]):
                a, b = j * page, min(m, (j + 1) * page)
                k[rows[i][j], :, :b - a] = kk[a:b].transpose(0, 1)
                v[rows[i][j], :, :b - a] = vv[a:b].transpose(0, 1)
        self.rows = rows
        self.cache = qz().PagedKV(k, v)
        cu = [before]
        for q in qs:
            cu.append(cu[-1] + q)
        self.cu = cu
        self.T = cu[-1]
        self.seqs = qz().SeqBatch(i32(cu), i32(kvs), i32(rows).view(len(qs), width))


def attention_ref(p, q, hq, scale, softcap, window):
    """(out, sum of weights * |v|, largest sum |q k| * scale) in 64 bits."""
    out = torch.zeros(q.shape, dtype=F64, device=DEV)
    mag = torch.zeros(q.shape, dtype=F64, device=DEV)
    dot = torch.zeros(q.shape[:2] + (1,), dtype=F64, device=DEV)
    G = hq // p.hkv
    for i, (n, L) in enumerate(zip(p.qs, p.kvs)):
        rows = slice(p.cu[i], p.cu[i] + n)
        pos = torch.arange(L - n, L, device=DEV)[:, None]
        j = torch.arange(L, device=DEV)[None, :]
        seen = j <= pos
        if window:
            seen &= j > pos - window
        for h in range(hq):
            k, v = p.kc[i][:, h // G].to(F64), p.vc[i][:, h // G].to(F64)
            qq = q[rows, h].to(F64)
            x = qq @ k.T * scale
            if softcap:
                x = softcap * torch.tanh(x / softcap)
            x = x.masked_fill(~seen, -math.inf)
            live = seen.any(1, keepdim=True)
            w = torch.where(live, torch.softmax(x, 1), 0.0) if L else x
            w = torch.nan_to_num(w)
            out[rows, h] = w @ v
            mag[rows, h] = w @ v.abs()
            if L:
                a = (qq.abs() @ k.abs().T * abs(scale)).masked_fill(~seen, 0.0)
                dot[rows, h] = a.amax(1, keepdim=True)
    return out, mag, dot


def attention_tol(out, mag, dot, D, keys):
    # weights rounded to fp16 (relative U16, absolute S16 / 2 below its normal
    # range), the output once more; logits are fp32 sums of D products, their
    # scaling, exp and the running rescales a few more roundings of |x| <= dot,
    # entering numerator and denominator
    return (U16 * (mag + out.abs()) + S16 + keys * S16 / 2 * 4.0
            + 2 * mag * ((D + 64) * U32 * (dot + 1) + keys * U32))


def check_attention(qs, kvs, hq, hkv, D, page, softcap=0.0, window=0, scale=None, seed=1,
                    nhd=False, qscale=1.0, before=0):
    p = Paged(qs, kvs, hkv, page, D, seed, nhd=nhd, before=before)
    q = randn(gen(seed + 1), p.T, hq, D, scale=qscale)
    ws = qz().attention_workspace(p.T, len(qs), hq, hkv, D)
    out = torch.full_like(q, float("nan"))
    got = qz().attention_paged(q, p.cache, p.seqs, scale=scale, softcap=softcap, window=window,
                               out=out, workspace=ws)
    assert got is out
    s = D ** -0.5 if scale is None else scale
    want, mag, dot = attention_ref(p, q, hq, s, softcap, window)
    assert bool(out[:before].isnan().all())  # rows outside every sequence keep their contents
    tol = attention_tol(want, mag, dot, D, max(kvs))
    within(out[before:], want[before:], tol[before:], "out")
    again = qz().attention_paged(q, p.cache, p.seqs, scale=scale, softcap=softcap, window=window,
                                 workspace=ws)
    assert torch.equal(again[before:], out[before:])
    return p, q, out


HEADS = [(1, 1), (8, 8), (6, 2), (8, 1), (5, 1), (32, 2)]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", HEADS)
def test_attention_decode(hq, hkv, D):
    kvs = [1, 2, 15, 16, 17, 127, 128, 129, 255, 300, 1]
    check_attention([1] * len(kvs), kvs, hq, hkv, D, 16)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", HEADS)
def test_attention_chunks(hq, hkv, D):
    check_attention([3, 1, 0, 33, 70, 5], [3, 200, 40, 64, 333, 129], hq, hkv, D, 32, seed=3)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens", [[1, 2, 127, 128, 129], [513, 31], [1025]])
@pytest.mark.parametrize("hq,hkv", [(4, 4), (6, 2)])
def test_attention_prompts(lens, hq, hkv, D):
    check_attention(lens, lens, hq, hkv, D, 64, seed=4)


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("nhd", [False, True])
def test_attention_pages(page, nhd):
    check_attention([1, 40, 129], [page, page + 1, 3 * page + 130], 8, 2, 128, page, nhd=nhd,
                    seed=5)
    check_attention([1, 20], [page * 2 - 1, 300], 2, 2, 64, page, nhd=nhd, seed=6)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [1, 2, 100, 128, 300, 5000])
def test_attention_window(window, D):
    check_attention([1, 1, 50, 200], [1, 1000, 500, 200], 4, 2, D, 16, window=window, seed=7)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_softcap(D):
    check_attention([1, 90], [700, 300], 4, 2, D, 32, softcap=50.0, qscale=8.0, seed=8)
    check_attention([1, 90], [700, 300], 4, 2, D, 32, softcap=2.0, window=64, seed=8)


def test_attention_rows_that_see_nothing():
    # nothing held; fewer held than new (the first new tokens lie before the cache)
    p, q, out = check_attention([2, 5, 140, 1], [0, 3, 10, 20], 4, 2, 128, 16, seed=9)
    assert not out[:2].any() and not out[2:4].any() and not out[7:7 + 130].any()
    assert bool(out[4:7].any()) and bool(out[7 + 130].any())


@pytest.mark.parametrize("window", [2**31 - 1, 2**31, 2**40])
def test_attention_window_longer_than_any_cache(window):
    # with tokens before the cache's first position, whose window starts below 32 bits
    check_attention([5, 140, 1], [3, 10, 300], 4, 2, 128, 16, window=window, seed=9)


def test_attention_rows_outside_sequences():
    check_attention([1, 3], [50, 60], 4, 2, 64, 16, seed=10, before=3)


def test_attention_peaked_and_scales():
    check_attention([1, 64], [2000, 1500], 8, 2, 128, 64, qscale=30.0, seed=11)
    check_attention([1, 64], [300, 300], 8, 2, 128, 64, scale=0.0, seed=12)
    check_attention([1, 64], [300, 300], 8, 2, 128, 64, scale=-0.2, seed=12)


def test_attention_rising_logits():
    """Keys whose logits climb by more than the running maximum may lag."""
    D, n = 128, 1200
    p = Paged([1, 150], [n, n], 1, 32, D, 13)
    for i in range(2):
        ramp = torch.linspace(-3, 3, n, device=DEV)[:, None, None].to(F16)
        p.kc[i] = (ramp * torch.ones((n, 1, D), dtype=F16, device=DEV)).contiguous()
        for j in range(-(-n // 32)):
            a, b = j * 32, min(n, j * 32 + 32)
            p.cache.k[p.rows[i][j], :, :b - a] = p.kc[i][a:b].transpose(0, 1)
    q = torch.ones((p.T, 2, D), dtype=F16, device=DEV)
    out = qz().attention_paged(q, p.cache, p.seqs, scale=0.25)
    want, mag, dot = attention_ref(p, q, 2, 0.25, 0.0, 0)
    within(out, want, attention_tol(want, mag, dot, D, n))


def test_attention_long_context_split():
    check_attention([1], [40000], 8, 1, 128, 64, seed=14)
    check_attention([1, 1, 1], [20001, 7, 12345], 4, 2, 256, 128, seed=15)
    check_attention([17, 2], [30000, 9000], 8, 2, 128, 16, seed=16)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_many_tiles_of_several_blocks(D):
    """Every SM walks through several tiles of a few key blocks each."""
    check_attention([1] * 160, [257 + (i * 29) % 300 for i in range(160)], 8, 8, D, 16, seed=50)
    check_attention([i % 5 for i in range(120)], [300 + (i * 31) % 400 for i in range(120)], 24, 8,
                    D, 64, window=290, seed=51)
    lens = [130 + (i * 41) % 300 for i in range(24)]
    check_attention(lens, [n + (i % 3) * 200 for i, n in enumerate(lens)], 16, 8, D, 32, seed=52)


def test_attention_many_sequences():
    n = 700
    check_attention([1 + (i % 3 == 0) for i in range(n)], [1 + (i * 37) % 90 for i in range(n)], 4,
                    1, 64, 16, seed=17)


def test_attention_strided_queries():
    p = Paged([4, 9], [100, 30], 2, 16, 64, 18)
    g = gen(19)
    qkv = randn(g, p.T, 8 + 4, 64)
    big = torch.full((p.T, 20, 64), 7.0, dtype=F16, device=DEV)
    out = qz().attention_paged(qkv[:, :8], p.cache, p.seqs, out=big[:, 4:12])
    want = qz().attention_paged(qkv[:, :8].contiguous(), p.cache, p.seqs)
    assert torch.equal(out, want)
    assert bool((big[:, :4] == 7).all()) and bool((big[:, 12:] == 7).all())
    # heads ahead of tokens
    qh = qkv[:, :8].transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(qz().attention_paged(qh, p.cache, p.seqs), want)


def test_attention_bad_pages_read_as_zeros():
    p = Paged([1, 5], [40, 40], 2, 16, 64, 20)
    p.seqs.page_table[0, 1] = 1 << 30
    p.seqs.page_table[1, 0] = -1
    p.kc[0][16:32] = 0
    p.vc[0][16:32] = 0
    p.kc[1][:16] = 0
    p.vc[1][:16] = 0
    q = randn(gen(21), p.T, 4, 64)
    out = qz().attention_paged(q, p.cache, p.seqs)
    assert qz().device_error() == 4
    want, mag, dot = attention_ref(p, q, 4, 0.125, 0.0, 0)
    within(out, want, attention_tol(want, mag, dot, 64, 40))


def test_attention_length_beyond_the_table():
    """kv_len past the page table's columns: the keys there read as zeros."""
    p = Paged([1], [48], 1, 16, 64, 22)
    short = qz().SeqBatch(p.seqs.cu_q, p.seqs.kv_len, p.seqs.page_table[:, :2].contiguous())
    p.kc[0][32:] = 0
    p.vc[0][32:] = 0
    q = randn(gen(23), 1, 2, 64)
    out = qz().attention_paged(q, p.cache, short)
    assert qz().device_error() == 4
    want, mag, dot = attention_ref(p, q, 2, 0.125, 0.0, 0)
    within(out, want, attention_tol(want, mag, dot, 64, 48))


def test_attention_own_stream_and_graph():
    p = Paged([1, 40], [900, 300], 2, 16, 128, 24)
    q = randn(gen(25), p.T, 8, 128)
    want = qz().attention_paged(q, p.cache, p.seqs)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = qz().attention_paged(q, p.cache, p.seqs, stream=s)  # allocates on s
    s.synchronize()
    assert torch.equal(got, want)
    ws = qz().attention_workspace(p.T, 2, 8, 2, 128)
    out = torch.zeros_like(q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qz().attention_paged(q, p.cache, p.seqs, out=out, workspace=ws)
    for kv in ([900, 300], [500, 41]):  # replays read the lengths of the moment
        p.seqs.kv_len.copy_(i32(kv))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, qz().attention_paged(q, p.cache, p.seqs))


def test_attention_workspace_shared_by_sizes():
    """One workspace serves calls of different sizes and shapes in turn."""
    ws = qz().attention_workspace(200, 8, 16, 2, 256)
    for qs, kvs, hq, hkv, D in [([1], [5000], 8, 1, 128), ([90, 1], [90, 4000], 8, 2, 64),
                                ([1] * 8, [700] * 8, 16, 2, 256), ([130], [3000], 4, 1, 256)]:
        p = Paged(qs, kvs, hkv, 32, D, 26)
        q = randn(gen(27), p.T, hq, D)
        out = qz().attention_paged(q, p.cache, p.seqs, workspace=ws)
        assert torch.equal(out, qz().attention_paged(q, p.cache, p.seqs))


def test_attention_refusals():
    p = Paged([1], [5], 2, 16, 64, 28)
    q = randn(gen(1), 1, 4, 64)
    Q = qz()
    for bad in [lambda: Q.attention_paged(q.float(), p.cache, p.seqs),
                lambda: Q.attention_paged(q.cpu(), p.cache, p.seqs),
                lambda: Q.attention_paged(q[..., :32], p.cache, p.seqs),
                lambda: Q.attention_paged(q, p.cache, p.seqs, out=q[:, :2]),
                lambda: Q.PagedKV(p.cache.k.float(), p.cache.v.float()),
                lambda: Q.PagedKV(p.cache.k.cpu(), p.cache.v.cpu()),
                lambda: Q.PagedKV(p.cache.k, p.cache.v[:1]),
                lambda: Q.SeqBatch(p.seqs.cu_q, p.seqs.kv_len, p.seqs.page_table.long()),
                lambda: Q.SeqBatch(p.seqs.cu_q[:1], p.seqs.kv_len, p.seqs.page_table),
                lambda: Q.attention_paged(q[:, :3].contiguous(), p.cache, p.seqs),
                lambda: Q.attention_workspace(1, 1, 8, 3, 64)]:
        with pytest.raises(ValueError):
            bad()
    for bad in [lambda: Q.attention_paged(q, p.cache, p.seqs, window=-1),
                lambda: Q.attention_paged(q, p.cache, p.seqs, scale=float("nan")),
                lambda: Q.attention_paged(q, p.cache, p.seqs,
                                          workspace=torch.zeros(1, dtype=torch.uint8, device=DEV))]:
        with pytest.raises(Q.QzError):
            bad()
    none = Q.SeqBatch(i32([0]), i32([]), torch.empty((0, 1), dtype=torch.int32, device=DEV))
    assert Q.attention_paged(q[:0], p.cache, none).shape == (0, 4, 64)


# ---------------------------------------------------------------- append ---
def rotate_ref(x, rope, pos):
    half = x.shape[-1] // 2
    c, s = rope[pos, None, :half].to(F64), rope[pos, None, half:].to(F64)
    a, b = x[..., :half].to(F64), x[..., half:].to(F64)
    return (torch.cat([a * c - b * s, b * c + a * s], -1),
            torch.cat([(a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()], -1))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (6, 2), (8, 8)])
@pytest.mark.parametrize("page,nhd", [(8, False), (16, True), (64, False)])
def test_rope_append(D, hq, hkv, page, nhd):
    qs, kvs = [1, 0, 5, 70, 1], [1, 4, 30, 70, 129]
    p = Paged(qs, kvs, hkv, page, D, 30, nhd=nhd, before=2)
    g = gen(31)
    qkv = randn(g, p.T, hq + 2 * hkv, D)
    q, k, v = qkv.split([hq, hkv, hkv], dim=1)
    rope = qz().rope_table(200, D)
    kw, vw = p.cache.k.clone(), p.cache.v.clone()
    out = torch.full((p.T, hq, D), 7.0, dtype=F16, device=DEV)
    got = qz().rope_append(q, k, v, p.cache, p.seqs, rope, q_out=out)
    assert got is out and bool((out[:2] == 7).all())
    seen = torch.zeros(p.cache.k.shape[0], page, dtype=torch.bool, device=DEV)
    for i, (n, L) in enumerate(zip(qs, kvs)):
        rows = slice(p.cu[i], p.cu[i] + n)
        pos = torch.arange(L - n, L, device=DEV)
        want, mag = rotate_ref(q[rows], rope, pos)
        within(out[rows], want, U16 * want.abs() + 3 * U32 * mag + S16)
        want, mag = rotate_ref(k[rows], rope, pos)
        pages = i32(p.rows[i])[pos // page].long()
        slots = pos % page
        within(p.cache.k[pages, :, slots], want, U16 * want.abs() + 3 * U32 * mag + S16)
        assert torch.equal(p.cache.v[pages, :, slots], v[rows])
        seen[pages, slots] = True
    rest = ~seen[:, None, :, None].expand(p.cache.k.shape)
    for now, was in ((p.cache.k, kw), (p.cache.v, vw)):  # nothing else was written
        assert torch.equal(now[rest].view(torch.int16), was[rest].view(torch.int16))
    # in place, and without a rotation
    q2 = q.contiguous()
    assert torch.equal(qz().rope_append(q2, k, v, p.cache, p.seqs, rope, q_out=q2)[2:], out[2:])
    q3 = qz().rope_append(q, k, v, p.cache, p.seqs, None)
    assert torch.equal(q3[2:], q[2:])
    last = p.cu[5] - 1  # the last sequence's token, position 128
    assert torch.equal(p.cache.k[p.rows[4][128 // page], :, 128 % page], k[last])


@pytest.mark.parametrize("hq,hkv", [(1, 1), (9, 3), (32, 8)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_rope_append_long_steps(D, hq, hkv):
    # more blocks than the GPU holds at once: several heads a thread
    qs, kvs, page = [2500, 0, 333], [2500, 7, 400], 64
    p = Paged(qs, kvs, hkv, page, D, 36)
    g = gen(37)
    q, k, v = randn(g, p.T, hq, D), randn(g, p.T, hkv, D), randn(g, p.T, hkv, D)
    rope = qz().rope_table(2500, D)
    out = qz().rope_append(q, k, v, p.cache, p.seqs, rope)
    for i, (n, L) in enumerate(zip(qs, kvs)):
        if n == 0:
            continue
        rows = slice(p.cu[i], p.cu[i] + n)
        pos = torch.arange(L - n, L, device=DEV)
        pages, slots = i32(p.rows[i])[pos // page].long(), pos % page
        want, mag = rotate_ref(q[rows], rope, pos)
        within(out[rows], want, U16 * want.abs() + 3 * U32 * mag + S16)
        want, mag = rotate_ref(k[rows], rope, pos)
        within(p.cache.k[pages, :, slots], want, U16 * want.abs() + 3 * U32 * mag + S16)
        assert torch.equal(p.cache.v[pages, :, slots], v[rows])
    assert qz().device_error() == 0


def test_rope_append_many_sequences():
    n, D = 1500, 64
    p = Paged([i % 3 for i in range(n)], [2 + i % 20 for i in range(n)], 1, 8, D, 32)
    g = gen(33)
    q, k, v = randn(g, p.T, 2, D), randn(g, p.T, 1, D), randn(g, p.T, 1, D)
    qz().rope_append(q, k, v, p.cache, p.seqs, None)
    t = 0
    for i in range(n):
        for j in range(p.qs[i]):
            pos = p.kvs[i] - p.qs[i] + j
            p.kc[i][pos] = k[t]
            t += 1
    want = torch.cat([p.kc[i] for i in range(n)])
    at = [(p.rows[i][j // 8], j % 8) for i in range(n) for j in range(p.kvs[i])]
    pages, slots = (torch.tensor(z, device=DEV) for z in zip(*at))
    assert torch.equal(p.cache.k[pages, :, slots], want)


def test_rope_append_outside_the_tables():
    p = Paged([3, 1], [2, 20], 1, 16, 64, 34)
    g = gen(35)
    q, k, v = randn(g, 4, 2, 64), randn(g, 4, 1, 64), randn(g, 4, 1, 64)
    # the first of three new tokens of a sequence that holds two: not stored, no error
    out = qz().rope_append(q, k, v, p.cache, p.seqs, None)
    assert qz().device_error() == 0
    assert not out[0].any() and torch.equal(out[1:], q[1:])
    # a page outside the pool, a position beyond the rotary table
    kw = p.cache.k.clone()
    p.seqs.page_table[1, 1] = p.cache.k.shape[0]
    out = qz().rope_append(q, k, v, p.cache, p.seqs, None)
    assert qz().device_error() == 4 and not out[3].any()
    p.seqs.page_table[1, 1] = p.rows[1][1]
    out = qz().rope_append(q, k, v, p.cache, p.seqs, qz().rope_table(19, 64))
    assert qz().device_error() == 4 and not out[3].any()
    assert torch.equal(p.cache.k[p.rows[1][1], :, 3], kw[p.rows[1][1], :, 3])


# ------------------------------------------------------------------ LoRA ---
def lora_ref(x, y, a, b, scale, rank, index):
    out, mag = y.to(F64).clone(), torch.zeros(y.shape, dtype=F64, device=DEV)
    for t, i in enumerate(index):
        if 0 <= i < a.shape[0]:
            r = a.shape[1] if rank is None else max(0, min(a.shape[1], rank[i]))
            A, B, s = a[i, :r].to(F64), b[i, :, :r].to(F64), float(scale[i])
            out[t] += s * (B @ (A @ x[t].to(F64)))
            mag[t] = abs(s) * (B.abs() @ (A.abs() @ x[t].to(F64).abs()))
    return out, mag


def check_lora(T, K, N, R, n, index, rank=None, seed=40, pad=0, offset=0, wide=False):
    g = gen(seed)
    x, y = randn(g, T, K), randn(g, T, N)
    a, b = randn(g, n, R, K, scale=K ** -0.5), randn(g, n, N, R, scale=0.5)
    if wide:  # adapters as parts of larger buffers
        a = torch.cat([a, torch.full_like(a, float("nan"))], 2)[:, :, :K]
        b = torch.cat([b, torch.full_like(b, float("nan"))], 2)[:, :, :R]
    scale = torch.rand((n,), generator=g, device=DEV) + 0.5
    ad = qz().LoraAdapters(a, b, scale, None if rank is None else i32(rank))
    xs, ys = (strided(x, pad, offset), strided(y, pad, offset)) if pad or offset else (x, y)
    out = strided(torch.zeros_like(y), pad, offset) if pad or offset else None
    got = qz().lora(xs, ys, ad, i32(index), out=out)
    want, mag = lora_ref(x, y, a, b, scale, rank, index)
    within(got, want, U16 * want.abs() + S16 + (K + R + 16) * U32 * mag, "out")
    y2 = ys.clone() if out is None else ys
    qz().lora(xs, y2, ad, i32(index), out=y2)  # in place, same bits
    assert torch.equal(y2, got)


def runs(T, run, n):
    return [-1 if (t // run) % 5 == 4 else (t // run) % n for t in range(T)]


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 33, 64, 200])
@pytest.mark.parametrize("R", [1, 8, 13, 16, 64, 128])
def test_lora_rows_and_ranks(T, R):
    check_lora(T, 512, 384, R, 7, runs(T, 1, 7))
    check_lora(T, 512, 384, R, 3, runs(T, 11, 3))


@pytest.mark.parametrize("K,N", [(1, 1), (7, 9), (64, 8), (200, 1000), (1000, 200), (4096, 130),
                                 (8192, 64), (57, 8200), (12000, 16)])
@pytest.mark.parametrize("R", [8, 5])
def test_lora_sizes(K, N, R):
    check_lora(19, K, N, R, 4, runs(19, 3, 4))


@pytest.mark.parametrize("T", [127, 128, 129, 500, 2100, 4500])
def test_lora_rows_in_any_order(T):
    # rows of an adapter far apart, over several sorted segments; more adapters
    # than bins of the sort; every row the same one
    g = torch.Generator().manual_seed(T)
    mixed = torch.randint(-1, 9, (T,), generator=g).tolist()
    check_lora(T, 128, 136, 24, 9, mixed, rank=[24, 0, 3, 8, 16, 24, 99, 1, 17])
    wide = [-1 if i % 7 == 6 else i * 523 % 1500 for i in range(T)]
    check_lora(T, 64, 72, 8, 1500, wide)
    check_lora(T, 64, 72, 8, 2, [1] * T)
    check_lora(T, 64, 72, 8, 2, [-1] * T)


def test_lora_indices_outside_the_pool_in_any_order():
    g = gen(46)
    T = 300
    x, y = randn(g, T, 64), randn(g, T, 64)
    ad = qz().LoraAdapters(randn(g, 3, 8, 64), randn(g, 3, 64, 8), torch.ones(3, device=DEV))
    idx = [(t % 7) - 2 for t in range(T)]  # -2 .. 4
    out = qz().lora(x, y, ad, i32(idx))
    assert qz().device_error() == 4
    for t, a in enumerate(idx):
        assert torch.equal(out[t], y[t]) == (a < 0 or a > 2)


def test_lora_mixed_ranks():
    check_lora(60, 1024, 512, 64, 6, runs(60, 2, 6), rank=[64, 32, 0, 1, 17, 99])
    check_lora(300, 1024, 512, 32, 3, runs(300, 70, 3), rank=[32, 8, 24])


def test_lora_strides_and_alignment():
    check_lora(20, 256, 128, 16, 4, runs(20, 2, 4), pad=8)
    check_lora(20, 256, 128, 16, 4, runs(20, 2, 4), pad=3, offset=1)
    check_lora(20, 256, 128, 16, 4, runs(20, 2, 4), wide=True)
    check_lora(1, 256, 128, 16, 4, [2], wide=True)


def test_lora_no_adapter_is_a_copy():
    g = gen(41)
    x, y = randn(g, 40, 128), randn(g, 40, 96)
    ad = qz().LoraAdapters(randn(g, 2, 8, 128), randn(g, 2, 96, 8), torch.ones(2, device=DEV))
    assert torch.equal(qz().lora(x, y, ad, i32([-1] * 40)), y)
    # rows without an adapter keep their bits beside rows with one
    idx = [-1 if t % 2 else 1 for t in range(40)]
    out = qz().lora(x, y, ad, i32(idx))
    assert torch.equal(out[1::2], y[1::2])


def test_lora_index_outside_the_pool():
    g = gen(42)
    x, y = randn(g, 4, 64), randn(g, 4, 64)
    ad = qz().LoraAdapters(randn(g, 2, 8, 64), randn(g, 2, 64, 8), torch.ones(2, device=DEV))
    out = qz().lora(x, y, ad, i32([2, 0, -5, 1]))
    assert qz().device_error() == 4
    assert torch.equal(out[0], y[0]) and torch.equal(out[2], y[2])
    assert not torch.equal(out[1], y[1])


def test_lora_large_inner_values():
    """u far beyond fp16's range, brought back by a small B."""
    g = gen(43)
    x, y = randn(g, 18, 1024, scale=300.0), randn(g, 18, 64)
    a, b = randn(g, 2, 16, 1024, scale=20.0), randn(g, 2, 64, 16, scale=1e-3)
    ad = qz().LoraAdapters(a, b, torch.full((2,), 1e-3, device=DEV))
    idx = runs(18, 1, 2)
    got = qz().lora(x, y, ad, i32(idx))
    want, mag = lora_ref(x, y, a, b, ad.scale, None, idx)
    within(got, want, U16 * want.abs() + S16 + (1024 + 32) * U32 * mag)


def test_lora_own_stream():
    g = gen(44)
    x, y = randn(g, 33, 512), randn(g, 33, 256)
    ad = qz().LoraAdapters(randn(g, 4, 16, 512), randn(g, 4, 256, 16), torch.ones(4, device=DEV))
    idx = i32(runs(33, 2, 4))
    want = qz().lora(x, y, ad, idx)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = qz().lora(x, y, ad, idx, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("T", [20, 260])
def test_lora_in_a_graph(T):
    # captured once, replayed with other rows and indices
    g = gen(47)
    ad = qz().LoraAdapters(randn(g, 5, 16, 192), randn(g, 5, 320, 16), torch.ones(5, device=DEV))
    x, y, idx = randn(g, T, 192), randn(g, T, 320), i32(runs(T, 3, 5))
    out, ws = torch.empty_like(y), qz().lora_workspace(T, 192, 16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        qz().lora(x, y, ad, idx, out=out, workspace=ws)
    for k in range(3):
        x.copy_(randn(g, T, 192))
        idx.copy_(i32([(t * (k + 2)) % 6 - 1 for t in range(T)]))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, qz().lora(x, y, ad, idx))


def test_lora_refusals():
    g = gen(45)
    x, y = randn(g, 4, 64), randn(g, 4, 32)
    a, b, sc = randn(g, 2, 8, 64), randn(g, 2, 32, 8), torch.ones(2, device=DEV)
    Q = qz()
    ad = Q.LoraAdapters(a, b, sc)
    idx = i32([0, 1, 0, -1])
    for bad in [lambda: Q.LoraAdapters(a, b[:, :, :4], sc), lambda: Q.LoraAdapters(a, b[:1], sc),
                lambda: Q.LoraAdapters(a.float(), b, sc), lambda: Q.LoraAdapters(a, b, sc[:1]),
                lambda: Q.LoraAdapters(a.cpu(), b.cpu(), sc),
                lambda: Q.lora(x[:, :32], y, ad, idx), lambda: Q.lora(x, y[:3], ad, idx),
                lambda: Q.lora(x, y, ad, idx.long()), lambda: Q.lora(x, y, ad, idx[:3]),
                lambda: Q.lora(x, y, ad, idx, out=y[:, :16])]:
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(Q.QzError):
        Q.lora(x, y, ad, idx, workspace=torch.empty(1, dtype=torch.uint8, device=DEV))
    assert Q.lora(x[:0], y[:0], ad, idx[:0]).shape == (0, 32)
