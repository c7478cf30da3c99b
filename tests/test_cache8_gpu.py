"""The INT8 key/value cache against its definition in 64 bits: rows quantised as they are
written, read back, and attended over, at the sizes, masks and layouts where they can go
wrong.

Tolerances (U16, S16, U32 as for the fp16 cache): codes and scales enter exactly; a weight
times its value's scale is rounded once to fp16 (relative U16; below its range by 2^-25
where the largest is at least 2^6, so 2^-31 of the largest value for each key), logits are
fp32 sums of D products and two multiplications, the output is rounded once."""
import math

import pytest
import torch

from test_layer_gpu import DEV, F16, F64, S16, U16, U32, attention_ref, gen, i32, randn, within

pytestmark = pytest.mark.gpu

F32, I8 = torch.float32, torch.int8


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


class Paged8:
    """Sequences with new tokens `qs` and held tokens `kvs`, pages in random order; slots that
    hold no token have codes of 85 and scales that are NaN.  spread: of the scales, in
    powers of two."""

    def __init__(self, qs, kvs, hkv, page, D, seed, nhd=False, spare=2, before=0, spread=2.0,
                 size=0.01):
        g = gen(seed)
        self.qs, self.kvs, self.page, self.D, self.hkv = qs, kvs, page, D, hkv
        need = [-(-n // page) for n in kvs]
        n, width = sum(need) + spare, max(1, max(need, default=1)) + 1
        order = torch.randperm(n, generator=g, device=DEV).tolist()
        rows, at = [], 0
        for m in need:
            rows.append(order[at:at + m] + [-7] * (width - m))
            at += m
        shape = (n, page, hkv) if nhd else (n, hkv, page)

        def pool():
            c = torch.full(shape + (D,), 85, dtype=I8, device=DEV)
            s = torch.full(shape, float("nan"), dtype=F32, device=DEV)
            return (c.transpose(1, 2), s.transpose(1, 2)) if nhd else (c, s)

        (k, ks), (v, vs) = pool(), pool()
        self.kc, self.vc, self.rows = [], [], rows
        for i, m in enumerate(kvs):
            for c, s, to in ((k, ks, self.kc), (v, vs, self.vc)):
                codes = torch.randint(-127, 128, (m, hkv, D), generator=g, device=DEV).to(I8)
                scale = torch.exp2(torch.randn((m, hkv), generator=g, device=DEV) * spread / 2)
                scale *= size
                to.append(codes.to(F64) * scale.to(F64)[..., None])
                for j in range(need[i]):
                    a, b = j * page, min(m, (j + 1) * page)
                    c[rows[i][j], :, :b - a] = codes[a:b].transpose(0, 1)
                    s[rows[i][j], :, :b - a] = scale[a:b].transpose(0, 1)
        self.cache = qz().PagedKVInt8(k, v, ks, vs)
        cu = [before]
        for q in qs:
            cu.append(cu[-1] + q)
        self.cu, self.T = cu, cu[-1]
        self.seqs = qz().SeqBatch(i32(cu), i32(kvs), i32(rows).view(len(qs), width))


def tolerance(p, out, mag, dot, keys):
    vmax = max((float(v.abs().max()) for v in p.vc if v.numel()), default=0.0)
    return (U16 * (mag + out.abs()) + S16 + keys * 2.0 ** -31 * vmax
            + 2 * mag * ((p.D + 64) * U32 * (dot + 1) + keys * U32))


def check(qs, kvs, hq, hkv, D, page, softcap=0.0, window=0, scale=None, seed=1, nhd=False,
          qscale=1.0, before=0, spread=2.0, size=0.01):
    p = Paged8(qs, kvs, hkv, page, D, seed, nhd=nhd, before=before, spread=spread, size=size)
    q = randn(gen(seed + 1), p.T, hq, D, scale=qscale)
    ws = qz().attention_workspace(p.T, len(qs), hq, hkv, D)
    out = torch.full_like(q, float("nan"))
    got = qz().attention_paged(q, p.cache, p.seqs, scale=scale, softcap=softcap, window=window,
                               out=out, workspace=ws)
    assert got is out
    s = D ** -0.5 if scale is None else scale
    want, mag, dot = attention_ref(p, q, hq, s, softcap, window)
    assert bool(out[:before].isnan().all())  # rows outside every sequence keep their contents
    tol = tolerance(p, want, mag, dot, max(kvs))
    within(out[before:], want[before:], tol[before:], "out")
    again = qz().attention_paged(q, p.cache, p.seqs, scale=scale, softcap=softcap, window=window,
                                 workspace=ws)
    assert torch.equal(again[before:], out[before:])
    assert not bool(ws[:8192].any())  # the counters are left as they were
    return p, q, out


# ------------------------------------------------------------- attention ---
HEADS = [(1, 1), (8, 8), (6, 2), (8, 1), (5, 1), (32, 2)]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", HEADS)
def test_decode(hq, hkv, D):
    kvs = [1, 2, 15, 16, 17, 127, 128, 129, 255, 300, 1]
    check([1] * len(kvs), kvs, hq, hkv, D, 16)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", HEADS)
def test_drafts(hq, hkv, D):
    check([3, 2, 0, 4, 1], [3, 200, 40, 64, 333], hq, hkv, D, 32, seed=2)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", HEADS)
def test_chunks(hq, hkv, D):
    check([3, 1, 0, 33, 70, 5], [3, 200, 40, 64, 333, 129], hq, hkv, D, 32, seed=3)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("qs", [[4, 4], [5, 4], [8, 8], [9, 8], [57] + [1] * 7, [58] + [1] * 7])
def test_between_drafts_and_chunks(qs, D):
    """Rows around the number at which another kernel takes them, evenly and on one
    sequence."""
    check(qs, [700 + 57 * i for i in range(len(qs))], 8, 2, D, 32, seed=21)
    check(qs, [q + 3 * i for i, q in enumerate(qs)], 8, 2, D, 16, seed=22, window=40)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens", [[1, 2, 127, 128, 129], [513, 31], [1025]])
@pytest.mark.parametrize("hq,hkv", [(4, 4), (6, 2)])
def test_prompts(lens, hq, hkv, D):
    check(lens, lens, hq, hkv, D, 64, seed=4)


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("nhd", [False, True])
def test_pages(page, nhd):
    check([1, 40, 129], [page, page + 1, 3 * page + 130], 8, 2, 128, page, nhd=nhd, seed=5)
    check([1, 1, 2], [page * 2 - 1, 300, 1000], 2, 2, 64, page, nhd=nhd, seed=6)
    check([1, 2], [page * 2 + 1, 300], 4, 2, 256, page, nhd=nhd, seed=6)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [1, 2, 100, 128, 300, 5000])
def test_window(window, D):
    check([1, 1, 50, 200], [1, 1000, 500, 200], 4, 2, D, 16, window=window, seed=7)
    check([1, 1, 2], [1, 1000, 500], 4, 2, D, 16, window=window, seed=7)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 90])
def test_softcap(D, new):
    check([1, new], [700, 300], 4, 2, D, 32, softcap=50.0, qscale=8.0, seed=8)
    check([1, new], [700, 300], 4, 2, D, 32, softcap=2.0, window=64, seed=8)
    check([1, new], [700, 300], 4, 2, D, 32, softcap=200.0, qscale=8.0, seed=8)


@pytest.mark.parametrize("window", [0, 2**31 - 1, 2**31, 2**40])
def test_rows_that_see_nothing(window):
    p, q, out = check([2, 5, 140, 1], [0, 3, 10, 20], 4, 2, 128, 16, seed=9, window=window)
    assert not out[:2].any() and not out[2:4].any() and not out[7:7 + 130].any()
    assert bool(out[4:7].any()) and bool(out[7 + 130].any())
    p, q, out = check([1, 2, 1], [0, 1, 20], 4, 2, 128, 16, seed=9, window=window)
    assert not out[:2].any() and bool(out[2].any())


def test_rows_outside_sequences():
    check([1, 3], [50, 60], 4, 2, 64, 16, seed=10, before=3)
    check([40, 30], [50, 60], 8, 2, 64, 16, seed=10, before=3)


@pytest.mark.parametrize("new", [1, 64])
def test_peaked_and_scales(new):
    check([1, new], [2000, 1500], 8, 2, 128, 64, qscale=30.0, seed=11)
    check([1, new], [300, 300], 8, 2, 128, 64, scale=0.0, seed=12)
    check([1, new], [300, 300], 8, 2, 128, 64, scale=-0.2, seed=12)
    check([1, new], [300, 300], 8, 2, 128, 64, scale=-0.2, softcap=5.0, seed=12)


@pytest.mark.parametrize("size", [2.0 ** -31, 1e-6, 1.0])
@pytest.mark.parametrize("new", [1, 64])
def test_small_and_large_values(size, new):
    """Values from fp16's smallest to its largest: no weight is lost in its scale.  (Queries
    that keep the logits of large keys moderate.)"""
    for D in (64, 128, 256):
        check([1, new], [700, 300], 8, 2, D, 32, size=size, seed=13, qscale=min(1.0, 0.02 / size))
    check([1, new], [700, 300], 8, 2, 128, 32, size=size, spread=6.0, seed=13,
          qscale=min(1.0, 0.002 / size))


@pytest.mark.parametrize("new", [1, 100])
@pytest.mark.parametrize("order", [1, -1])
def test_values_that_grow_and_shrink(new, order):
    """Scales of the values that climb (fall) by 2^20 along the sequence, and rows of zeros."""
    p = Paged8([1, new], [1500, 1500], 1, 32, 128, 14, size=1.0, spread=0.0)
    ramp = torch.exp2(torch.linspace(-10, 6, 1500, device=DEV))
    ramp = ramp if order > 0 else ramp.flip(0)
    ramp[::7] = 0.0
    for i in range(2):
        codes = p.vc[i].clone()
        p.vc[i] = codes * ramp.to(F64)[:, None, None]
        p.kc[i] *= 2.0 ** -8
        for j in range(-(-1500 // 32)):
            a, b = j * 32, min(1500, j * 32 + 32)
            p.cache.v_scale[p.rows[i][j], :, :b - a] = ramp[a:b]
            p.cache.k_scale[p.rows[i][j], :, :b - a] = 2.0 ** -8
    q = randn(gen(15), p.T, 2, 128)
    out = qz().attention_paged(q, p.cache, p.seqs)
    want, mag, dot = attention_ref(p, q, 2, 128 ** -0.5, 0.0, 0)
    within(out, want, tolerance(p, want, mag, dot, 1500))


@pytest.mark.parametrize("new", [1, 150])
def test_rising_logits(new):
    """Keys whose logits climb by more than the running maximum may lag."""
    D, n = 128, 1200
    p = Paged8([1, new], [n, n], 1, 32, D, 13)
    ramp = torch.linspace(-3, 3, n, device=DEV)
    for i in range(2):
        p.kc[i] = (ramp.sign() * ramp.abs()).to(F64)[:, None, None].expand(n, 1, D).contiguous()
        for j in range(-(-n // 32)):
            a, b = j * 32, min(n, j * 32 + 32)
            p.cache.k[p.rows[i][j], :, :b - a] = ramp[a:b].sign().to(I8)[None, :, None]
            p.cache.k_scale[p.rows[i][j], :, :b - a] = ramp[a:b].abs()
    q = torch.ones((p.T, 2, D), dtype=F16, device=DEV)
    out = qz().attention_paged(q, p.cache, p.seqs, scale=0.25)
    want, mag, dot = attention_ref(p, q, 2, 0.25, 0.0, 0)
    within(out, want, tolerance(p, want, mag, dot, n))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_long_contexts_cut_between_ctas(D):
    check([1], [40000], 8, 1, D, 64, seed=14)
    check([1, 1, 1], [20001, 7, 12345], 4, 2, D, 128, seed=15)
    check([17, 2], [30000, 9000], 8, 2, D, 16, seed=16)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_tiles_of_several_blocks(D):
    check([1] * 160, [257 + (i * 29) % 300 for i in range(160)], 8, 8, D, 16, seed=50)
    check([i % 5 for i in range(120)], [300 + (i * 31) % 400 for i in range(120)], 24, 8, D, 64,
          window=290, seed=51)
    lens = [130 + (i * 41) % 300 for i in range(24)]
    check(lens, [n + (i % 3) * 200 for i, n in enumerate(lens)], 16, 8, D, 32, seed=52)


def test_many_sequences():
    n = 700
    check([1 + (i % 3 == 0) for i in range(n)], [1 + (i * 37) % 90 for i in range(n)], 4, 1, 64, 16,
          seed=17)


def test_strided_queries():
    for qs, kvs in (([4, 9], [100, 30]), ([40, 90], [100, 130])):
        p = Paged8(qs, kvs, 2, 16, 64, 18)
        qkv = randn(gen(19), p.T, 8 + 4, 64)
        big = torch.full((p.T, 20, 64), 7.0, dtype=F16, device=DEV)
        out = qz().attention_paged(qkv[:, :8], p.cache, p.seqs, out=big[:, 4:12])
        want = qz().attention_paged(qkv[:, :8].contiguous(), p.cache, p.seqs)
        assert torch.equal(out, want)
        assert bool((big[:, :4] == 7).all()) and bool((big[:, 12:] == 7).all())
        qh = qkv[:, :8].transpose(0, 1).contiguous().transpose(0, 1)  # heads ahead of tokens
        assert torch.equal(qz().attention_paged(qh, p.cache, p.seqs), want)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new,hq", [(4, 2), (8, 8), (100, 8)])
def test_rows_that_are_not_finite(new, hq, D, which, bad):
    """A new token's key or value that is not finite (scale so, codes 0): queries that see it
    get NaN; earlier ones of the step their own answer, or NaN beside such a value."""
    n, pos = 600, 600 - new // 2
    p = Paged8([new, 1], [n, 300], 2, 32, D, 60)
    page = p.rows[0][pos // 32]
    codes, scale = (p.cache.k, p.cache.k_scale) if which == "k" else (p.cache.v, p.cache.v_scale)
    codes[page, :, pos % 32] = 0
    scale[page, :, pos % 32] = bad
    q = randn(gen(61), p.T, hq, D)
    out = qz().attention_paged(q, p.cache, p.seqs)
    want, mag, dot = attention_ref(p, q, hq, D ** -0.5, 0.0, 0)
    first = new - (n - pos)  # new tokens before it
    assert bool(out[first:new].isnan().all())
    tol = tolerance(p, want, mag, dot, n)
    keep = torch.tensor([i for i in range(p.T) if not first <= i < new], device=DEV)
    got = out[keep].double()
    if which == "v":
        assert not bool(got[-1].isnan().any())  # (another sequence's)
        got = torch.where(got.isnan(), want[keep], got)
    within(got, want[keep], tol[keep], "out")


@pytest.mark.parametrize("new", [1, 40])
def test_bad_pages_read_as_zeros(new):
    p = Paged8([1, new], [40, 40], 2, 16, 64, 20)
    p.seqs.page_table[0, 1] = 1 << 30
    p.seqs.page_table[1, 0] = -1
    for x in (p.kc, p.vc):
        x[0][16:32] = 0
        x[1][:16] = 0
    q = randn(gen(21), p.T, 4, 64)
    out = qz().attention_paged(q, p.cache, p.seqs)
    assert qz().device_error() == 4
    want, mag, dot = attention_ref(p, q, 4, 0.125, 0.0, 0)
    within(out, want, tolerance(p, want, mag, dot, 40))


@pytest.mark.parametrize("new", [1, 40])
def test_length_beyond_the_table(new):
    p = Paged8([new], [48], 1, 16, 64, 22)
    short = qz().SeqBatch(p.seqs.cu_q, p.seqs.kv_len, p.seqs.page_table[:, :2].contiguous())
    p.kc[0][32:] = 0
    p.vc[0][32:] = 0
    q = randn(gen(23), new, 2, 64)
    out = qz().attention_paged(q, p.cache, short)
    assert qz().device_error() == 4
    want, mag, dot = attention_ref(p, q, 2, 0.125, 0.0, 0)
    within(out, want, tolerance(p, want, mag, dot, 48))


@pytest.mark.parametrize("new", [1, 100])
def test_captured_calls_on_other_streams(new):
    """Two captured calls with workspaces of their own, replayed side by side on streams other
    than their tensors', read the lengths that are there when they run."""
    both = []
    for seed in (30, 31):
        p = Paged8([new, 1], [900, 500], 2, 16, 128, seed)
        q = randn(gen(seed), p.T, 8, 128)
        want = [qz().attention_paged(q, p.cache, p.seqs)]
        lens = p.seqs.kv_len.clone()
        p.seqs.kv_len[1] = 137
        want.append(qz().attention_paged(q, p.cache, p.seqs))
        p.seqs.kv_len.copy_(lens)
        ws, out = qz().attention_workspace(p.T, 2, 8, 2, 128), torch.empty_like(q)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            qz().attention_paged(q, p.cache, p.seqs, out=out, workspace=ws)
        both.append((p, graph, side, out, want, (q, ws, lens)))
    for step in (0, 1, 0):
        for p, _, _, _, _, keep in both:
            p.seqs.kv_len.copy_(keep[2])
            if step:
                p.seqs.kv_len[1] = 137
        torch.cuda.synchronize()
        for _, graph, side, _, _, _ in both:
            with torch.cuda.stream(side):
                graph.replay()
        torch.cuda.synchronize()
        for _, _, _, out, want, _ in both:
            assert torch.equal(out, want[step])


# ---------------------------------------------------------------- append ---
def quantised(y):
    """(codes, scale) of fp32 rows by the rule, on the host (IEEE fp32)."""
    y = y.cpu()
    s = y.abs().amax(-1) / 127.0
    safe = torch.where(s > 0, s, 1.0)[..., None]
    return torch.round(y / safe).clamp(-127, 127).to(I8), s


def new_tokens(qs, kvs, hq, hkv, page, D, seed, nhd=False, before=0):
    p = Paged8(qs, kvs, hkv, page, D, seed, nhd=nhd, before=before)
    g = gen(seed + 1)
    qkv = randn(g, p.T, hq + 2 * hkv, D)
    return p, *qkv.split([hq, hkv, hkv], dim=1)


@pytest.mark.parametrize("hq,hkv,D,page,nhd,before", [
    (4, 4, 64, 8, False, 0), (8, 2, 128, 16, True, 0), (5, 1, 256, 64, False, 3),
    (64, 8, 128, 256, False, 0), (28, 4, 128, 32, True, 1), (1, 1, 64, 16, False, 0)])
@pytest.mark.parametrize("rotate", [True, False])
def test_append(hq, hkv, D, page, nhd, before, rotate):
    qs, kvs = [3, 0, 1, 40, 7], [3, 12, 300, 41, 129]
    p, q, k, v = new_tokens(qs, kvs, hq, hkv, page, D, 60 + D, nhd, before)
    k[before] = 0  # a row of zeros
    v[before] *= 2.0 ** -12  # and one near fp16's smallest
    rope = qz().rope_table(310, D) if rotate else None
    was = [t.clone() for t in (p.cache.k, p.cache.v, p.cache.k_scale, p.cache.v_scale)]
    q_out = torch.full((p.T, hq, D), 9.0, dtype=F16, device=DEV)
    qz().rope_append(q, k, v, p.cache, p.seqs, rope, q_out=q_out)
    assert bool((q_out[:before] == 9).all())
    half = D // 2
    touched = torch.zeros(was[2].shape, dtype=torch.bool, device=DEV)
    for i, (n, L) in enumerate(zip(qs, kvs)):
        rows = slice(p.cu[i], p.cu[i] + n)
        pos = torch.arange(L - n, L, device=DEV)

        def turn(x):
            x = x.to(F64)
            if not rotate:
                return x
            c, s = (rope[pos, None, a:a + half].to(F64) for a in (0, half))
            a, b = x[..., :half], x[..., half:]
            return torch.cat([a * c - b * s, b * c + a * s], -1)

        within(q_out[rows], turn(q[rows]), U16 * turn(q[rows]).abs() + 4 * U32 * 8 + S16, "q")
        pages = p.seqs.page_table[i, (pos // page).long()].long()
        slots = (pos % page).long()
        touched[pages, :, slots] = True
        for x, c, sc in ((turn(k[rows]), p.cache.k, p.cache.k_scale),
                         (v[rows].to(F64), p.cache.v, p.cache.v_scale)):
            codes, scale = quantised(x.float())
            assert torch.equal(sc[pages, :, slots].cpu(), scale)
            assert torch.equal(c[pages, :, slots].cpu(), codes)
    for t, w in zip((p.cache.k, p.cache.v, p.cache.k_scale, p.cache.v_scale), was):
        same = torch.where(touched.view(touched.shape + (1,) * (t.dim() - 3)), w, t)
        assert torch.equal(same.nan_to_num(-1.0) if t.is_floating_point() else same,
                           w.nan_to_num(-1.0) if t.is_floating_point() else w)


def test_append_codes_at_borders():
    """Values of which many lie on a half code: ties go to even."""
    D, T = 128, 64
    p, q, k, v = new_tokens([T], [T], 1, 1, 16, D, 70)
    v[:, 0, 0] = 127.0  # scale 1
    v[:, 0, 1:] = (torch.arange(T * (D - 1), device=DEV).view(T, D - 1) % 253 - 126) / 2
    qz().rope_append(q, k, v, p.cache, p.seqs, None)
    codes, _ = quantised(v.float())
    got = p.cache.v[p.seqs.page_table[0, :T // 16].long()].transpose(1, 2).reshape(T, 1, D)
    assert torch.equal(got.cpu(), codes)


def test_append_rows_that_are_not_finite():
    D = 128
    p, q, k, v = new_tokens([3], [3], 2, 2, 16, D, 71)
    k[0, 0, 5], k[1, 1, 100], v[2, 0, 0] = float("nan"), float("inf"), -float("inf")
    rope = qz().rope_table(4, D)
    qz().rope_append(q, k, v, p.cache, p.seqs, rope)
    page = int(p.seqs.page_table[0, 0])
    ks, vs = p.cache.k_scale[page, :, :3], p.cache.v_scale[page, :, :3]
    bad_k, bad_v = torch.zeros((2, 3), dtype=torch.bool), torch.zeros((2, 3), dtype=torch.bool)
    bad_k[0, 0] = bad_k[1, 1] = bad_v[0, 2] = True
    assert torch.equal(~ks.isfinite().cpu(), bad_k) and torch.equal(~vs.isfinite().cpu(), bad_v)
    assert not p.cache.k[page, 0, 0].any() and not p.cache.v[page, 0, 2].any()


def test_append_and_read_of_missing_places():
    p, q, k, v = new_tokens([5, 2], [3, 40], 2, 1, 16, 64, 72)
    p.seqs.page_table[1, 2] = 1 << 20
    was = p.cache.k.clone()
    q_out = qz().rope_append(q, k, v, p.cache, p.seqs, None)
    assert qz().device_error() == 4
    assert not q_out[:2].any() and not q_out[5:].any() and torch.equal(q_out[2:5], q[2:5])
    assert int((p.cache.k != was).any(-1).sum()) <= 3
    kk, vv = qz().cache_read(p.cache, p.seqs, p.T)
    assert qz().device_error() == 4
    assert not kk[:2].any() and not kk[5:].any() and not vv[5:].any() and bool(kk[2:5].any())
    far = qz().rope_table(38, 64)  # the second sequence's tokens lie behind its end
    p.seqs.page_table[1, 2] = 0
    q_out = qz().rope_append(q, k, v, p.cache, p.seqs, far)
    assert qz().device_error() == 4 and not q_out[5:].any()


# ------------------------------------------------------------------ read ---
@pytest.mark.parametrize("hkv,D,page,nhd,before", [
    (1, 64, 8, False, 0), (2, 128, 16, True, 0), (3, 256, 64, False, 5), (8, 128, 256, False, 1),
    (33, 64, 32, True, 0)])
def test_read(hkv, D, page, nhd, before):
    kvs = [1, 0, 300, 17, 64, 5]
    p = Paged8(kvs, kvs, hkv, page, D, 80, nhd=nhd, before=before)
    T = p.T + 3  # three rows behind the last sequence
    k = torch.full((T, hkv + 1, D + 8), 5.0, dtype=F16, device=DEV)
    v = torch.full((hkv, T, D), 5.0, dtype=F16, device=DEV).transpose(0, 1)
    got = qz().cache_read(p.cache, p.seqs, T, k=k[:, 1:, :D], v=v)
    assert got[1] is v
    for x, want in ((k[:, 1:, :D], p.kc), (v, p.vc)):
        want = torch.cat(want)
        assert torch.equal(x[before:p.T], want.float().to(F16))
        assert bool((x[:before] == 5).all()) and bool((x[p.T:] == 5).all())
    assert bool((k[:, 0] == 5).all()) and bool((k[..., D:] == 5).all())
    # the last tokens of each alone
    qs = [min(n, 2) for n in kvs]
    cu = [0]
    for n in qs:
        cu.append(cu[-1] + n)
    new = qz().SeqBatch(i32(cu), p.seqs.kv_len, p.seqs.page_table)
    kk, _ = qz().cache_read(p.cache, new, cu[-1])
    want = torch.cat([x[len(x) - n:] for x, n in zip(p.kc, qs)])
    assert torch.equal(kk, want.float().to(F16))


# ------------------------------------------------------- all of a step ---
def test_steps_of_a_cache_that_fills():
    """Prompts, then steps of one to three tokens: append, read back and attend, against the
    attention over what the rows stand for."""
    hq, hkv, D, page, S = 8, 2, 128, 16, 3
    cache = qz().PagedKVInt8.empty(40, hkv, page, D)
    table = torch.randperm(39, generator=gen(90), device=DEV)[:36].to(torch.int32).view(S, 12)
    rope, g, lens = qz().rope_table(200, D), gen(91), [0] * S
    held = [[torch.zeros((0, hkv, D), dtype=F64, device=DEV)] * 2 for _ in range(S)]
    for qs in ([50, 1, 130], [1, 1, 1], [2, 0, 1], [1, 3, 1], [30, 30, 30]):
        lens = [a + b for a, b in zip(lens, qs)]
        cu = [0, qs[0], qs[0] + qs[1], sum(qs)]
        seqs = qz().SeqBatch(i32(cu), i32(lens), table)
        q, k, v = (randn(g, sum(qs), h, D) for h in (hq, hkv, hkv))
        qz().rope_append(q, k, v, cache, seqs, rope, q_out=q)
        out = qz().attention_paged(q, cache, seqs)
        whole = qz().SeqBatch(i32([0, lens[0], lens[0] + lens[1], sum(lens)]), i32(lens), table)
        kk, vv = qz().cache_read(cache, whole, sum(lens))

        class P:
            pass
        P.qs, P.kvs, P.cu, P.hkv, P.D, P.kc, P.vc = qs, lens, cu, hkv, D, [], []
        at = 0
        for i, L in enumerate(lens):
            pages = table[i, :-(-L // page)].long()
            for codes, scale, to, half in ((cache.k, cache.k_scale, P.kc, kk),
                                           (cache.v, cache.v_scale, P.vc, vv)):
                x = codes[pages].to(F64) * scale[pages].to(F64)[..., None]
                to.append(x.transpose(1, 2).reshape(-1, hkv, D)[:L])
                within(half[at:at + L], to[-1], 2 * U16 * to[-1].abs() + S16)
            at += L
        want, mag, dot = attention_ref(P, q, hq, D ** -0.5, 0.0, 0)
        within(out, want, tolerance(P, want, mag, dot, max(lens)))
        # and what they stand for is the new rows, to half a step of a code
        for i in range(S):
            n = qs[i]
            if n:
                x = v[cu[i]:cu[i] + n].to(F64)
                step = x.abs().amax(-1, keepdim=True) / 127
                within(P.vc[i][lens[i] - n:], x, step * (0.5 + 127 * 4 * U32))


def test_refusals():
    p, q, k, v = new_tokens([2], [20], 2, 1, 16, 64, 95)
    c = p.cache
    for bad in [lambda: qz().PagedKVInt8(c.k.half(), c.v, c.k_scale, c.v_scale),
                lambda: qz().PagedKVInt8(c.k, c.v, c.k_scale.half(), c.v_scale),
                lambda: qz().PagedKVInt8(c.k, c.v, c.k_scale[:1], c.v_scale),
                lambda: qz().PagedKVInt8(c.k, c.v, c.k_scale.cpu(), c.v_scale),
                lambda: qz().cache_read(qz().PagedKV.empty(2, 1, 16, 64), p.seqs, 2),
                lambda: qz().cache_read(c, p.seqs, -1),
                lambda: qz().cache_read(c, p.seqs, 2, k=torch.empty((2, 1, 64), device=DEV)),
                lambda: qz().rope_append(q, k[..., :32], v, c, p.seqs, None),
                lambda: qz().attention_paged(q.float(), c, p.seqs)]:
        with pytest.raises(ValueError):
            bad()
    kk, vv = qz().cache_read(c, p.seqs, 0)
    assert kk.shape == (0, 1, 64) and vv.shape == (0, 1, 64)
    assert math.isclose(float(q[:0].sum()), 0.0)
