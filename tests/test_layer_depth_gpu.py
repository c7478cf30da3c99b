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


# ------------------------------------------------------------------- norm ---
@pytest.mark.parametrize("K,pad", [(64, 0), (1000, 0), (4096, 0), (4096, 1), (16384, 0),
                                   (20000, 0)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_rmsnorm_int8_shows_what_is_not_finite(K, pad, bad):
    """A row with a NaN or an infinity gets a scale that is not finite: rmsnorm's row
    holds a NaN too.  The other rows are what they are without it."""
    g = gen(70)
    x, w = randn(g, 9, K + pad)[:, :K], randn(g, K)
    q0, s0, _ = qz().rmsnorm_int8(x, w, 1e-5)
    for at in (0, K // 3, K - 1):
        y = torch.empty((9, K + pad), dtype=F16, device=DEV)[:, :K].copy_(x)
        y[4, at] = bad
        q, s, _ = qz().rmsnorm_int8(y, w, 1e-5)
        assert not bool(qz().rmsnorm(y, w, 1e-5)[0][4].isfinite().all())
        assert not bool(s[4].isfinite()) and not q[4].any()
        keep = torch.arange(9, device=DEV) != 4
        assert torch.equal(q[keep], q0[keep]) and torch.equal(s[keep], s0[keep])
    r = torch.zeros_like(x)
    r[4, 0] = bad  # through the residual
    assert not bool(qz().rmsnorm_int8(x, w, 1e-5, residual=r)[1][4].isfinite())
    v = w.clone()
    v[K // 2] = bad  # through the weight: every row
    q, s, _ = qz().rmsnorm_int8(x, v, 1e-5)
    assert not bool(s.isfinite().any()) and not bool(q.any())


@pytest.mark.parametrize("K", [64, 1000, 4096, 20000])
def test_rmsnorm_int8_rows_of_zeros_without_eps(K):
    x, w = torch.zeros((3, K), dtype=F16, device=DEV), torch.ones((K,), dtype=F16, device=DEV)
    x[1, K // 2] = 2.0
    q, s, _ = qz().rmsnorm_int8(x, w, 0.0)
    assert not bool(s[::2].any()) and not bool(q[::2].any())
    assert int(q[1, K // 2]) == 127 and bool(s[1] > 0)


# -------------------------------------------------------------- attention ---
def paged(ks, vs, page, D, hkv, nan=True):
    """A cache of the sequences' keys and values, pages in random order, NaN elsewhere."""
    need = [-(-k.shape[0] // page) for k in ks]
    order = torch.randperm(sum(need) + 2, generator=gen(90), device=DEV)
    kc = torch.full((sum(need) + 2, hkv, page, D), float("nan"), dtype=F16, device=DEV)
    vc = torch.full_like(kc, float("nan"))
    table = torch.full((len(ks), max(need) + 1), -7, dtype=torch.int32, device=DEV)
    at = 0
    for i, (k, v) in enumerate(zip(ks, vs)):
        pages = order[at:at + need[i]]
        at += need[i]
        table[i, :need[i]] = pages
        j = torch.arange(k.shape[0], device=DEV)
        kc[pages[j // page], :, j % page] = k
        vc[pages[j // page], :, j % page] = v
    return qz().PagedKV(kc, vc), table


def batch(qs, kvs, table):
    cu = torch.tensor([0] + qs, device=DEV).cumsum(0).to(torch.int32)
    return qz().SeqBatch(cu, torch.tensor(kvs, dtype=torch.int32, device=DEV), table)


@pytest.mark.parametrize("qs,kvs,hq,hkv,D,page,window", C.CONTEXTS)
def test_attention_takes_every_block_once(qs, kvs, hq, hkv, D, page, window):
    q, ks, vs = C.signal_inputs(qs, kvs, hq, hkv, D, 91, DEV)
    cache, table = paged(ks, vs, page, D, hkv)
    got = qz().attention_paged(q, cache, batch(qs, kvs, table), window=window)
    within(got, *C.signal_reference(q, ks, vs, qs, kvs, hq, window))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,window", [(1, 300), (1, 1), (140, 200), (3, 128)])
def test_attention_at_the_last_position(D, n, window):
    """2^31 - 1 tokens held: the last slot of the last block lies past them."""
    L, page, hkv = 2**31 - 1, 256, 1
    held = 2 * page - 1  # the slots that exist, the last one past the end
    g = gen(95)
    kc, vc = randn(g, 3, hkv, page, D), randn(g, 3, hkv, page, D)
    k, v = kc[[2, 0], 0].reshape(-1, D)[:held], vc[[2, 0], 0].reshape(-1, D)[:held]
    k, v = k.clone(), v.clone()
    kc[0, :, -1] = float("nan")
    vc[0, :, -1] = float("nan")
    kc[1], vc[1] = float("nan"), float("nan")
    table = torch.full((1, 2**31 // page), -1, dtype=torch.int32, device=DEV)
    table[0, -2:] = torch.tensor([2, 0], dtype=torch.int32, device=DEV)
    q = randn(g, n, 2, D)
    got = qz().attention_paged(q, qz().PagedKV(kc, vc), batch([n], [L], table), window=window)
    pos = torch.arange(held - n, held, device=DEV)
    for h in range(2):
        w, dot = C.weights(q[:, h], k, pos, window, D ** -0.5)
        w = w / w.sum(1, keepdim=True)
        tol = C.U16 * (w @ v.to(F64).abs()) + 4 * (D + 64) * 2.0 ** -24 * (dot[:, None] + 1)
        want = w @ v.to(F64)
        within(got[:, h], want, tol + C.U16 * want.abs() + held * C.S16)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 150])
def test_attention_weights_far_below_the_largest(D, n):
    """One key stands e^18 above 6000 others: each of them is below half of fp16's smallest
    value beside it, all of them together are not.  The values are 0 at the one and 1 at the
    others; enough sequences that one SM walks through the whole context."""
    L, S, page = 6000, 160, 64
    k = torch.zeros((L, 1, D), dtype=F16, device=DEV)
    v = torch.ones_like(k)
    k[0, :, 0] = 18.0
    v[0] = 0.0
    cache, table = paged([k], [v], page, D, 1)
    seqs = batch([n] * S, [L] * S, table.expand(S, -1).contiguous())  # all hold the same pages
    q = torch.zeros((n * S, 2, D), dtype=F16, device=DEV)
    q[..., 0] = 1.0
    got = qz().attention_paged(q, cache, seqs, scale=1.0)
    e = torch.exp(torch.tensor(-18.0, dtype=F64, device=DEV))
    others = torch.arange(L - n, L, device=DEV, dtype=F64).repeat(S)[:, None, None]
    want = (others * e / (1.0 + others * e)).expand(q.shape)
    # weights are held to 2^-32 of the largest; exponentials and sums; the rounding of out
    within(got, want, others * 2.0 ** -32 + want * (2.0 ** -9) + C.S16)


CAPS = [1e-38, 1e-6, 0.5, 50.0, 64.0, 65.0, 1e3, 1e4, 1e6, 1e8, 1e15, 3e38]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("cap", CAPS)
def test_attention_caps_of_any_size(cap, D):
    """Logits of up to several hundred, small ones among them, under caps from far below
    to far above them."""
    qs, kvs, hq, hkv = [1, 140, 5], [300, 200, 517], 4, 2
    g = gen(96)
    ks, vs = ([randn(g, n, hkv, D) for n in kvs] for _ in range(2))
    q = randn(g, sum(qs), hq, D, scale=1.0) * torch.logspace(-2, 1.5, hq, device=DEV)[:, None]
    q = q.to(F16)
    cache, table = paged(ks, vs, 32, D, hkv)
    got = qz().attention_paged(q, cache, batch(qs, kvs, table), softcap=cap)
    t = 0
    for n, L, k, v in zip(qs, kvs, ks, vs):
        seen = torch.arange(L, device=DEV)[None, :] <= torch.arange(L - n, L, device=DEV)[:, None]
        for h in range(hq):
            qq, kk, vv = q[t:t + n, h].to(F64), k[:, h // 2].to(F64), v[:, h // 2].to(F64)
            raw = qq @ kk.T * D ** -0.5
            x = cap * torch.tanh(raw / cap)
            w = torch.softmax(x.masked_fill(~seen, float("-inf")), 1)
            want, mag = w @ vv, w @ vv.abs()
            # a logit: a fp32 sum of D products, the cap's few roundings of it, and for caps
            # up to 64 those of 1 beside the tanh; then exp; the weights and out to fp16
            dot = (qq.abs() @ kk.abs().T * D ** -0.5).masked_fill(~seen, 0.0).amax(1, keepdim=True)
            x_max = x.abs().masked_fill(~seen, 0.0).amax(1, keepdim=True)
            dx = (D + 8) * 2.0 ** -24 * torch.minimum(dot, 64 * x_max + cap * (cap < 1)) \
                + 32 * 2.0 ** -24 * (x_max + 1) + (4 * 2.0 ** -22 * cap if cap <= 64 else 0.0)
            within(got[t:t + n, h], want, 2 * mag * dx + C.U16 * (mag + want.abs()) + 4 * L * C.S16)
        t += n


@pytest.mark.parametrize("cap", CAPS)
def test_attention_caps_of_logits_of_zero(cap):
    k, v = (randn(gen(97), 200, 1, 64) for _ in range(2))
    cache, table = paged([k], [v], 16, 64, 1)
    q = torch.zeros((1, 1, 64), dtype=F16, device=DEV)
    got = qz().attention_paged(q, cache, batch([1], [200], table), softcap=cap)
    want = v.to(F64).mean(0)[None]
    within(got, want, C.U16 * want.abs() + 2.0 ** -18)


@pytest.mark.parametrize("hq,hkv,D", [(4, 4, 64), (8, 2, 128), (6, 2, 128), (2, 1, 256)])
@pytest.mark.parametrize("scale", [None, -0.1])
def test_attention_rows_of_others_do_not_matter(hq, hkv, D, scale):
    """Rows before, behind and of another sequence that are not finite."""
    qs, kvs, before, behind = [5, 140, 1], [40, 300, 77], 3, 4
    g = gen(98)
    ks, vs = ([randn(g, n, hkv, D) for n in kvs] for _ in range(2))
    q = randn(g, sum(qs), hq, D)
    cache, table = paged(ks, vs, 32, D, hkv)
    want = qz().attention_paged(q, cache, batch(qs, kvs, table), scale=scale)
    bad = torch.full((before + q.shape[0] + behind, hq, D), float("nan"), dtype=F16, device=DEV)
    bad[before:before + q.shape[0]] = q
    bad[before + 5:before + 145] = float("inf")  # the second sequence
    seqs = batch(qs, kvs, table)
    seqs = qz().SeqBatch(seqs.cu_q + before, seqs.kv_len, table)
    out = torch.full_like(bad, 7.0)
    qz().attention_paged(bad, cache, seqs, scale=scale, out=out)
    assert bool((out[:before] == 7).all()) and bool((out[-behind:] == 7).all())
    out = out[before:-behind]
    assert torch.equal(out[:5], want[:5]) and torch.equal(out[145:], want[145:])


def test_a_single_token_of_a_wider_row():
    """One token's heads out of a row whose length is no multiple of 8."""
    g = gen(99)
    wide = randn(g, 1, 8 * 64 + 3)[:, :8 * 64]
    assert wide.stride(0) % 8
    q, k, v = wide.view(1, 8, 64).split([4, 2, 2], dim=1)
    ks, vs = [randn(g, 50, 2, 64)], [randn(g, 50, 2, 64)]
    rope = qz().rope_table(60, 64)
    outs = []
    for a, b, c in ((q, k, v), (q.contiguous(), k.contiguous(), v.contiguous())):
        cache, table = paged(ks, vs, 16, 64, 2)
        seqs = batch([1], [50], table)
        r = qz().rope_append(a, b, c, cache, seqs, rope)
        outs += [r, cache.k.nan_to_num(), qz().attention_paged(r, cache, seqs)]
    assert all(torch.equal(a, b) for a, b in zip(outs[:3], outs[3:]))


# ---------------------------------------------------------- 64-bit offsets ---
def far_apart(n, inner):
    """fp16 [n, *inner] whose parts lie 2^31 + 64 halves apart or more."""
    size = 1
    for d in inner:
        size *= d
    step = 2**31 // (n - 1) // 8 * 8 + 64 + size
    buf = torch.empty(((n - 1) * step + size,), dtype=F16, device=DEV)
    strides, s = [], size
    for d in inner:
        s //= d
        strides.append(s)
    return buf.as_strided((n, *inner), (step, *strides))


def test_cache_and_adapters_past_32_bits():
    """Pages, adapters and rows more than 2^32 bytes behind the first."""
    g = gen(100)
    kc, vc = far_apart(3, (2, 16, 64)), far_apart(3, (2, 16, 64))
    assert kc.stride(0) * 2 * kc.element_size() > 2**32
    near = [torch.empty((3, 2, 16, 64), dtype=F16, device=DEV) for _ in range(2)]
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device=DEV)
    q, k, v = randn(g, 40, 4, 64), randn(g, 40, 2, 64), randn(g, 40, 2, 64)
    outs = []
    for a, b in ((kc, vc), near):
        cache, seqs = qz().PagedKV(a, b), batch([40], [40], table)
        r = qz().rope_append(q, k, v, cache, seqs, qz().rope_table(40, 64))
        outs.append([r, a[:, :, :8], b[:, :, :8], qz().attention_paged(r, cache, seqs)])
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    del kc, vc
    a, b = far_apart(3, (16, 128)), far_apart(3, (96, 16))
    a.copy_(randn(g, 3, 16, 128, scale=0.1))
    b.copy_(randn(g, 3, 96, 16))
    x, y = randn(g, 200, 128), randn(g, 200, 96)
    scale = torch.ones(3, device=DEV)
    index = (torch.arange(200, device=DEV) % 4 - 1).to(torch.int32)
    for rows in (200, 20):
        got = qz().lora(x[:rows], y[:rows], qz().LoraAdapters(a, b, scale), index[:rows])
        near = qz().LoraAdapters(a.contiguous(), b.contiguous(), scale)
        want = qz().lora(x[:rows], y[:rows], near, index[:rows])
        assert torch.equal(got, want)
    del a, b
    rows = far_apart(3, (512,))
    rows.copy_(randn(g, 3, 512))
    w, out = randn(g, 512), far_apart(3, (512,))
    qz().rmsnorm(rows, w, out=out)
    assert torch.equal(out, qz().rmsnorm(rows.contiguous(), w)[0])
