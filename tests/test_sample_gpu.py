"""The choice of tokens against its definition in 64 bits: filters, ties, borders, types,
strides and rows that have no token to offer.

Tokens have to be equal.  A border between two of them would have to lie within the weights'
error (2^-30 of each, random) of u times the total: with the few hundred distinct values
and the u of these tests the nearest is further.  Log probabilities: one rounding to fp32
and the weights' errors, 2^-24 of the value and 2^-28."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
F64, F32, F16, BF16 = torch.float64, torch.float32, torch.float16, torch.bfloat16
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from weight_only_quantized_dequant_gb300 import build
    build.build()


def qz():
    import weight_only_quantized_dequant_gb300 as m
    return m


def f32(v):
    return torch.tensor(v, dtype=F32).item()


def reference(x, u, T, k, p, min_p):
    """(token, log probability, kept) of one row of logits, on the host."""
    x = x.cpu().to(F64)
    x = torch.where(x.isnan(), -INF, x)
    V = x.numel()
    if float(x.max()) == -INF:
        return -1, -INF, 0
    T, p, min_p = f32(T), f32(p), f32(min_p)
    order = sorted(range(V), key=lambda i: (-float(x[i]), i)) if V < 4000 else \
        torch.sort(x, descending=True, stable=True).indices.tolist()
    if not T > 0:
        return order[0], 0.0, 1
    m = x[order[0]]
    if m == INF:
        w = (x == INF).to(F64)
    else:
        w = torch.where(x == -INF, 0.0, torch.exp((x - m) / T))
    ws = w[order]
    n = min(k, V) if k > 0 else V
    if p < 1:
        sums = torch.cumsum(ws[:n], 0)
        n = min(n, int((sums < max(p, 0.0) * sums[-1]).sum()) + 1)
    if min_p > 0:
        n = min(n, int((ws >= min(min_p, 1.0)).sum()))
    keep = torch.zeros(V, dtype=F64)
    keep[order[:n]] = 1
    sums = torch.cumsum(w * keep, 0)
    u = min(max(f32(u), 0.0), 1 - 2.0 ** -24)
    t = int((sums <= u * sums[-1]).sum())
    return t, float(torch.log(w[t] / sums[-1])), n


def check(x, u, T=1.0, k=0, p=1.0, min_p=0.0):
    B = x.shape[0]
    tok, lp = qz().sample(x, u, T, k, p, min_p)
    row = [[o[i].item() if isinstance(o, torch.Tensor) else o for o in (T, k, p, min_p)]
           for i in range(B)]
    for i in range(B):
        t, l, n = reference(x[i], u[i].item(), *row[i])
        assert tok[i].item() == t, (i, row[i], u[i].item(), tok[i].item(), t, n)
        got = lp[i].item()
        assert got == l or abs(got - l) <= 2.0 ** -24 * abs(l) + 2.0 ** -28, (i, got, l)
    return tok, lp


def logits(B, V, seed, dtype=F16, scale=3.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return ((torch.randn((B, V), generator=g, device=DEV) * scale).to(dtype),
            torch.rand((B,), generator=g, device=DEV))


SIZES = [1, 2, 7, 31, 32, 33, 255, 1000, 4096, 8193, 32000, 50001, 131072, 262144]


@pytest.mark.parametrize("V", SIZES)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_sizes_and_types(V, dtype):
    x, u = logits(3, V, V, dtype)
    check(x, u)
    check(x, u, T=0.7, k=40, p=0.9, min_p=0.02)
    check(x, u, p=0.8)
    check(x, u, k=max(1, V // 3))
    check(x, u, T=0.0)


@pytest.mark.parametrize("B", [1, 2, 40, 300])
def test_rows(B):
    x, u = logits(B, 3000, B)
    check(x, u, T=1.3, k=100, p=0.95)


@pytest.mark.parametrize("V,pad,offset", [(100, 0, 1), (4099, 0, 0), (5000, 8, 0), (20001, 3, 5)])
@pytest.mark.parametrize("dtype", [F16, F32])
def test_strides_and_alignment(V, pad, offset, dtype):
    x, u = logits(5, V, 3, dtype)
    buf = torch.full((5 * (V + pad) + offset,), NAN, dtype=dtype, device=DEV)
    y = buf[offset:].view(5, V + pad)[:, :V]
    y.copy_(x)
    want = qz().sample(x, u, 0.9, 50, 0.9)
    got = check(y, u, 0.9, 50, 0.9)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("T", [1e-4, 0.05, 0.5, 1.0, 2.0, 50.0, 1e4])
@pytest.mark.parametrize("dtype", [F16, F32])
def test_temperatures(T, dtype):
    x, u = logits(6, 9000, 5, dtype)
    check(x, u, T)
    check(x, u, T, p=0.7)
    check(x, u, T, k=700, p=0.99, min_p=1e-4)


@pytest.mark.parametrize("k", [-1, 0, 1, 2, 3, 999, 1000, 1001, 5000])
def test_top_k(k):
    x, u = logits(8, 1000, 6)
    check(x, u, k=k)


@pytest.mark.parametrize("p", [-1.0, 0.0, 1e-30, 1e-6, 0.1, 0.5, 0.999, 0.9999999, 1.0, 2.0, NAN])
def test_top_p(p):
    x, u = logits(8, 5000, 7)
    check(x, u, p=p)
    check(x, u, k=30, p=p)


@pytest.mark.parametrize("m", [-0.5, 0.0, 1e-30, 1e-3, 0.3, 0.999, 1.0, 3.0, NAN])
def test_min_p(m):
    x, u = logits(8, 5000, 8, F32)
    check(x, u, min_p=m)
    check(x, u, T=0.6, k=500, p=0.9, min_p=m)


@pytest.mark.parametrize("V", [10, 1000, 40000])
def test_ties_go_to_the_lowest_index(V):
    u = torch.linspace(0, 1, 9, device=DEV)[:8].contiguous()
    flat = torch.zeros((8, V), dtype=F16, device=DEV)
    flat[1::2] = -0.0  # equal to 0
    flat[3, ::2] = 0.0
    check(flat, u)
    check(flat, u, k=max(1, V // 2 - 1))
    check(flat, u, p=0.5)
    check(flat, u, T=0.0)
    g = torch.Generator(device=DEV).manual_seed(1)
    few = torch.randint(-3, 4, (8, V), generator=g, device=DEV).to(F16)  # seven values
    for k in (1, 3, V // 5 + 1):
        check(few, u, k=k)
        check(few, u, k=k, p=0.6)
    check(few, u, p=0.3)
    check(few, u, p=0.9, min_p=0.1)


def test_masked_places():
    x, u = logits(8, 3001, 9)
    x[0] = -INF                      # nothing to choose
    x[1] = NAN
    x[2, :3000] = -INF               # one token
    x[3, 5] = INF                    # takes all
    x[4, [7, 2000]] = INF            # share it
    x[5, ::2] = torch.finfo(F16).min
    x[6] = torch.finfo(F16).min      # as good as any other value
    x[7, ::3] = NAN
    for T in (1.0, 0.0, 0.3, INF):
        for k, p, m in ((0, 1.0, 0.0), (5, 1.0, 0.0), (0, 0.5, 0.0), (2900, 0.9, 0.01)):
            check(x, u, T, k, p, m)
    tok, lp = qz().sample(x, u)
    assert tok[:2].tolist() == [-1, -1] and lp[:2].tolist() == [-INF, -INF]


def test_numbers_at_the_ends():
    x, _ = logits(8, 700, 10)
    u = torch.tensor([0.0, -1.0, 1.0, 2.0, 1 - 2.0 ** -24, 2.0 ** -149, NAN, -0.0], device=DEV)
    tok, _ = qz().sample(x, u, 1.0, 20)
    for i, at in enumerate([0.0, 0.0, 1.0, 1.0, 1.0, 2.0 ** -149, 0.0, 0.0]):
        assert tok[i].item() == reference(x[i], at, 1.0, 20, 1.0, 0.0)[0]


def test_options_of_every_row():
    B = 30
    x, u = logits(B, 6000, 11, F32)
    i = torch.arange(B, device=DEV)
    T = torch.where(i % 5 == 0, 0.0, 0.5 + 0.1 * (i % 7)).to(F32)
    k = torch.where(i % 3 == 0, 0, 1 + 17 * i).to(torch.int32)
    p = torch.where(i % 4 == 0, 1.0, 0.99 - 0.03 * i).to(F32)
    m = torch.where(i % 2 == 0, 0.0, 0.01 * i).to(F32)
    check(x, u, T, k, p, m)
    check(x, u, T, 40, p, 0.01)
    check(x, u, 0.8, k, 0.9, m)


def test_every_token_has_its_share():
    """u over a fine grid gives every token as often as its probability says, to one count
    at each border."""
    V, n = 60, 4096
    x, _ = logits(1, V, 12, scale=1.0)
    u = (torch.arange(n, device=DEV, dtype=F32) + 0.5) / n
    tok, lp = qz().sample(x.expand(n, V).contiguous(), u, 1.2, 50, 0.97)
    count = torch.bincount(tok.long(), minlength=V).to(F64)
    prob = torch.zeros(V, dtype=F64, device=DEV).scatter_(0, tok.long(), lp.to(F64).exp())
    assert abs(float(prob.sum()) - 1) < 1e-6
    assert bool(((count - prob * n).abs() <= 1 + 1e-3).all())
    assert bool((tok[1:] >= tok[:-1]).all())


def test_borders_are_sharp():
    """u just below and on the border between two tokens of a flat row."""
    V = 4096
    x = torch.zeros((6, V), dtype=F32, device=DEV)
    u = torch.tensor([1 / 4096, 1 / 4096 - 2.0 ** -36, 0.5, 0.5 - 2.0 ** -25, 1 - 2.0 ** -12,
                      1 - 2.0 ** -12 - 2.0 ** -24], device=DEV)
    tok, _ = qz().sample(x, u)
    assert tok.tolist() == [1, 0, 2048, 2047, 4095, 4094]
    # a nucleus that its tokens' sum reaches exactly
    _, lp = qz().sample(x, u, 1.0, 0, 0.25)
    assert torch.allclose(lp, torch.full_like(lp, -math.log(1024)), atol=1e-6)


@pytest.mark.parametrize("scale", [1e-3, 1.0, 30.0])
def test_repeats_and_does_not_depend_on_other_rows(scale):
    x, u = logits(20, 30000, 13, F32, scale)
    a = qz().sample(x, u, 0.9, 300, 0.95, 0.001)
    for _ in range(3):
        b = qz().sample(x, u, 0.9, 300, 0.95, 0.001)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for i in (0, 7, 19):
        c = qz().sample(x[i:i + 1], u[i:i + 1], 0.9, 300, 0.95, 0.001)
        assert c[0][0] == a[0][i] and c[1][0] == a[1][i]


def test_captured_on_another_stream():
    x, u = logits(4, 40000, 14)
    tok = torch.empty(4, dtype=torch.int32, device=DEV)
    lp = torch.empty(4, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        qz().sample(x, u, 0.8, 60, 0.9, out=tok, logprob=lp)
    for seed in (15, 16):
        y, w = logits(4, 40000, seed)
        x.copy_(y)
        u.copy_(w)
        graph.replay()
        torch.cuda.synchronize()
        want = qz().sample(y, w, 0.8, 60, 0.9)
        assert torch.equal(tok, want[0]) and torch.equal(lp, want[1])


def test_refusals():
    x, u = logits(4, 100, 17)
    for bad in [lambda: qz().sample(x.cpu(), u), lambda: qz().sample(x, u[:3]),
                lambda: qz().sample(x.double(), u), lambda: qz().sample(x[0], u),
                lambda: qz().sample(x.t(), u), lambda: qz().sample(x, u.half()),
                lambda: qz().sample(x, u, torch.ones(3, device=DEV)),
                lambda: qz().sample(x, u, 1.0, torch.ones(4, device=DEV)),
                lambda: qz().sample(x, u, 1.0, 2 ** 40),
                lambda: qz().sample(x[:, :0], u),
                lambda: qz().sample(x, u, out=torch.empty(4, device=DEV))]:
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(qz().QzError):
        qz().sample(torch.zeros((1, 2 ** 18 + 1), dtype=F16, device=DEV), u[:1])
    tok, lp = qz().sample(x[:0], u[:0])
    assert tok.shape == (0,) and lp.shape == (0,)


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("V", [60000, 200000])
def test_nearly_equal_logits(V, dtype):
    """Most of a row lies around the cut: more than a warp lists."""
    g = torch.Generator(device=DEV).manual_seed(31)
    x = (torch.randn((4, V), generator=g, device=DEV) * 0.02 + 3).to(dtype)
    x[1, ::3] -= 1.0
    x[2, : V // 8] += 0.3  # all of them on one part of the row
    u = torch.tensor([0.1, 0.5, 0.9, 0.999], device=DEV)
    check(x, u, p=torch.tensor([0.5, 0.95, 0.2, 0.9], device=DEV))
    check(x, u, T=0.7, p=0.6, min_p=0.98)
