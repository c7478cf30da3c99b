"""What the bounds of the layer operators' tests can see: mistakes planted in the 64-bit
references, on the host, have to fall outside."""
import pytest
import torch

import layer_cases as C

F64 = torch.float64


@pytest.mark.parametrize("qs,kvs,hq,hkv,D,page,window", C.CONTEXTS[:8])
def test_a_lost_or_doubled_key_block_is_seen(qs, kvs, hq, hkv, D, page, window):
    for i, L in enumerate(kvs):
        q, ks, vs = C.signal_inputs([1], [L], 1, 1, D, 80 + i, "cpu")
        pos = torch.tensor([L - 1])
        w, dot = C.weights(q[:, 0], ks[0][:, 0], pos, window, D ** -0.5)
        v = vs[0][:, 0].to(F64)
        want = w @ v / w.sum()
        tol = C.signal_bound(want, w, v, dot, D)
        n = -(-L // C.BLOCK)
        pad = n * C.BLOCK - L
        wb = torch.nn.functional.pad(w, (0, pad)).view(n, 1, C.BLOCK)
        vb = torch.nn.functional.pad(v, (0, 0, 0, pad)).view(n, C.BLOCK, D)
        num, den = (wb @ vb)[:, 0], wb.sum((1, 2))  # of every block
        live = den > 0
        for f in (-1.0, 1.0):  # lost, doubled
            got = ((w @ v) + f * num) / (w.sum() + f * den[:, None])
            off = ((got - want).abs() > tol).any(1)
            if n == 1:  # all there is: its weight cancels
                continue
            assert bool(off[live].all()), (L, f, int((~off[live]).sum()))


@pytest.mark.parametrize("case", range(len(C.ADAPTERS)))
def test_an_inner_vector_in_fewer_bits_is_seen(case):
    T, run, n, R, K, N, mixed, _ = C.ADAPTERS[case]
    g = torch.Generator().manual_seed(81)

    def randn(*shape, scale=1.0):
        return (torch.randn(shape, generator=g) * scale).to(C.F16)

    T, N = 24, 192  # rows and outputs are alike
    x, y = randn(T, K), randn(T, N, scale=0.01)
    a, b = randn(1, R, K, scale=K ** -0.5), randn(1, N, R, scale=0.5)
    want, tol = C.adapter_reference(x, y, a, b, torch.ones(1), None, [0] * T)
    u = x.to(F64) @ a[0].to(F64).T

    def out(u):
        return y.to(F64) + u @ b[0].to(F64).T

    assert bool(((out(u) - want).abs() <= tol).all())
    big = 2.0 ** (9 - torch.floor(torch.log2(u.abs().amax(1, keepdim=True))))
    h = (u * big).to(torch.bfloat16).to(F64) / big
    assert bool(((out(h) - want).abs() > tol).any())
    lost = u.clone()
    lost[:, 0] = 0.0  # a rank
    assert bool(((out(lost) - want).abs() > tol).any())
    lost = x.to(F64).clone()
    lost[:, K // 2:K // 2 + 64] = 0.0  # a warp's step of K
    assert bool(((out(lost @ a[0].to(F64).T) - want).abs() > tol).any())


def test_exact_products_need_both_parts():
    x, y, a, b, index, want = C.cancelling_adapters(8, 3, 16, 4096, 200, "cpu")
    u = torch.einsum("tk,trk->tr", x.to(F64), a.to(F64)[index.clamp(min=0).long()])
    B = b.to(F64)[index.clamp(min=0).long()] * (index >= 0)[:, None, None]
    assert torch.equal(y.to(F64) + torch.einsum("tnr,tr->tn", B, u), want)
    one = (u / 2).to(C.F16).to(F64) * 2
    assert not torch.equal(y.to(F64) + torch.einsum("tnr,tr->tn", B, one), want)
