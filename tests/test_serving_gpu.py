"""The layer operators running together: a small decoder served from INT8 and
INT4-outlier weights, with adapters, against its definition in 64 bits."""
import math
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F64 = torch.float64


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from weight_only_quantized_dequant_gb300 import build
    build.build()


def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import serve_adapters
    return serve_adapters


def dense(w) -> torch.Tensor:
    """The matrix that the codes stand for, in 64 bits."""
    if hasattr(w, "q"):
        return w.q[:, :w.K].to(F64) * w.scale.to(F64)
    kb = w.K - w.n_out
    b = w.q4.to(torch.int32)
    q = torch.stack([b & 15, b >> 4], dim=2).reshape(w.N, -1)[:, :kb]
    q = torch.where(q > 7, q - 16, q).to(F64) * w.scale.to(F64)[:, None]
    out = torch.empty((w.N, w.K), dtype=F64, device=w.q4.device)
    out[:, w.perm[:w.n_out].long()] = w.w_out[:, :w.n_out].to(F64)
    out[:, w.perm[w.n_out:].long()] = q
    return out


def reference(E, model, x, lens, adapter):
    """Whole sequences (no cache) through the model, in 64 bits."""
    def norm(h):
        return h / (h.square().mean(1, keepdim=True) + 1e-5).sqrt()

    def linear(lay, n, v, a):
        y = v @ dense(lay.mats[n]).T
        ad = lay.adapters.get(n)
        if ad is not None and a >= 0:
            y = y + (v @ ad.a[a].to(F64).T) @ ad.b[a].to(F64).T
        return y

    outs, at = [], 0
    for L, a in zip(lens, adapter):
        h = x[at:at + L].to(F64)
        at += L
        pos = torch.arange(L, device=x.device)
        for lay in model:
            D, half = E.HEAD_DIM, E.HEAD_DIM // 2
            c = lay.rope[pos, None, :half].to(F64)
            s = lay.rope[pos, None, half:].to(F64)

            def rot(v, heads):
                v = v.view(L, heads, D)
                p, q = v[..., :half], v[..., half:]
                return torch.cat([p * c - q * s, q * c + p * s], -1)

            y = norm(h)
            q = rot(linear(lay, "q", y, a), E.HEADS)
            k = rot(linear(lay, "k", y, a), E.KV_HEADS).repeat_interleave(E.HEADS // E.KV_HEADS, 1)
            v = linear(lay, "v", y, a).view(L, E.KV_HEADS, D).repeat_interleave(
                E.HEADS // E.KV_HEADS, 1)
            z = torch.einsum("ihd,jhd->hij", q, k) / math.sqrt(D)
            z = z.masked_fill(pos[None, None, :] > pos[None, :, None], -math.inf)
            o = torch.einsum("hij,jhd->ihd", torch.softmax(z, -1), v).reshape(L, -1)
            h = h + linear(lay, "o", o, a)
            y = norm(h)
            g, u = linear(lay, "gate", y, a), linear(lay, "up", y, a)
            h = h + linear(lay, "down", torch.nn.functional.silu(g) * u, a)
        outs.append(norm(h))
    return torch.cat(outs)


# About a dozen fp16 roundings a layer, each up to 2^-11 of its vector, add at
# most linearly and no step of the layer more than doubles a relative error.
LAYERS = 2
TOL = 2 * LAYERS * 12 * 2.0 ** -11


@pytest.mark.parametrize("fmt", ["int8", "int4"])
def test_prompts_and_decode_steps_match_the_definition(fmt):
    import weight_only_quantized_dequant_gb300 as qz
    from weight_only_quantized_dequant_gb300 import serving, synthetic as S
    E = example()
    lens, more = [70, 5, 130, 33], 6
    adapter = [0, -1, 3, 1]
    n = len(lens)
    table = serving.PageTable(n * E.MAX_PAGES, E.PAGE, E.MAX_PAGES)
    model = E.build(LAYERS, fmt, n * E.MAX_PAGES, 512)
    ws = qz.attention_workspace(sum(lens), n, E.HEADS, E.KV_HEADS, E.HEAD_DIM)
    full = [S.activation(L + more, E.HIDDEN, 500 + i, "cuda") for i, L in enumerate(lens)]
    want = reference(E, model, torch.cat(full), [L + more for L in lens], adapter)
    want = want.split([L + more for L in lens])

    def check(got, ref):
        err = float((got.to(F64) - ref).norm() / ref.norm())
        assert err <= TOL, err

    # the prompts, packed, in two chunks: all but the third, then it beside decode steps
    index = torch.tensor(sum(([adapter[i]] * lens[i] for i in (0, 1, 3)), []), dtype=torch.int32,
                         device="cuda")
    x = torch.cat([full[i][:lens[i]] for i in (0, 1, 3)])
    y, _ = E.step(model, x, table, {i: lens[i] for i in (0, 1, 3)}, index, ws)
    check(y, torch.cat([want[i][:lens[i]] for i in (0, 1, 3)]))
    index = torch.tensor([adapter[0]] + [adapter[2]] * lens[2], dtype=torch.int32, device="cuda")
    y, _ = E.step(model, torch.cat([full[0][lens[0]:lens[0] + 1], full[2][:lens[2]]]), table,
                  {0: 1, 2: lens[2]}, index, ws)
    check(y, torch.cat([want[0][lens[0]:lens[0] + 1], want[2][:lens[2]]]))
    # decode steps of all of them (the first is one token ahead)
    one = torch.tensor(adapter, dtype=torch.int32, device="cuda")
    at = [L + (i == 0) for i, L in enumerate(lens)]
    for _ in range(more - 1):
        y, _ = E.step(model, torch.stack([full[i][at[i]] for i in range(n)]), table,
                      {i: 1 for i in range(n)}, one, ws)
        check(y, torch.stack([want[i][at[i]] for i in range(n)]))
        at = [p + 1 for p in at]
    assert qz.device_error() == 0


def test_page_table_reuses_pages():
    from weight_only_quantized_dequant_gb300 import serving
    t = serving.PageTable(4, 16, 3)
    b = t.step({7: 40, 8: 1})
    assert b.cu_q.tolist() == [0, 40, 41] and b.kv_len.tolist() == [40, 1]
    with pytest.raises(RuntimeError):
        t.step({8: 16})
    t.release(7)
    assert t.step({9: 33}).page_table.shape == (1, 3)


def test_example_runs(capsys, monkeypatch):
    E = example()
    monkeypatch.setattr(sys, "argv", ["serve_adapters", "--layers", "1", "--tokens", "3"])
    E.main()
    assert "decode steps of 6 requests" in capsys.readouterr().out
