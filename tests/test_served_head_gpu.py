"""Served layers over a cache of INT8 rows with the head behind them: prompts, decode steps
and the choice of tokens running together, against the model's definition in 64 bits."""
import sys

import pytest
import torch

import test_sample_gpu as sampling
from test_serving_gpu import LAYERS, TOL, dense, example, reference

pytestmark = pytest.mark.gpu

F64 = torch.float64
VOCAB = 1003  # odd: rows of logits that end inside a vector

# To the fp16 roundings the cache adds codes half a step off: of rows whose largest entry is
# at most 4 times their root mean square, 4/127/sqrt(12) = 0.9% of the values and as much
# of the keys, which a logit of unit variance passes on; twice 1.8% a layer, and the head's
# norm and product (2 roundings).
TOL8 = TOL + LAYERS * 2 * 0.018 + 2 * 2.0 ** -11


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from weight_only_quantized_dequant_gb300 import build
    build.build()


@pytest.mark.parametrize("softcap", [0.0, 5.0])
def test_prompts_tokens_and_decode_steps(softcap):
    import weight_only_quantized_dequant_gb300 as qz
    from weight_only_quantized_dequant_gb300 import serving, synthetic as S
    E = example()
    lens, more, adapter = [70, 5, 130, 33], 4, [0, -1, 3, 1]
    n = len(lens)
    pages = serving.PageTable(n * E.MAX_PAGES, E.PAGE, E.MAX_PAGES)
    model = E.build(LAYERS, "int8", n * E.MAX_PAGES, 512, "int8")
    head = serving.ServedHead(qz.quantize_int8(S.weight(VOCAB, E.HIDDEN, 9, device="cuda")),
                              model[-1].norms[1], softcap=softcap)
    ws = qz.attention_workspace(sum(lens), n, E.HEADS, E.KV_HEADS, E.HEAD_DIM)
    g = torch.Generator(device="cuda").manual_seed(3)
    tokens = torch.randint(VOCAB, (sum(lens),), generator=g, device="cuda", dtype=torch.int32)
    text = [head.embed(t) for t in tokens.split(lens)]
    index = torch.tensor(sum(([a] * L for a, L in zip(adapter, lens)), []), dtype=torch.int32,
                         device="cuda")
    one = torch.tensor(adapter, dtype=torch.int32, device="cuda")
    options = dict(temperature=0.8, top_k=50, top_p=0.9)
    x, r, seqs = E.run_layers(model, torch.cat(text), pages, dict(enumerate(lens)), index, ws)
    last = (seqs.cu_q[1:] - 1).long()
    for _ in range(more):
        want = reference(E, model, torch.cat(text), [t.shape[0] for t in text], adapter)
        ends = torch.tensor([t.shape[0] for t in text], device="cuda").cumsum(0) - 1
        z = want[ends] @ dense(head.table).T
        z = z if softcap == 0 else torch.tanh(z / softcap) * softcap
        got = head.logits(x[last], r[last])
        err = float((got.to(F64) - z).norm() / z.norm())
        assert got.shape == (n, VOCAB) and err <= TOL8, err
        u = torch.rand((n,), generator=g, device="cuda")
        tok, lp = head(x[last], r[last], u, **options)
        for i in range(n):
            t, l, _ = sampling.reference(got[i], u[i].item(), 0.8, 50, 0.9, 0.0)
            assert tok[i].item() == t and abs(lp[i].item() - l) <= 2.0 ** -24 * abs(l) + 2.0 ** -28
        new = head.embed(tok)
        text = [torch.cat([a, b[None]]) for a, b in zip(text, new)]
        x, r, _ = E.run_layers(model, new, pages, {i: 1 for i in range(n)}, one, ws)
        last = torch.arange(n, device="cuda")
    assert qz.device_error() == 0


def test_what_a_layer_holds_reads_back():
    """The cache of a served layer, read as fp16 for a request's whole length, gives the
    attention that its INT8 rows give."""
    import weight_only_quantized_dequant_gb300 as qz
    from weight_only_quantized_dequant_gb300 import serving
    E = example()
    L = 100
    pages = serving.PageTable(E.MAX_PAGES, E.PAGE, E.MAX_PAGES)
    (lay,) = E.build(1, "int8", E.MAX_PAGES, 512, "int8")
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((L, E.HIDDEN), generator=g, device="cuda").half()
    seqs = pages.step({0: L})
    lay(x, None, seqs)
    k, v = qz.cache_read(lay.cache, seqs, L)
    q = torch.randn((L, E.HEADS, E.HEAD_DIM), generator=g, device="cuda").half()
    got = qz.attention_paged(q, lay.cache, seqs)
    rep = E.HEADS // E.KV_HEADS
    z = torch.einsum("ihd,jhd->hij", q.to(F64), k.to(F64).repeat_interleave(rep, 1))
    pos = torch.arange(L, device="cuda")
    z = (z / E.HEAD_DIM ** 0.5).masked_fill(pos[None] > pos[:, None], -torch.inf).softmax(-1)
    want = torch.einsum("hij,jhd->ihd", z, v.to(F64).repeat_interleave(rep, 1))
    # rounded: k (logits of up to 8 or so, 2^-11 of each), v, weights and outputs
    assert float((got.to(F64) - want).norm() / want.norm()) <= (2 * 8 + 3) * 2.0 ** -11
    assert qz.device_error() == 0


@pytest.mark.parametrize("extra", [["--cache", "int8"], ["--vocab", "1003"],
                                   ["--cache", "int8", "--vocab", "1003", "--format", "int4"]])
def test_example_runs(capsys, monkeypatch, extra):
    E = example()
    monkeypatch.setattr(sys, "argv", ["serve_adapters", "--layers", "1", "--tokens", "3"] + extra)
    E.main()
    out = capsys.readouterr().out
    assert "decode steps of 6 requests" in out
    assert ("tokens [" in out) == ("--vocab" in extra)
