"""The served head's cap of its logits: those that differ stay different, so that the largest
is the one chosen, whatever comes before it by index."""
import pytest
import torch

from test_serving_gpu import example

pytestmark = pytest.mark.gpu

F64 = torch.float64


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from weight_only_quantized_dequant_gb300 import build
    build.build()


def heads(softcap, vocab=5000, spread=1.0):
    """A head with a cap, the same one without, and a step's end [T, hidden] for them."""
    import weight_only_quantized_dequant_gb300 as qz
    from weight_only_quantized_dequant_gb300 import serving, synthetic as S
    K = example().HIDDEN
    table = qz.quantize_int8(S.weight(vocab, K, 9, device="cuda"))
    g = torch.Generator(device="cuda").manual_seed(7)
    x, r = (torch.randn((64, K), generator=g, device="cuda").half() for _ in range(2))
    norm = torch.full((K,), 1.0, dtype=torch.float16, device="cuda")
    plain = serving.ServedHead(table, norm)
    top = float(plain.logits(x, r).float().amax(1).mean())
    norm *= spread * softcap / top  # the largest logits at about `spread` caps
    return serving.ServedHead(table, norm, softcap=softcap), serving.ServedHead(table, norm), x, r


@pytest.mark.parametrize("softcap", [5.0, 30.0])
@pytest.mark.parametrize("spread", [0.5, 1.0, 2.0, 3.0])
def test_capped_logits_keep_their_order(softcap, spread):
    capped, plain, x, r = heads(softcap, spread=spread)
    z = plain.logits(x, r)
    want = softcap * torch.tanh(z.to(F64) / softcap)
    got = capped.logits(x, r)
    # fp32: a quotient (a reciprocal and a product), a hyperbolic tangent (2 units in the last
    # place, 4 roundings) and a product; the quotient's error enters the result once at most
    assert bool(((got.to(F64) - want).abs() <= 8 * 2.0 ** -24 * want.abs()).all())
    u = torch.full((x.shape[0],), 0.5, device="cuda")
    index = torch.arange(want.shape[1], device="cuda")
    first = torch.where(want == want.amax(1, keepdim=True), index, want.shape[1]).amin(1)
    for options in (dict(temperature=0.0), dict(top_k=1)):
        tokens, _ = capped(x, r, u, **options)
        assert torch.equal(tokens.long(), first)
