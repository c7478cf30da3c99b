"""Serve a few requests with different adapters from one compressed decoder.

Prompts of different lengths run packed in one step, then every request decodes
token by token, all of them in one step each.  Weights, adapters and inputs are
synthetic (seeded).  Without a vocabulary the hidden state of a token is fed back as
the next input; with one (--vocab N) the next token is chosen from its logits and
embedded.  The key/value cache is fp16 or INT8 rows (--cache).

    python examples/serve_adapters.py [--format int8|int4] [--cache fp16|int8] [--layers N]
                                      [--tokens N] [--vocab N] [--temperature T] [--top-p P]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import weight_only_quantized_dequant_gb300 as qz  # noqa: E402
from weight_only_quantized_dequant_gb300 import serving, synthetic as S  # noqa: E402

HIDDEN, HEADS, KV_HEADS, HEAD_DIM, INTER = 1024, 16, 4, 64, 2816
SHAPES = {"q": (HEADS * HEAD_DIM, HIDDEN), "k": (KV_HEADS * HEAD_DIM, HIDDEN),
          "v": (KV_HEADS * HEAD_DIM, HIDDEN), "o": (HIDDEN, HEADS * HEAD_DIM),
          "gate": (INTER, HIDDEN), "up": (INTER, HIDDEN), "down": (HIDDEN, INTER)}
RANK, N_ADAPTERS, PAGE, MAX_PAGES = 16, 4, 16, 64


def quantize(W: dict, fmt: str) -> dict:
    if fmt == "int8":
        return {n: qz.quantize_int8(w) for n, w in W.items()}
    mats = {}
    for names in serving.GROUPS:  # matrices that share an input share its permutation
        K = W[names[0]].shape[1]
        n_out = qz.default_n_out(K)
        colsum = torch.zeros((K,), dtype=torch.int64, device="cuda")
        for n in names:
            qz.saliency_accumulate(W[n], colsum)
        perm = qz.select_outliers(colsum, S.x_profile(K, n_out, 5, "cuda"), n_out)
        for n in names:
            mats[n] = qz.quantize_int4_outlier(W[n], perm, n_out)
    return mats


def build(layers: int, fmt: str, n_pages: int, positions: int, cache_fmt: str = "fp16"):
    kind = qz.PagedKV if cache_fmt == "fp16" else qz.PagedKVInt8
    rope = qz.rope_table(positions, HEAD_DIM)
    model = []
    for l in range(layers):
        W = {n: S.weight(*shape, 1000 * l + i, device="cuda")
             for i, (n, shape) in enumerate(SHAPES.items())}
        adapters = {}
        for i, n in enumerate(("q", "v", "o", "down")):
            N, K = SHAPES[n]
            a = S.activation(N_ADAPTERS * RANK, K, 1000 * l + 20 + i, "cuda") * K ** -0.5
            b = S.activation(N_ADAPTERS * N, RANK, 1000 * l + 40 + i, "cuda") * 0.05
            adapters[n] = qz.LoraAdapters(a.view(N_ADAPTERS, RANK, K), b.view(N_ADAPTERS, N, RANK),
                                          torch.ones(N_ADAPTERS, device="cuda"))
        norms = tuple(torch.ones(HIDDEN, dtype=torch.float16, device="cuda") for _ in range(2))
        cache = kind.empty(n_pages, KV_HEADS, PAGE, HEAD_DIM)
        model.append(serving.ServedLayer(quantize(W, fmt), norms, cache, rope, adapters))
    return model


def run_layers(model, x, table, new, index, workspace):
    seqs, residual = table.step(new), None
    for lay in model:
        x, residual = lay(x, residual, seqs, index, workspace)
    return x, residual, seqs


def step(model, x, table, new, index, workspace):
    x, residual, seqs = run_layers(model, x, table, new, index, workspace)
    return qz.rmsnorm(x, model[-1].norms[1], residual=residual)[0], seqs


def next_input(head, x, residual, last, g, options):
    """Tokens of the rows `last`, and the next step's input."""
    u = torch.rand((len(last),), generator=g, device="cuda")
    tokens, _ = head(x[last], residual[last], u, **options)
    return tokens, head.embed(tokens)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--format", choices=("int8", "int4"), default="int4")
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=32)
    ap.add_argument("--cache", choices=("fp16", "int8"), default="fp16")
    ap.add_argument("--vocab", type=int, default=0)
    ap.add_argument("--temperature", type=float, default=0.8)
    ap.add_argument("--top-p", type=float, default=0.95)
    ap.add_argument("--prompts", type=int, nargs="*", default=[300, 17, 129, 64, 5, 200])
    args = ap.parse_args()
    n = len(args.prompts)
    total = sum(args.prompts)
    table = serving.PageTable(n * MAX_PAGES, PAGE, MAX_PAGES)
    model = build(args.layers, args.format, n * MAX_PAGES, PAGE * MAX_PAGES, args.cache)
    head, g, texts = None, torch.Generator(device="cuda").manual_seed(5), []
    options = dict(temperature=args.temperature, top_k=50, top_p=args.top_p)
    if args.vocab:
        head = serving.ServedHead(qz.quantize_int8(S.weight(args.vocab, HIDDEN, 9, device="cuda")),
                                  model[-1].norms[1])
    ws = qz.attention_workspace(total, n, HEADS, KV_HEADS, HEAD_DIM)
    adapter = [i % (N_ADAPTERS + 1) - 1 for i in range(n)]  # one request in five without one

    x = S.activation(total, HIDDEN, 77, "cuda")
    rows = torch.tensor(sum(([adapter[i]] * p for i, p in enumerate(args.prompts)), []),
                        dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    t = time.perf_counter()
    if head is None:
        y, seqs = step(model, x, table, dict(enumerate(args.prompts)), rows, ws)
        x = y[(seqs.cu_q[1:] - 1).long()]
    else:
        y, r, seqs = run_layers(model, x, table, dict(enumerate(args.prompts)), rows, ws)
        tokens, x = next_input(head, y, r, (seqs.cu_q[1:] - 1).long(), g, options)
        texts.append(tokens)
    torch.cuda.synchronize()
    print(f"prompts of {args.prompts} tokens: {1e3 * (time.perf_counter() - t):.2f} ms")

    one = torch.tensor(adapter, dtype=torch.int32, device="cuda")
    t = time.perf_counter()
    each = torch.arange(n, device="cuda")
    for _ in range(args.tokens):
        if head is None:
            x, _ = step(model, x, table, {i: 1 for i in range(n)}, one, ws)
        else:
            y, r, _ = run_layers(model, x, table, {i: 1 for i in range(n)}, one, ws)
            tokens, x = next_input(head, y, r, each, g, options)
            texts.append(tokens)
    torch.cuda.synchronize()
    ms = 1e3 * (time.perf_counter() - t) / args.tokens
    print(f"{args.tokens} decode steps of {n} requests: {ms:.2f} ms each, "
          f"{args.layers} layers, {args.format}, {args.cache} cache")
    assert qz.device_error() == 0 and bool(torch.isfinite(x).all())
    for i in range(n):
        print(f"request {i}: adapter {adapter[i]:2d}, {table.lens[i]} tokens held, "
              f"state norm {float(x[i].float().norm()):.4f}"
              + (f", tokens {[int(t[i]) for t in texts[:8]]}" if texts else ""))


if __name__ == "__main__":
    main()
