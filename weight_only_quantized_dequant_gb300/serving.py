"""One decoder layer of a served model: the quantized products with everything
between them, for steps that mix whole prompts, chunks of prompts and single
tokens of many requests, each request with its own low-rank adapter.

    norm -> q, k, v (+ adapters) -> rotary, cache -> attention -> o (+ adapter)
    norm -> gate, up (+ adapters) -> silu(gate) * up -> down (+ adapter)

and behind the last layer the head: norm -> vocabulary product -> the next tokens, whose
embeddings come from the same INT8 table.

The residual stream is one fp16 buffer that the norms update in place.  The
products take at most QZ_MAX_BATCH rows a call, so longer steps run them in
slices; everything else takes the whole step at once.
"""
from __future__ import annotations

from dataclasses import dataclass, field

import torch

from . import _lib, api, layer

GROUPS = (("q", "k", "v"), ("o",), ("gate", "up"), ("down",))


class Products:
    """Grouped products of up to n_rows inputs (slices of QZ_MAX_BATCH rows)."""

    def __init__(self, mats: dict, device="cuda"):
        self.int8 = isinstance(next(iter(mats.values())), api.Int8Matrix)
        self.mats = mats
        need = max(api.gemm_workspace_bytes(_lib.QZ_MAX_BATCH, w.K, 0 if self.int8 else w.n_out)
                   for w in mats.values())
        self.workspace = torch.empty((need,), dtype=torch.uint8, device=device)

    def __call__(self, names, x: torch.Tensor) -> list:
        """[x @ W^T for the matrices `names`, which share the input x [T, K]]."""
        ws = [self.mats[n] for n in names]
        T = x.shape[0]
        ys = [torch.empty((T, -(-w.N // 8) * 8), dtype=torch.float16, device=x.device)[:, :w.N]
              for w in ws]
        gemm = api.gemm_int8_grouped if self.int8 else api.gemm_int4_outlier_grouped
        for a in range(0, T, _lib.QZ_MAX_BATCH):
            b = min(T, a + _lib.QZ_MAX_BATCH)
            gemm(ws, x[a:b], [y[a:b] for y in ys], workspace=self.workspace)
        return ys


@dataclass
class ServedLayer:
    """mats: q, k, v, o, gate, up, down as Int8Matrix or Int4oMatrix; norms:
    the two fp16 weights; cache: fp16 or INT8 rows; adapters: LoraAdapters by
    matrix name (those that have any).  window and softcap as in layer.attention_paged."""
    mats: dict
    norms: tuple
    cache: layer.PagedKV | layer.PagedKVInt8
    rope: torch.Tensor
    adapters: dict = field(default_factory=dict)
    eps: float = 1e-5
    w_bias: float = 0.0
    window: int = 0
    softcap: float = 0.0

    def __post_init__(self):
        self.products = Products(self.mats, self.cache.k.device)
        self.heads = self.mats["q"].N // self.cache.head_dim

    def _linear(self, names, x, index):
        ys = self.products(names, x)
        for n, y in zip(names, ys):
            if n in self.adapters and index is not None:
                layer.lora(x, y, self.adapters[n], index, out=y)
        return ys

    def __call__(self, x: torch.Tensor, residual: torch.Tensor | None, seqs: layer.SeqBatch,
                 index: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
        """(output [T, hidden], residual): x is the previous layer's output (the
        embeddings in the first one, with residual None), index the adapter of
        every row (int32, -1: none; None: no row has one), workspace from
        layer.attention_workspace."""
        T, D, hkv = x.shape[0], self.cache.head_dim, self.cache.n_kv_heads
        y, residual = layer.rmsnorm(x, self.norms[0], self.eps, residual=residual,
                                    w_bias=self.w_bias, residual_out=residual)
        q, k, v = self._linear(("q", "k", "v"), y, index)
        q = q.view(T, self.heads, D)
        layer.rope_append(q, k.view(T, hkv, D), v.view(T, hkv, D), self.cache, seqs, self.rope,
                          q_out=q)
        a = layer.attention_paged(q, self.cache, seqs, softcap=self.softcap, window=self.window,
                                  workspace=workspace)
        (o,) = self._linear(("o",), a.view(T, -1), index)
        # x belongs to the caller: the first layer's residual moves to a buffer of its own
        y, residual = layer.rmsnorm(o, self.norms[1], self.eps, residual=residual,
                                    w_bias=self.w_bias,
                                    residual_out=None if residual is x else residual)
        gate, up = self._linear(("gate", "up"), y, index)
        h = torch.nn.functional.silu(gate.float()).mul_(up).half()
        (out,) = self._linear(("down",), h, index)
        return out, residual


@dataclass
class ServedHead:
    """The end of a step: norm, logits from the INT8 vocabulary table (tied with the
    embeddings), and the choice of every row's next token."""
    table: api.Int8Matrix
    norm: torch.Tensor
    eps: float = 1e-5
    w_bias: float = 0.0
    softcap: float = 0.0

    def __post_init__(self):
        self.products = Products({"head": self.table}, self.table.q.device)

    def embed(self, tokens: torch.Tensor) -> torch.Tensor:
        """The first layer's input for int32 tokens [T]."""
        return api.embed_int8(self.table, tokens)

    def logits(self, x: torch.Tensor, residual: torch.Tensor) -> torch.Tensor:
        """[T, vocabulary] of the last layer's output and residual (or those rows of them that
        are wanted): fp16, and fp32 with a cap, which would make ties of neighbours in fp16."""
        y, _ = layer.rmsnorm(x, self.norm, self.eps, residual=residual, w_bias=self.w_bias)
        (z,) = self.products(("head",), y)
        if self.softcap == 0.0:
            return z
        return z.float().div_(self.softcap).tanh_().mul_(self.softcap)

    def __call__(self, x: torch.Tensor, residual: torch.Tensor, u: torch.Tensor, **options):
        """(tokens, log probabilities) with the options of layer.sample."""
        return layer.sample(self.logits(x, residual), u, **options)


class PageTable:
    """Pages of a pool handed to sequences as they grow (host side)."""

    def __init__(self, n_pages: int, page_size: int, max_pages: int):
        self.free = list(range(n_pages - 1, -1, -1))
        self.page_size, self.max_pages = page_size, max_pages
        self.pages: dict = {}
        self.lens: dict = {}

    def step(self, new: dict, device="cuda") -> layer.SeqBatch:
        """The SeqBatch of a step that brings new[i] tokens to sequence i (in the
        order of the dict); pages are taken from the pool as needed.  A step that
        does not fit raises and changes nothing, so that it can be tried again once
        other sequences have given pages back."""
        cu, lens, pages, at = [0], {}, {}, len(self.free)
        for i, n in new.items():
            if n < 0:
                raise ValueError(f"sequence {i}: {n} new tokens")
            lens[i] = self.lens.get(i, 0) + n
            held = self.pages.get(i, [])
            more = max(0, -(-lens[i] // self.page_size) - len(held))
            if more > at or len(held) + more > self.max_pages:
                raise RuntimeError(f"no page for sequence {i}")
            pages[i] = held + self.free[at - more:at][::-1]
            at -= more
            cu.append(cu[-1] + n)
        rows = [p + [0] * (self.max_pages - len(p)) for p in pages.values()]
        batch = layer.SeqBatch(*(torch.tensor(t, dtype=torch.int32, device=device)
                                 for t in (cu, list(lens.values()), rows)))
        del self.free[at:]
        self.pages.update(pages)
        self.lens.update(lens)
        return batch

    def release(self, i) -> None:
        """Give a finished sequence's pages back."""
        self.free.extend(self.pages.pop(i, []))
        self.lens.pop(i, None)
