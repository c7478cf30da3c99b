"""The steps of a decoder layer around its quantized products, as thin calls
of the library (include/qz.h, "Layer glue for serving"): ``rmsnorm`` and
``rmsnorm_int8``, ``rope_append`` and ``attention_paged`` over a ``PagedKV``
cache, and ``lora`` for the low-rank adapters beside a shared projection.

Every function takes ``stream`` (default: the current one); outputs and
workspaces that a call allocates belong to that stream.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass, field

import torch

from . import _lib

_F16 = torch.float16
_raw_stream = torch._C._cuda_getCurrentRawStream  # torch.cuda.current_stream() costs 10x as much


def _stream_of(t: torch.Tensor, stream) -> int:
    return _raw_stream(t.device.index) if stream is None else stream.cuda_stream


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """torch.empty on the stream the call runs on, so that the memory is not
    handed to other streams while the kernels use it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _rows(t: torch.Tensor, what: str, shape=None, dtype=_F16) -> torch.Tensor:
    """A CUDA matrix whose rows are contiguous."""
    if not t.is_cuda:
        raise ValueError("libqz works on CUDA tensors only (no CPU fallback)")
    if t.dtype != dtype or t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{what}: a 2-D {dtype} tensor with contiguous rows is needed")
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {shape}")
    return t


def _ld(t: torch.Tensor) -> int:
    """Row stride; that of one row (which torch may report as anything) is its length."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _vec(t: torch.Tensor, what: str, n: int, dtype) -> torch.Tensor:
    if not t.is_cuda:
        raise ValueError("libqz works on CUDA tensors only (no CPU fallback)")
    if t.dtype != dtype or t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{what}: a contiguous {dtype} vector of {n} is needed")
    return t


# ------------------------------------------------------------------ norm ---
def _norm_args(x, weight, residual, residual_out):
    x = _rows(x, "x")
    T, K = x.shape
    _vec(weight, "weight", K, _F16)
    if residual is not None:
        _rows(residual, "residual", (T, K))
    if residual_out is not None:
        _rows(residual_out, "residual_out", (T, K))
    return T, K


def rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
            residual: torch.Tensor | None = None, w_bias: float = 0.0,
            out: torch.Tensor | None = None, residual_out: torch.Tensor | None = None,
            stream=None):
    """(y, h): h = x + residual and y = h * rsqrt(mean(h^2) + eps) * (w_bias +
    weight) for fp16 rows x [T, K].  h, the next residual, goes to residual_out
    (may be residual or x; allocated if None); without a residual h is x itself
    and is not written."""
    T, K = _norm_args(x, weight, residual, residual_out)
    if out is None:
        out = _empty((T, K), _F16, x.device, stream)
    else:
        _rows(out, "out", (T, K))
    h = residual_out
    if h is None and residual is not None:
        h = _empty((T, K), _F16, x.device, stream)
    _lib.call("qz_rmsnorm", x.data_ptr(), _ld(x),
              None if residual is None else residual.data_ptr(),
              0 if residual is None else _ld(residual), weight.data_ptr(), w_bias, eps, T, K,
              out.data_ptr(), _ld(out), None if h is None else h.data_ptr(),
              0 if h is None else _ld(h), _stream_of(x, stream))
    return out, (x if h is None else h)


def rmsnorm_int8(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                 residual: torch.Tensor | None = None, w_bias: float = 0.0,
                 out: torch.Tensor | None = None, scale: torch.Tensor | None = None,
                 residual_out: torch.Tensor | None = None, stream=None):
    """(q, scale, h): the rows of ``rmsnorm`` as int8 codes [T, K] and one fp32
    scale per row (y ~ q * scale, scale = max|y| / 127)."""
    T, K = _norm_args(x, weight, residual, residual_out)
    if out is None:
        out = _empty((T, K), torch.int8, x.device, stream)
    else:
        _rows(out, "out", (T, K), torch.int8)
    if scale is None:
        scale = _empty((T,), torch.float32, x.device, stream)
    else:
        _vec(scale, "scale", T, torch.float32)
    h = residual_out
    if h is None and residual is not None:
        h = _empty((T, K), _F16, x.device, stream)
    _lib.call("qz_rmsnorm_int8", x.data_ptr(), _ld(x),
              None if residual is None else residual.data_ptr(),
              0 if residual is None else _ld(residual), weight.data_ptr(), w_bias, eps, T, K,
              out.data_ptr(), _ld(out), scale.data_ptr(), None if h is None else h.data_ptr(),
              0 if h is None else _ld(h), _stream_of(x, stream))
    return out, scale, (x if h is None else h)


# ----------------------------------------------------------- paged cache ---
@dataclass
class PagedKV:
    """A paged key/value cache: k and v fp16 [n_pages, n_kv_heads, page_size,
    head_dim] with any strides that are multiples of 8 (a pool laid out
    [n_pages, page_size, n_kv_heads, head_dim] is given as .transpose(1, 2))."""
    k: torch.Tensor
    v: torch.Tensor
    _arg: object = field(default=None, repr=False, compare=False)

    def __post_init__(self):
        k, v = self.k, self.v
        _need(k.is_cuda and v.is_cuda, "libqz works on CUDA tensors only (no CPU fallback)")
        _need(k.dtype == _F16 and v.dtype == _F16 and k.dim() == 4 and k.shape == v.shape,
              "k and v: fp16 [n_pages, n_kv_heads, page_size, head_dim]")
        _need(k.stride(3) == 1 and v.stride(3) == 1, "k and v: contiguous head_dim")
        self._arg = _lib.KvCache(k.data_ptr(), v.data_ptr(), k.shape[0], k.shape[2], k.shape[1],
                                 k.shape[3], k.stride(0), k.stride(1), k.stride(2), v.stride(0),
                                 v.stride(1), v.stride(2))
        self._ref = ctypes.byref(self._arg)

    @classmethod
    def empty(cls, n_pages: int, n_kv_heads: int, page_size: int, head_dim: int,
              device="cuda") -> "PagedKV":
        shape = (n_pages, n_kv_heads, page_size, head_dim)
        return cls(torch.empty(shape, dtype=_F16, device=device),
                   torch.empty(shape, dtype=_F16, device=device))

    @property
    def n_kv_heads(self) -> int:
        return self.k.shape[1]

    @property
    def head_dim(self) -> int:
        return self.k.shape[3]


@dataclass
class SeqBatch:
    """The sequences of a step: cu_q int32 [S+1] (rows cu_q[i]..cu_q[i+1]-1 are
    the new tokens of sequence i), kv_len int32 [S] (tokens held, the new ones
    last), page_table int32 [S, pages].  The tensors' contents may change
    between calls (a captured graph replays with the new lengths)."""
    cu_q: torch.Tensor
    kv_len: torch.Tensor
    page_table: torch.Tensor
    _arg: object = field(default=None, repr=False, compare=False)

    def __post_init__(self):
        S = self.kv_len.shape[0]
        _vec(self.cu_q, "cu_q", S + 1, torch.int32)
        _vec(self.kv_len, "kv_len", S, torch.int32)
        _rows(self.page_table, "page_table", dtype=torch.int32)
        _need(self.page_table.shape[0] == S, "page_table: one row per sequence")
        # a row's stride bounds what may be read of it
        ld = self.page_table.stride(0) if S > 1 else self.page_table.shape[1]
        _need(ld >= self.page_table.shape[1], "page_table: rows must not overlap")
        self.page_table = self.page_table if ld == self.page_table.shape[1] \
            else self.page_table.contiguous()
        self._arg = _lib.SeqBatchArg(S, 0, self.cu_q.data_ptr(), self.kv_len.data_ptr(),
                                     self.page_table.data_ptr(), self.page_table.shape[1])
        self._ref = ctypes.byref(self._arg)

    @property
    def n_seqs(self) -> int:
        return self.kv_len.shape[0]


def _heads(t: torch.Tensor, what: str, T: int, heads: int | None, D: int) -> torch.Tensor:
    if not t.is_cuda:
        raise ValueError("libqz works on CUDA tensors only (no CPU fallback)")
    if t.dtype != _F16 or t.dim() != 3 or t.shape[0] != T or t.shape[2] != D or t.stride(2) != 1:
        raise ValueError(f"{what}: fp16 [{T}, heads, {D}] with contiguous rows is needed")
    if heads is not None and t.shape[1] != heads:
        raise ValueError(f"{what}: {t.shape[1]} heads, expected {heads}")
    return t


def rope_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cache: PagedKV,
                seqs: SeqBatch, rope: torch.Tensor | None, q_out: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """Rotate the new queries q [T, heads, D] (returned, in q_out; may be q) and
    keys k [T, kv_heads, D] by their positions, and store keys and values v
    into their slots of the cache.  rope: fp32 [positions, D], cosines then
    sines (``rope_table``), or None for no rotation."""
    T, D, hkv = q.shape[0], cache.head_dim, cache.n_kv_heads
    _heads(q, "q", T, None, D)
    _heads(k, "k", T, hkv, D)
    _heads(v, "v", T, hkv, D)
    if rope is not None and (rope.dtype != torch.float32 or rope.dim() != 2
                             or rope.shape[1] != D or not rope.is_contiguous()
                             or not rope.is_cuda):
        raise ValueError(f"rope: a contiguous fp32 CUDA tensor [positions, {D}] is needed")
    if q_out is None:
        q_out = _empty(q.shape, _F16, q.device, stream)
    else:
        _heads(q_out, "q_out", T, q.shape[1], D)
    seqs._arg.n_tokens = T
    _lib.call("qz_rope_append", q.data_ptr(), q.shape[1], q.stride(0), q.stride(1),
              k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(), v.stride(0), v.stride(1),
              None if rope is None else rope.data_ptr(), 0 if rope is None else rope.shape[0],
              cache._ref, seqs._ref, q_out.data_ptr(), q_out.stride(0), q_out.stride(1),
              _stream_of(q, stream))
    return q_out


def rope_table(positions: int, head_dim: int, theta: float = 10000.0,
               device="cuda") -> torch.Tensor:
    """fp32 [positions, head_dim]: cosines then sines of position * theta^(-2j/D)."""
    half = head_dim // 2
    f = theta ** (-torch.arange(half, dtype=torch.float64) / half)
    a = torch.arange(positions, dtype=torch.float64)[:, None] * f[None, :]
    return torch.cat([a.cos(), a.sin()], dim=1).float().to(device)


def attention_workspace(n_tokens: int, n_seqs: int, n_heads: int, n_kv_heads: int,
                        head_dim: int, device="cuda", stream=None) -> torch.Tensor:
    """A ready workspace (its counters zeroed) for attention_paged calls of up
    to that many tokens and sequences; calls that may overlap on the GPU need
    one each."""
    nbytes = int(_lib.load().qz_attention_workspace_bytes(n_tokens, n_seqs, n_heads, n_kv_heads,
                                                          head_dim))
    _need(nbytes > 0, "attention_workspace: invalid sizes")
    ws = _empty((nbytes,), torch.uint8, device, stream)
    with torch.cuda.stream(stream):
        ws[:_lib.QZ_ATTENTION_SYNC_BYTES].zero_()
    return ws


def attention_paged(q: torch.Tensor, cache: PagedKV, seqs: SeqBatch, scale: float | None = None,
                    softcap: float = 0.0, window: int = 0, out: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Causal attention of the new tokens q [T, heads, D] over the cache, which
    already holds their keys and values (``rope_append``).  scale defaults to
    D^-0.5; softcap > 0 caps logits as softcap * tanh(x / softcap); window > 0
    limits every query to its last `window` keys.  workspace: from
    ``attention_workspace`` (made here if None)."""
    T, D = q.shape[0], cache.head_dim
    _heads(q, "q", T, None, D)
    if q.shape[1] < 1 or q.shape[1] % cache.n_kv_heads:
        raise ValueError(f"q: {q.shape[1]} heads over {cache.n_kv_heads} KV heads")
    if out is None:
        out = _empty(q.shape, _F16, q.device, stream)
    else:
        _heads(out, "out", T, q.shape[1], D)
    if workspace is None:
        workspace = attention_workspace(T, seqs.n_seqs, q.shape[1], cache.n_kv_heads, D,
                                        q.device, stream)
    seqs._arg.n_tokens = T
    _lib.call("qz_attention_paged", q.data_ptr(), q.shape[1], q.stride(0), q.stride(1),
              cache._ref, seqs._ref, D ** -0.5 if scale is None else scale, softcap, window,
              out.data_ptr(), out.stride(0), out.stride(1), workspace.data_ptr(),
              workspace.numel(), _stream_of(q, stream))
    return out


# ------------------------------------------------------------------ LoRA ---
@dataclass
class LoraAdapters:
    """A pool of low-rank adapters of one projection: a fp16 [n, R, K], b fp16
    [n, N, R], scale fp32 [n], rank int32 [n] (None: every adapter has rank R)."""
    a: torch.Tensor
    b: torch.Tensor
    scale: torch.Tensor
    rank: torch.Tensor | None = None
    _arg: object = field(default=None, repr=False, compare=False)

    def __post_init__(self):
        a, b = self.a, self.b
        _need(a.is_cuda and b.is_cuda, "libqz works on CUDA tensors only (no CPU fallback)")
        _need(a.dtype == _F16 and b.dtype == _F16 and a.dim() == 3 and b.dim() == 3,
              "a and b: fp16 [n, R, K] and [n, N, R]")
        n, R, K = a.shape
        _need(b.shape[0] == n and b.shape[2] == R, "b: shape does not match a")
        _need((a.stride(2) == 1 or K == 1) and (b.stride(2) == 1 or R == 1),
              "a and b: contiguous rows")
        _vec(self.scale, "scale", n, torch.float32)
        if self.rank is not None:
            _vec(self.rank, "rank", n, torch.int32)
        self._arg = _lib.LoraArg(a.data_ptr(), b.data_ptr(), self.scale.data_ptr(),
                                 None if self.rank is None else self.rank.data_ptr(), n, R, K,
                                 b.shape[1], a.stride(0), a.stride(1) if R > 1 else K,
                                 b.stride(0), b.stride(1) if b.shape[1] > 1 else R)
        self._ref = ctypes.byref(self._arg)

    @property
    def K(self) -> int:
        return self.a.shape[2]

    @property
    def N(self) -> int:
        return self.b.shape[1]

    @property
    def R(self) -> int:
        return self.a.shape[1]


def lora_workspace(T: int, K: int, R: int, device="cuda", stream=None) -> torch.Tensor:
    """Workspace for lora calls of up to T rows (contents need not be kept)."""
    nbytes = int(_lib.load().qz_lora_workspace_bytes(T, K, R))
    _need(nbytes > 0, "lora_workspace: invalid sizes")
    return _empty((nbytes,), torch.uint8, device, stream)


def lora(x: torch.Tensor, y: torch.Tensor, adapters: LoraAdapters, index: torch.Tensor,
         out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
         stream=None) -> torch.Tensor:
    """out[t] = y[t] + scale_a * B_a (A_a x[t]) with a = index[t] (int32; -1: no
    adapter).  x [T, K] is the projection's input and y [T, N] its output (out
    may be y)."""
    T = x.shape[0]
    _rows(x, "x", (T, adapters.K))
    _rows(y, "y", (T, adapters.N))
    _vec(index, "index", T, torch.int32)
    if out is None:
        out = _empty((T, adapters.N), _F16, x.device, stream)
    else:
        _rows(out, "out", (T, adapters.N))
    if workspace is None:
        workspace = lora_workspace(T, adapters.K, adapters.R, x.device, stream)
    _lib.call("qz_lora", adapters._ref, index.data_ptr(), T, x.data_ptr(), _ld(x), y.data_ptr(),
              _ld(y), out.data_ptr(), _ld(out), workspace.data_ptr(), workspace.numel(),
              _stream_of(x, stream))
    return out
