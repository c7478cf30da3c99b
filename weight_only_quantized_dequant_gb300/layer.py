"""The steps of a decoder layer around its quantized products, as thin calls
of the library (include/qz.h, "Layer glue for serving"): ``rmsnorm`` and
``rmsnorm_int8``, ``rope_append`` and ``attention_paged`` over a ``PagedKV``
(fp16) or ``PagedKVInt8`` cache, ``cache_read`` of the latter, ``lora`` for the
low-rank adapters beside a shared projection, and ``sample`` for the choice of
the next tokens from their logits.

Every function takes ``stream`` (default: the current one); outputs and
workspaces that a call allocates belong to that stream.  All tensors of a call
lie on the current device.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass, field

import torch

from . import _lib

_F16, _F32, _I32 = torch.float16, torch.float32, torch.int32
_raw_stream = torch._C._cuda_getCurrentRawStream  # torch.cuda.current_stream() costs 10x as much
_current_device = torch._C._cuda_getDevice  # any tensor on a GPU has started CUDA by then

# A decode step makes hundreds of these calls and the kernels of small batches
# take a few microseconds, so the checks below are few attribute reads each and
# the library is called without another layer.


def _stream_of(dev: int, stream) -> int:
    return _raw_stream(dev) if stream is None else stream.cuda_stream


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """torch.empty on the stream the call runs on, so that the memory is not
    handed to other streams while the kernels use it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _like(t: torch.Tensor, stream) -> torch.Tensor:
    """A contiguous tensor of t's shape and type, allocated as by _empty."""
    if stream is None and t.is_contiguous():
        return torch.empty_like(t)
    return _empty(t.shape, t.dtype, t.device, stream)


# Handles hold the addresses of their tensors for the kernels, made once, so their
# fields are frozen; a handle with another tensor is dataclasses.replace(handle, ...).
def _set(handle, **values) -> None:
    for name, v in values.items():
        object.__setattr__(handle, name, v)


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _cuda_or_raise(t) -> None:
    if not t.is_cuda:
        raise ValueError("libqz works on CUDA tensors only (no CPU fallback)")


def _place_or_raise(t, what: str, dev: int) -> None:
    """Why t does not lie on GPU dev, if so."""
    _cuda_or_raise(t)
    if t.get_device() != dev:
        raise ValueError(f"{what}: on GPU {t.get_device()}, but the call runs on GPU {dev}")


def _wrong_device(t, what: str) -> None:
    _cuda_or_raise(t)
    raise ValueError(f"{what}: on GPU {t.get_device()}, but the current device is GPU "
                     f"{_current_device()}; torch.cuda.device selects another")


def _device(t: torch.Tensor, what: str) -> int:
    """The GPU of a call's first operand: the current one, where the library launches."""
    dev = t.get_device()
    if dev < 0 or dev != _current_device():
        _wrong_device(t, what)
    return dev


def _rows(t: torch.Tensor, what: str, dev: int, shape, dtype=_F16) -> int:
    """Row stride of a matrix with contiguous rows on GPU dev (that of a single row,
    which torch may report as anything, is its length)."""
    if t.get_device() == dev and t.dtype is dtype and t.shape == shape:
        if t.is_contiguous():
            return shape[1]
        if t.stride(1) == 1 or shape[1] <= 1:
            return t.stride(0) if shape[0] > 1 else shape[1]
    _place_or_raise(t, what, dev)
    raise ValueError(f"{what}: {t.dtype} {tuple(t.shape)} with strides {t.stride()}; a {dtype} "
                     f"matrix {tuple(shape)} with contiguous rows is needed")


def _vec(t: torch.Tensor, what: str, dev: int, n: int, dtype) -> int:
    """Address of a contiguous vector of n on GPU dev."""
    if t.get_device() == dev and t.dtype is dtype and t.shape == (n,) and t.is_contiguous():
        return t.data_ptr()
    _place_or_raise(t, what, dev)
    raise ValueError(f"{what}: a contiguous {dtype} vector of {n} is needed")


def _space(t: torch.Tensor, dev: int) -> int:
    """Bytes of a workspace on GPU dev."""
    if t.get_device() == dev and t.is_contiguous():
        return t.nbytes
    _place_or_raise(t, "workspace", dev)
    raise ValueError("workspace: a contiguous tensor is needed")


def _far(handle, what: str, dev: int) -> None:
    raise ValueError(f"{what}: on GPU {handle.device_index}, but the call runs on GPU {dev}")


# ------------------------------------------------------------------ norm ---
def rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
            residual: torch.Tensor | None = None, w_bias: float = 0.0,
            out: torch.Tensor | None = None, residual_out: torch.Tensor | None = None,
            stream=None):
    """(y, h): h = x + residual and y = h * rsqrt(mean(h^2) + eps) * (w_bias +
    weight) for fp16 rows x [T, K].  h, the next residual, goes to residual_out
    (may be residual or x; allocated if None); without a residual h is x itself
    and is not written."""
    shape = x.shape
    _need(len(shape) == 2, "x: two dimensions are needed")
    T, K = shape
    dev = _device(x, "x")
    ldx = _rows(x, "x", dev, shape)
    w = _vec(weight, "weight", dev, K, _F16)
    r = ldr = h = ldh = 0
    if residual is not None:
        r, ldr = residual.data_ptr(), _rows(residual, "residual", dev, shape)
        if residual_out is None:
            residual_out = _like(x, stream)
    if residual_out is not None:
        h, ldh = residual_out.data_ptr(), _rows(residual_out, "residual_out", dev, shape)
    if out is None:
        out = _like(x, stream)
    ldy = _rows(out, "out", dev, shape)
    st = _lib.load().qz_rmsnorm(x.data_ptr(), ldx, r, ldr, w, w_bias, eps, T, K, out.data_ptr(),
                                ldy, h, ldh, _stream_of(dev, stream))
    if st:
        _lib.fail("qz_rmsnorm", st)
    return out, (x if residual_out is None else residual_out)


def rmsnorm_int8(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                 residual: torch.Tensor | None = None, w_bias: float = 0.0,
                 out: torch.Tensor | None = None, scale: torch.Tensor | None = None,
                 residual_out: torch.Tensor | None = None, stream=None):
    """(q, scale, h): the rows of ``rmsnorm`` as int8 codes [T, K] and one fp32
    scale per row (y ~ q * scale, scale = max|y| / 127; a row that is not finite
    gets such a scale)."""
    shape = x.shape
    _need(len(shape) == 2, "x: two dimensions are needed")
    T, K = shape
    dev = _device(x, "x")
    ldx = _rows(x, "x", dev, shape)
    w = _vec(weight, "weight", dev, K, _F16)
    r = ldr = h = ldh = 0
    if residual is not None:
        r, ldr = residual.data_ptr(), _rows(residual, "residual", dev, shape)
        if residual_out is None:
            residual_out = _like(x, stream)
    if residual_out is not None:
        h, ldh = residual_out.data_ptr(), _rows(residual_out, "residual_out", dev, shape)
    if out is None:
        out = _empty(shape, torch.int8, x.device, stream)
    ldq = _rows(out, "out", dev, shape, torch.int8)
    if scale is None:
        scale = _empty((T,), _F32, x.device, stream)
    s = _vec(scale, "scale", dev, T, _F32)
    st = _lib.load().qz_rmsnorm_int8(x.data_ptr(), ldx, r, ldr, w, w_bias, eps, T, K,
                                     out.data_ptr(), ldq, s, h, ldh, _stream_of(dev, stream))
    if st:
        _lib.fail("qz_rmsnorm_int8", st)
    return out, scale, (x if residual_out is None else residual_out)


# ----------------------------------------------------------- paged cache ---
@dataclass(frozen=True)
class PagedKV:
    """A paged key/value cache: k and v fp16 [n_pages, n_kv_heads, page_size,
    head_dim] with any strides that are multiples of 8 (a pool laid out
    [n_pages, page_size, n_kv_heads, head_dim] is given as .transpose(1, 2))."""
    k: torch.Tensor
    v: torch.Tensor
    _arg: object = field(default=None, repr=False, compare=False)

    def __post_init__(self):
        k, v = self.k, self.v
        _cuda_or_raise(k)
        dev = k.get_device()
        _place_or_raise(v, "v", dev)
        _need(k.dtype == _F16 and v.dtype == _F16 and k.dim() == 4 and k.shape == v.shape,
              "k and v: fp16 [n_pages, n_kv_heads, page_size, head_dim]")
        _need(k.stride(3) == 1 and v.stride(3) == 1, "k and v: contiguous head_dim")
        pages, heads, size, D = k.shape  # a single page, head or token has no stride of its own
        k_st, v_st = ([s if n > 1 else D for s, n in zip(t.stride(), k.shape)] for t in (k, v))
        arg = _lib.KvCache(k.data_ptr(), v.data_ptr(), pages, size, heads, D, *k_st[:3], *v_st[:3])
        _set(self, _arg=arg, _ref=ctypes.byref(arg), shape=tuple(k.shape), device_index=dev)

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


@dataclass(frozen=True)
class PagedKVInt8:
    """A paged key/value cache of INT8 rows: k and v int8 codes [n_pages, n_kv_heads,
    page_size, head_dim] with contiguous head_dim and other strides that are
    multiples of 16, k_scale and v_scale fp32 [n_pages, n_kv_heads, page_size] with
    any strides; a row stands for its codes times its scale."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor
    _arg: object = field(default=None, repr=False, compare=False)

    def __post_init__(self):
        k, v, ks, vs = self.k, self.v, self.k_scale, self.v_scale
        _cuda_or_raise(k)
        dev = k.get_device()
        for t, what in ((v, "v"), (ks, "k_scale"), (vs, "v_scale")):
            _place_or_raise(t, what, dev)
        _need(k.dtype == torch.int8 and v.dtype == torch.int8 and k.dim() == 4
              and k.shape == v.shape, "k and v: int8 [n_pages, n_kv_heads, page_size, head_dim]")
        _need(k.stride(3) == 1 and v.stride(3) == 1, "k and v: contiguous head_dim")
        _need(ks.dtype == _F32 and vs.dtype == _F32 and ks.shape == k.shape[:3]
              and vs.shape == k.shape[:3],
              "k_scale and v_scale: fp32 [n_pages, n_kv_heads, page_size]")
        pages, heads, size, D = k.shape  # a single page, head or token has no stride of its own
        st = [[s if n > 1 else least for s, n in zip(t.stride(), k.shape[:3])]
              for t, least in ((k, D), (v, D), (ks, 1), (vs, 1))]
        arg = _lib.KvCacheInt8(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), pages,
                               size, heads, D, *st[0], *st[1], *st[2], *st[3])
        _set(self, _arg=arg, _ref=ctypes.byref(arg), shape=tuple(k.shape), device_index=dev)

    @classmethod
    def empty(cls, n_pages: int, n_kv_heads: int, page_size: int, head_dim: int,
              device="cuda") -> "PagedKVInt8":
        shape = (n_pages, n_kv_heads, page_size, head_dim)
        return cls(*(torch.empty(shape, dtype=torch.int8, device=device) for _ in range(2)),
                   *(torch.empty(shape[:3], dtype=_F32, device=device) for _ in range(2)))

    @property
    def n_kv_heads(self) -> int:
        return self.k.shape[1]

    @property
    def head_dim(self) -> int:
        return self.k.shape[3]


@dataclass(frozen=True)
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
        S, dev = self.kv_len.shape[0], self.kv_len.get_device()
        _vec(self.kv_len, "kv_len", dev, S, _I32)
        _vec(self.cu_q, "cu_q", dev, S + 1, _I32)
        _need(self.page_table.dim() == 2 and self.page_table.shape[0] == S,
              "page_table: one row per sequence")
        # the row stride is also the number of entries that may be read
        _need(_rows(self.page_table, "page_table", dev, self.page_table.shape, _I32)
              == self.page_table.shape[1], "page_table: a contiguous table is needed")
        _set(self, _arg=(self.cu_q.data_ptr(), self.kv_len.data_ptr(),
                         self.page_table.data_ptr(), self.page_table.shape[1]),
             n_seqs=S, device_index=dev, _last=(-1, None))

    def _ref(self, n_tokens: int):
        """The library's view of a step of n_tokens rows.  Another thread may call with
        another count, so a view is never changed once it is made."""
        n, ref = self._last
        if n != n_tokens:
            ref = ctypes.byref(_lib.SeqBatchArg(self.n_seqs, n_tokens, *self._arg))
            _set(self, _last=(n_tokens, ref))
        return ref


def _heads(t: torch.Tensor, what: str, dev: int, T: int, heads: int, D: int):
    """Token and head strides of an fp16 [T, heads, D] with contiguous rows on GPU dev (a
    single token or head has none of its own: torch may report anything)."""
    if t.get_device() == dev and t.dtype is _F16 and t.shape == (T, heads, D):
        st, sh, sd = t.stride()
        if sd == 1:
            return st if T > 1 else heads * D, sh if heads > 1 else D
    _place_or_raise(t, what, dev)
    raise ValueError(f"{what}: {t.dtype} {tuple(t.shape)} with strides {t.stride()}; fp16 "
                     f"{(T, heads, D)} with contiguous rows is needed")


def rope_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cache: PagedKV | PagedKVInt8,
                seqs: SeqBatch, rope: torch.Tensor | None, q_out: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """Rotate the new queries q [T, heads, D] (returned, in q_out; may be q) and
    keys k [T, kv_heads, D] by their positions, and store keys and values v
    into their slots of the cache (as INT8 rows in a PagedKVInt8: scale = max|x| /
    127, code = round(x / scale)).  rope: fp32 [positions, D], cosines then
    sines (``rope_table``), or None for no rotation."""
    _need(q.dim() == 3, "q: three dimensions are needed")
    T, H, _ = q.shape
    _, hkv, _, D = cache.shape
    dev = _device(q, "q")
    if cache.device_index != dev:
        _far(cache, "cache", dev)
    if seqs.device_index != dev:
        _far(seqs, "seqs", dev)
    qt, qh = _heads(q, "q", dev, T, H, D)
    kt, kh = _heads(k, "k", dev, T, hkv, D)
    vt, vh = _heads(v, "v", dev, T, hkv, D)
    rp = n = 0
    if rope is not None:
        if not (rope.get_device() == dev and rope.dtype is _F32 and rope.dim() == 2
                and rope.shape[1] == D and rope.is_contiguous()):
            _place_or_raise(rope, "rope", dev)
            raise ValueError(f"rope: a contiguous fp32 CUDA tensor [positions, {D}] is needed")
        rp, n = rope.data_ptr(), rope.shape[0]
    if q_out is None:
        q_out, ot, oh = _empty((T, H, D), _F16, q.device, stream), H * D, D
    else:
        ot, oh = _heads(q_out, "q_out", dev, T, H, D)
    lib = _lib.load()
    name = "qz_rope_append_int8" if isinstance(cache, PagedKVInt8) else "qz_rope_append"
    st = getattr(lib, name)(q.data_ptr(), H, qt, qh, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh,
                            rp, n, cache._ref, seqs._ref(T), q_out.data_ptr(), ot, oh,
                            _stream_of(dev, stream))
    if st:
        _lib.fail(name, st)
    return q_out


def cache_read(cache: PagedKVInt8, seqs: SeqBatch, n_tokens: int, k: torch.Tensor | None = None,
               v: torch.Tensor | None = None, stream=None):
    """(k, v): the cache's rows of the n_tokens tokens that seqs describes, as fp16
    [n_tokens, kv_heads, D] (codes times scales).  The sequences of a step give its
    new tokens; with cu_q the running sums of kv_len, all that is held."""
    _need(isinstance(cache, PagedKVInt8), "cache: a PagedKVInt8 is needed")
    _, hkv, _, D = cache.shape
    dev = _device(cache.k, "cache")
    if seqs.device_index != dev:
        _far(seqs, "seqs", dev)
    _need(n_tokens >= 0, "n_tokens: negative")
    shape = (n_tokens, hkv, D)
    if k is None:
        k, kt, kh = _empty(shape, _F16, cache.k.device, stream), hkv * D, D
    else:
        kt, kh = _heads(k, "k", dev, *shape)
    if v is None:
        v, vt, vh = _empty(shape, _F16, cache.k.device, stream), hkv * D, D
    else:
        vt, vh = _heads(v, "v", dev, *shape)
    st = _lib.load().qz_cache_read_int8(cache._ref, seqs._ref(n_tokens), k.data_ptr(), kt, kh,
                                        v.data_ptr(), vt, vh, _stream_of(dev, stream))
    if st:
        _lib.fail("qz_cache_read_int8", st)
    return k, v


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


def attention_paged(q: torch.Tensor, cache: PagedKV | PagedKVInt8, seqs: SeqBatch,
                    scale: float | None = None, softcap: float = 0.0, window: int = 0,
                    out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """Causal attention of the new tokens q [T, heads, D] over the cache, which
    already holds their keys and values (``rope_append``).  scale defaults to
    D^-0.5; softcap > 0 caps logits as softcap * tanh(x / softcap); window > 0
    limits every query to its last `window` keys.  workspace: from
    ``attention_workspace`` (made here if None)."""
    _need(q.dim() == 3, "q: three dimensions are needed")
    T, H, _ = q.shape
    _, hkv, _, D = cache.shape
    dev = _device(q, "q")
    if cache.device_index != dev:
        _far(cache, "cache", dev)
    if seqs.device_index != dev:
        _far(seqs, "seqs", dev)
    qt, qh = _heads(q, "q", dev, T, H, D)
    if H < 1 or H % hkv:
        raise ValueError(f"q: {H} heads over {hkv} KV heads")
    if out is None:
        out, ot, oh = _empty((T, H, D), _F16, q.device, stream), H * D, D
    else:
        ot, oh = _heads(out, "out", dev, T, H, D)
    if workspace is None:
        workspace = attention_workspace(T, seqs.n_seqs, H, hkv, D, q.device, stream)
    nbytes = _space(workspace, dev)
    lib = _lib.load()
    name = ("qz_attention_paged_int8" if isinstance(cache, PagedKVInt8) else
            "qz_attention_paged")
    st = getattr(lib, name)(q.data_ptr(), H, qt, qh, cache._ref, seqs._ref(T),
                            D ** -0.5 if scale is None else scale, softcap, window, out.data_ptr(),
                            ot, oh, workspace.data_ptr(), nbytes, _stream_of(dev, stream))
    if st:
        _lib.fail(name, st)
    return out


# ------------------------------------------------------------------ LoRA ---
@dataclass(frozen=True)
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
        _cuda_or_raise(a)
        dev = a.get_device()
        _place_or_raise(b, "b", dev)
        _need(a.dtype == _F16 and b.dtype == _F16 and a.dim() == 3 and b.dim() == 3,
              "a and b: fp16 [n, R, K] and [n, N, R]")
        n, R, K = a.shape
        _need(b.shape[0] == n and b.shape[2] == R, "b: shape does not match a")
        _need((a.stride(2) == 1 or K == 1) and (b.stride(2) == 1 or R == 1),
              "a and b: contiguous rows")
        _vec(self.scale, "scale", dev, n, _F32)
        if self.rank is not None:
            _vec(self.rank, "rank", dev, n, _I32)
        arg = _lib.LoraArg(a.data_ptr(), b.data_ptr(), self.scale.data_ptr(),
                           None if self.rank is None else self.rank.data_ptr(), n, R, K,
                           b.shape[1], a.stride(0), a.stride(1) if R > 1 else K,
                           b.stride(0), b.stride(1) if b.shape[1] > 1 else R)
        _set(self, _arg=arg, _ref=ctypes.byref(arg), sizes=(K, R, b.shape[1]), device_index=dev)

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
    _need(x.dim() == 2, "x: two dimensions are needed")
    T, K, R, N = x.shape[0], *adapters.sizes
    dev = _device(x, "x")
    if adapters.device_index != dev:
        _far(adapters, "adapters", dev)
    ldx = _rows(x, "x", dev, (T, K))
    ldy = _rows(y, "y", dev, (T, N))
    i = _vec(index, "index", dev, T, _I32)
    if out is None:
        out = _like(y, stream)
    ldo = _rows(out, "out", dev, (T, N))
    if workspace is None:
        workspace = lora_workspace(T, K, R, x.device, stream)
    nbytes = _space(workspace, dev)
    st = _lib.load().qz_lora(adapters._ref, i, T, x.data_ptr(), ldx, y.data_ptr(), ldy,
                             out.data_ptr(), ldo, workspace.data_ptr(), nbytes,
                             _stream_of(dev, stream))
    if st:
        _lib.fail("qz_lora", st)
    return out


# ---------------------------------------------------------------- sample ---
_LOGITS = {_F16: 0, torch.bfloat16: 1, _F32: 2}


def _option(v, what: str, dev: int, B: int, dtype):
    """(address, value) of an option of every row, or of all."""
    if isinstance(v, torch.Tensor):
        return _vec(v, what, dev, B, dtype), 0
    return None, v


def sample(logits: torch.Tensor, u: torch.Tensor, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0,
           out: torch.Tensor | None = None, logprob: torch.Tensor | None = None, stream=None):
    """(tokens, logprob): a token int32 [B] for every row of logits [B, V] (fp16, bf16
    or fp32), the first whose running probability, by index, exceeds u (fp32 [B], in
    [0, 1)), and the logarithm of its probability.  Probabilities are those of
    softmax(logits / temperature) with the top_k largest kept (0: all), of those the
    fewest of probability top_p together, of those the ones with at least min_p of the
    largest.  temperature 0 takes the largest logit.  Every option is a number or a
    tensor [B] (fp32; top_k int32).  A row without a logit above -inf gives token -1."""
    _need(logits.dim() == 2, "logits: two dimensions are needed")
    B, V = logits.shape
    dev = _device(logits, "logits")
    kind = _LOGITS.get(logits.dtype)
    _need(kind is not None, "logits: fp16, bf16 or fp32 is needed")
    _need(V >= 1, "logits: a vocabulary is needed")
    ld = _rows(logits, "logits", dev, (B, V), logits.dtype)
    up = _vec(u, "u", dev, B, _F32)
    t, t_all = _option(temperature, "temperature", dev, B, _F32)
    k, k_all = _option(top_k, "top_k", dev, B, _I32)
    p, p_all = _option(top_p, "top_p", dev, B, _F32)
    m, m_all = _option(min_p, "min_p", dev, B, _F32)
    _need(-2 ** 31 <= k_all < 2 ** 31, "top_k: 32 bits")
    if out is None:
        out = _empty((B,), _I32, logits.device, stream)
    else:
        _vec(out, "out", dev, B, _I32)
    if logprob is None:
        logprob = _empty((B,), _F32, logits.device, stream)
    else:
        _vec(logprob, "logprob", dev, B, _F32)
    opts = _lib.Sampling(t, k, p, m, t_all, k_all, p_all, m_all)
    st = _lib.load().qz_sample(logits.data_ptr(), kind, B, V, ld, up, ctypes.byref(opts),
                               out.data_ptr(), logprob.data_ptr(), _stream_of(dev, stream))
    if st:
        _lib.fail("qz_sample", st)
    return out, logprob
