"""Inputs and bounds of the layer operators' tests at depth, on any device: what is
checked on the GPU is checked on the host too, for what the bounds can see."""
import torch

F16, F64 = torch.float16, torch.float64
U16, S16 = 2.0 ** -11, 2.0 ** -24  # one rounding to fp16: relative, and absolute below its range


# --------------------------------------------------------------- adapters ---
# (rows, rows of an adapter in turn, adapters, rank, K, N, mixed ranks, offset in halves):
# calls of many rows, whose CTAs take 16 and 32 rows in both products
ADAPTERS = [(1500, 300, 8, 64, 4096, 11008, True, 0), (1500, 1, 48, 16, 4096, 11008, False, 0),
            (1500, 7, 20, 64, 2048, 4096, False, 0), (1500, 1, 9, 100, 4104, 4096, True, 0),
            (1500, 300, 5, 104, 8192, 1032, True, 0), (500, 3, 7, 64, 4096, 4104, True, 0),
            (500, 1, 500, 8, 512, 4096, False, 0), (500, 60, 4, 128, 4096, 4100, True, 0),
            (700, 90, 6, 32, 2050, 2050, False, 1), (1400, 1, 33, 40, 8192, 4160, False, 1),
            (260, 260, 1, 64, 4096, 11008, False, 0), (40, 40, 2, 16, 4096, 65536, False, 0)]


def adapter_index(T, run, n):
    """Adapter of every row: runs of equal rows, one run in seven without one."""
    return [-1 if (t // run) % 7 == 6 else (t // run) * 5 % n for t in range(T)]


def adapter_reference(x, y, a, b, scale, rank, index):
    """(out, bound) in 64 bits.  The bound: out's one rounding to fp16; every u_r off by
    its sum's roundings (64 at most one after another, of partial sums that stay below 8
    times the root of the sum of squares; a tensor core's may be a whole unit, 2^-23) and
    by 2^-22 of its row's largest (two fp16 parts); the second product's sums alike."""
    T, R = x.shape[0], a.shape[1]
    out, tol = y.to(F64).clone(), torch.zeros(y.shape, dtype=F64, device=y.device)
    idx = torch.as_tensor(index, device=x.device)
    for i in set(index) - {-1}:
        rows = (idx == i).nonzero()[:, 0]
        r = R if rank is None else max(0, min(R, rank[i]))
        A, B, s = a[i, :r].to(F64), b[i, :, :r].to(F64), float(scale[i])
        X = x[rows].to(F64)
        u = X @ A.T
        du = 64 * 2.0 ** -23 * 8 * (X.square() @ A.square().T).sqrt()
        if r:
            du = du + 2.0 ** -22 * u.abs().amax(1, keepdim=True)
        out[rows] += s * (u @ B.T)
        tol[rows] = abs(s) * (du @ B.abs().T + 32 * 2.0 ** -23 * (u.abs() @ B.abs().T))
    return out, tol + U16 * out.abs() + S16


def cancelling_adapters(T, n, R, K, N, device):
    """(x, y, a, b, index, out): u_r = 1024 + c / 16 takes 15 bits, and every output is
    y plus the difference of two of them, of which the 1024 leaves nothing.  All sums are
    exact in fp32 and out is exact in fp16."""
    step = (K // 2) // R
    j = torch.arange(R, device=device) * step
    t = torch.arange(T, device=device)[:, None]
    c = (t * 7 + torch.arange(R, device=device)[None, :] * 5) % 16
    x = torch.zeros((T, K), dtype=F16, device=device)
    x[:, j] = 1024.0
    x[:, K // 2 + j] = (c / 16).to(F16)
    a = torch.zeros((n, R, K), dtype=F16, device=device)
    a[:, torch.arange(R, device=device), j] = 1.0
    a[:, torch.arange(R, device=device), K // 2 + j] = 1.0
    i = torch.arange(N, device=device)
    b = torch.zeros((n, N, R), dtype=F16, device=device)
    for k in range(n):
        b[k, i, (i + k) % R] = 1.0
        b[k, i, (i + k + 1) % R] = -1.0
    index = (torch.arange(T, device=device) + 1) % (n + 1) - 1
    y = ((t * 3 + i[None, :]) % 64 / 16).to(F16)
    first = (i[None, :] + index.clamp(min=0)[:, None]) % R
    d = (c.gather(1, first) - c.gather(1, (first + 1) % R)) / 16
    out = y.to(F64) + torch.where(index[:, None] >= 0, d.to(F64), 0.0)
    return x, y, a, b, index.to(torch.int32), out


# -------------------------------------------------------------- attention ---
BLOCK = 128  # keys that the kernel takes at a time

# (new tokens, tokens held, heads, KV heads, D, page, window): long contexts, cut
# between many CTAs, and tiles of many blocks that one CTA walks through
CONTEXTS = [([1], [40000], 8, 1, 128, 64, 0), ([1, 1, 1], [20001, 7, 12345], 4, 2, 256, 128, 0),
            ([17, 2], [30000, 9000], 8, 2, 128, 16, 0), ([1, 1], [40000, 33333], 8, 2, 64, 32, 0),
            ([150, 1], [20000, 40000], 4, 2, 128, 64, 0), ([300], [9999], 4, 1, 64, 128, 0),
            ([40], [15000], 2, 2, 256, 64, 0), ([1, 60], [40000, 30000], 4, 1, 128, 16, 17000),
            ([1] * 40, [1500 + 97 * i for i in range(40)], 8, 4, 128, 32, 0)]


def signal_inputs(qs, kvs, hq, hkv, D, seed, device):
    """(queries of all sequences, keys and values of each).  Channel c of the values tells
    of the key blocks c, c + D, c + 2 D, ...: it is 1 to 2 there and 0 elsewhere, so that one
    output channel comes from five blocks at most.  The logits rise and fall by 2 from block
    to block (through channel 0 of the keys) around small random ones."""
    g = torch.Generator(device=device).manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=device)

    q = randn(sum(qs), hq, D) * 0.4
    q[..., 0] = D ** 0.5
    ks, vs = [], []
    for n in kvs:
        j = torch.arange(n, device=device)
        b = j // BLOCK
        k = randn(n, hkv, D)
        k[..., 0] = (2.0 * torch.sin(b * 0.7 + 0.1 * (j % BLOCK) / BLOCK))[:, None]
        v = torch.zeros((n, hkv, D), device=device)
        h = torch.arange(hkv, device=device)[None, :]
        v[j[:, None], h, b[:, None] % D] = 1.0 + (j[:, None] * 13 + h) % 8 / 8
        ks.append(k.to(F16))
        vs.append(v.to(F16))
    return q.to(F16), ks, vs


def weights(q, k, pos, window, scale):
    """(e^(x - max) of one head's rows, the largest sum of |q k| a row) in 64 bits."""
    j = torch.arange(k.shape[0], device=k.device)[None, :]
    seen = j <= pos[:, None]
    if window:
        seen &= j > pos[:, None] - window
    q, k = q.to(F64), k.to(F64)
    x = (q @ k.T * scale).masked_fill(~seen, float("-inf"))
    dot = (q.abs() @ k.abs().T * scale).masked_fill(~seen, 0.0).amax(1)
    return torch.exp(x - x.amax(1, keepdim=True)), dot


def signal_bound(out, w, v, dot, D):
    """Roundings of out = w v / sum(w), v >= 0: every weight to fp16 (relative, and half of
    the smallest fp16 beside the largest weight), logits by fp32 sums of D products and
    their exponential, the output once; sums of positive fp32 terms, a tensor core's with up
    to 2^-23 for each of a block's 8 steps, block after block (a drift of 2^-12 at 40000)."""
    rel = 2 * U16 + 2 * (D + 64) * 2.0 ** -24 * (dot[:, None] + 1) + 2.0 ** -12
    small = (w > 0).to(F64) @ v * (S16 / 2) / w.sum(1, keepdim=True)
    return rel * out + small + S16


def signal_reference(q, ks, vs, qs, kvs, hq, window):
    """(out, bound) of all rows."""
    D, G = q.shape[2], hq // ks[0].shape[1]
    out, tol, t = torch.empty(q.shape, dtype=F64, device=q.device), None, 0
    tol = torch.empty_like(out)
    for n, L, k, v in zip(qs, kvs, ks, vs):
        pos = torch.arange(L - n, L, device=q.device)
        for h in range(hq):
            w, dot = weights(q[t:t + n, h], k[:, h // G], pos, window, D ** -0.5)
            vv = v[:, h // G].to(F64)
            o = w @ vv / w.sum(1, keepdim=True)
            out[t:t + n, h], tol[t:t + n, h] = o, signal_bound(o, w, vv, dot, D)
        t += n
    return out, tol
