"""Cases of the operators around the quantized products of a decoder layer.

A decode or prompt step of the served stack runs, beside its INT8 / INT4
products: the residual addition with root-mean-square normalisation
(``rmsnorm``, ``rmsnorm_int8``), the rotation of queries and keys and their
storage into a paged cache (``rope_append``), the attention of the new tokens
over that cache (``attention_paged``), and the low-rank adapters of the
requests beside a shared projection (``lora``).  Each case is one call.

``own`` selects what ``run`` computes: False, the operators in elementary
torch operations held in 32 bits; True, the framework's kernels.
"""
import math

import torch

own = False

DEV = "cuda"
H = torch.float16


# ------------------------------------------------------------------ cases ---
def _norm(name, rows, K, residual=True, int8=False, bias=0.0):
    return {"name": name, "op": "rmsnorm", "rows": rows, "K": K, "residual": residual,
            "int8": int8, "bias": bias}


def _append(name, seqs, q, past, hq, hkv, D, page):
    return {"name": name, "op": "append", "seqs": seqs, "q": q, "past": past, "hq": hq,
            "hkv": hkv, "D": D, "page": page}


def _attn(name, seqs, q, past, hq, hkv, D, page, softcap=0.0, window=0):
    return {"name": name, "op": "attention", "seqs": seqs, "q": q, "past": past, "hq": hq,
            "hkv": hkv, "D": D, "page": page, "softcap": softcap, "window": window}


def _lora(name, rows, run, adapters, R, K, N, mixed=False):
    return {"name": name, "op": "lora", "rows": rows, "run": run, "adapters": adapters, "R": R,
            "K": K, "N": N, "mixed": mixed}


def listed():
    return [
        # the 70B-shaped stack's norm before a projection: 16 requests, one token each
        _norm("norm_16x8192", 16, 8192),
        # a prompt chunk through the same norm
        _norm("norm_2048x8192", 2048, 8192),
        # Gemma-2-9B-shaped rows, weight stored as w - 1, output as INT8 rows with scales
        _norm("norm_int8_1021x3584", 1021, 3584, int8=True, bias=1.0),
        # one decode step of 64 requests on the 7B-shaped stack (as many KV heads as heads)
        _append("append_64x1_h32", 64, 1, 2000, 32, 32, 128, 16),
        # packed chunks of different lengths on the 70B-shaped stack
        _append("append_9x300_h64kv8", 9, 300, 1000, 64, 8, 128, 64),
        # the smallest serving step: one request, one token, a short context
        _attn("attn_1x1_ctx200_h32kv8", 1, 1, 199, 32, 8, 128, 16),
        # a decode step of 32 requests with contexts up to 16k on the 70B-shaped stack
        _attn("attn_32x1_ctx16k_h64kv8", 32, 1, 16383, 64, 8, 128, 64),
        # Gemma-2-9B-shaped local layer: head size 256, capped logits, a window of 4096
        _attn("attn_8x1_ctx8k_d256_cap_win", 8, 1, 8000, 16, 8, 256, 32, softcap=50.0,
              window=4096),
        # chunks of new tokens beside long contexts (chunked prompts, verified drafts)
        _attn("attn_4x64_ctx24k_h64kv8", 4, 64, 24000, 64, 8, 128, 64),
        # whole prompts of different lengths, packed, on the 7B-shaped stack
        _attn("attn_4x4096_prompt_h32", 4, 4096, 0, 32, 32, 128, 64),
        # 32 requests with an adapter each beside a 70B-shaped projection
        _lora("lora_32_r16_8192x8192", 32, 1, 32, 16, 8192, 8192),
        # packed prompt rows of a few adapters of different ranks beside a 7B-shaped projection
        _lora("lora_1500_r64_4096x11008", 1500, 300, 8, 64, 4096, 11008, mixed=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


# (heads, KV heads, head size): the stacks' own, and groups that are odd or cover every head
_HEADS = [(32, 32, 128), (64, 8, 128), (16, 8, 256), (32, 8, 128), (32, 8, 64), (12, 4, 128),
          (5, 1, 64), (16, 16, 64), (8, 1, 256), (28, 4, 128)]


def draw(rng):
    op = rng.choice(["rmsnorm", "append", "attention", "attention", "lora"])
    if op == "rmsnorm":
        K = rng.choice([2048, 3584, 4096, 8192, _log(rng, 64, 16384)])
        return _norm("", _log(rng, 1, 2048), K, rng.random() < 0.75, rng.random() < 0.4,
                     float(rng.random() < 0.3))
    if op == "append":
        hq, hkv, D = rng.choice(_HEADS)
        return _append("", _log(rng, 1, 64), _log(rng, 1, 300), _log(rng, 1, 2000), hq, hkv, D,
                       rng.choice([16, 32, 64, 128]))
    if op == "attention":
        largest = listed()[9]
        while True:
            hq, hkv, D = rng.choice(_HEADS)
            q = rng.choice([1, 1, _log(rng, 2, 64), _log(rng, 64, 4096)])
            past = _log(rng, 1, 32768) if rng.random() < 0.85 else 0
            c = _attn("", _log(rng, 1, 64), q, past, hq, hkv, D, rng.choice([16, 32, 64, 128]),
                      rng.choice([0.0, 0.0, 50.0]), rng.choice([0, 0, 0, 500, 4096]))
            # no larger than the largest listed, and the plain form's scores fit
            if (c["seqs"] * hq * q * (q + past) <= 4 * 32 * 4096 * 4096
                    and c["seqs"] * hkv * D * (q + past) <= 32 * 8 * 128 * 16384
                    and work(c)["flops"] <= work(largest)["flops"]):
                return c
    while True:
        rows, R = _log(rng, 1, 1500), rng.choice([8, 16, 32, 64, _log(rng, 1, 64)])
        K, N = (rng.choice([2048, 3584, 4096, 8192, 11008, _log(rng, 200, 8192)])
                for _ in range(2))
        run = rng.choice([1, 1, _log(rng, 2, 300)])
        if rows * R * max(K, N) <= 1500 * 64 * 11008 and R * (K + N) <= 64 * (4096 + 11008):
            return _lora("", rows, run, _log(rng, 1, 48), R, K, N, rng.random() < 0.5)


# ---------------------------------------------------------------- lengths ---
def _lengths(c):
    """New tokens and cached tokens after them, of every sequence: the first
    has the case's full lengths, the others 25 % to 100 % of them."""
    qs, kvs = [], []
    for i in range(c["seqs"]):
        q = max(1, round(c["q"] * (1 - 0.75 * math.fmod(0.381966 * i, 1.0))))
        past = round(c["past"] * (1 - 0.75 * math.fmod(0.618034 * i, 1.0)))
        qs.append(q)
        kvs.append(past + q)
    return qs, kvs


def _tokens(c):
    return sum(_lengths(c)[0])


def _adapter_of(c):
    """Adapter of every row: runs of equal rows, one run in nine without one."""
    return [(-1 if (t // c["run"]) % 9 == 8 else (t // c["run"]) % c["adapters"])
            for t in range(c["rows"])]


def _ranks(c):
    return [max(1, c["R"] >> (i % 3)) if c["mixed"] else c["R"] for i in range(c["adapters"])]


# ---------------------------------------------------------------- prepare ---
def _randn(g, *shape, scale=1.0):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).mul_(scale).to(H)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _paged(c, g, poison):
    """Cache, sequence lengths and page table; pages in random order.  Slots
    of the pool that hold no token keep whatever was there (poison: NaN)."""
    qs, kvs = _lengths(c)
    page, hkv, D = c["page"], c["hkv"], c["D"]
    need = [-(-n // page) for n in kvs]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    width = max(need)
    first = _i32([sum(need[:i]) for i in range(len(need))])
    col = torch.arange(width, dtype=torch.int32, device=DEV)[None, :]
    used = col < _i32(need)[:, None]
    at = torch.where(used, first[:, None] + col, 0).long()
    table = torch.where(used, order[at], 0).contiguous()
    k = _randn(g, n_pages, hkv, page, D)
    v = _randn(g, n_pages, hkv, page, D)
    if poison:  # the tail of every sequence's last page, and the free pages
        last = torch.gather(table, 1, (_i32(need) - 1)[:, None].long())[:, 0].long()
        slot = torch.arange(page, device=DEV)[None, :]
        dead = torch.zeros((n_pages, page), dtype=torch.bool, device=DEV)
        dead[last] = slot >= (_i32(kvs) - (_i32(need) - 1) * page)[:, None]
        dead[order[sum(need):].long()] = True
        k.masked_fill_(dead[:, None, :, None], float("nan"))
        v.masked_fill_(dead[:, None, :, None], float("nan"))
    cu = [0]
    for q in qs:
        cu.append(cu[-1] + q)
    return {"k": k, "v": v, "table": table, "cu_q": _i32(cu), "kv_len": _i32(kvs)}


def _make(case, seed):
    c, g = case, torch.Generator(device=DEV)
    g.manual_seed(seed)
    if c["op"] == "rmsnorm":
        gain = 1.0 + 30.0 * (torch.rand((c["K"],), generator=g, device=DEV) < 0.01)  # outlier channels
        s = {"x": (_randn(g, c["rows"], c["K"]) * gain).to(H),
             "w": _randn(g, c["K"], scale=0.1) + (1.0 - c["bias"])}
        if c["residual"]:
            s["r"] = (_randn(g, c["rows"], c["K"], scale=2.0) * gain).to(H)
        return s
    if c["op"] == "append":
        s, T = _paged(c, g, False), _tokens(c)
        qkv = _randn(g, T, c["hq"] + 2 * c["hkv"], c["D"])  # one projection's output, sliced
        s["q"], s["kn"], s["vn"] = qkv.split([c["hq"], c["hkv"], c["hkv"]], dim=1)
        pos = torch.arange(max(_lengths(c)[1]), device=DEV, dtype=torch.float32)
        freq = 10000.0 ** (-torch.arange(c["D"] // 2, device=DEV, dtype=torch.float32)
                           / (c["D"] // 2))
        a = pos[:, None] * freq[None, :]
        s["rope"] = torch.cat([a.cos(), a.sin()], dim=1).contiguous()
        return s
    if c["op"] == "attention":
        s = _paged(c, g, True)
        s["q"] = _randn(g, _tokens(c), c["hq"], c["D"], scale=1.5)
        return s
    n, R = c["adapters"], c["R"]
    return {"x": _randn(g, c["rows"], c["K"]), "y": _randn(g, c["rows"], c["N"]),
            "a": _randn(g, n, R, c["K"], scale=c["K"] ** -0.5), "b": _randn(g, n, c["N"], R, scale=0.5),
            "scale": torch.rand((n,), generator=g, device=DEV) + 0.5,
            "rank": _i32(_ranks(c)) if c["mixed"] else None, "index": _i32(_adapter_of(c))}


def prepare(case, seed):
    s = _make(case, seed)
    s["case"] = dict(case)
    if own:  # the handles and workspaces that a serving program keeps
        import weight_only_quantized_dequant_gb300 as qz
        s["qz"] = qz
        if case["op"] in ("append", "attention"):
            s["cache"] = qz.PagedKV(s["k"], s["v"])
            s["seqs"] = qz.SeqBatch(s["cu_q"], s["kv_len"], s["table"])
        if case["op"] == "attention":
            s["workspace"] = qz.attention_workspace(s["q"].shape[0], case["seqs"], case["hq"],
                                                    case["hkv"], case["D"], device=DEV)
        if case["op"] == "lora":
            s["adapters"] = qz.LoraAdapters(s["a"], s["b"], s["scale"], s["rank"])
            s["workspace"] = qz.lora_workspace(case["rows"], case["K"], case["R"], device=DEV)
    return s


# -------------------------------------------------------------------- run ---
EPS = 1e-5


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    c, qz = s["case"], s["qz"]
    if c["op"] == "rmsnorm":
        if c["int8"]:
            q, scale, h = qz.rmsnorm_int8(s["x"], s["w"], EPS, residual=s.get("r"),
                                          w_bias=c["bias"])
            y = torch.mul(q, scale[:, None], out=torch.empty_like(s["x"]))
        else:
            y, h = qz.rmsnorm(s["x"], s["w"], EPS, residual=s.get("r"), w_bias=c["bias"])
        return (y, h) if c["residual"] else (y,)
    if c["op"] == "append":
        q = qz.rope_append(s["q"], s["kn"], s["vn"], s["cache"], s["seqs"], s["rope"])
        return q, s["k"], s["v"]
    if c["op"] == "attention":
        return (qz.attention_paged(s["q"], s["cache"], s["seqs"], softcap=c["softcap"],
                                   window=c["window"], workspace=s["workspace"]),)
    return (qz.lora(s["x"], s["y"], s["adapters"], s["index"], workspace=s["workspace"]),)


def _run_plain(s):
    return {"rmsnorm": _plain_norm, "append": _plain_append, "attention": _plain_attention,
            "lora": _plain_lora}[s["case"]["op"]](s)


def _plain_norm(s):
    c = s["case"]
    h = s["x"].float()
    if c["residual"]:
        h = h + s["r"].float()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * (c["bias"] + s["w"].float())
    if c["int8"]:
        scale = y.abs().amax(1, keepdim=True) / 127.0
        y = torch.round(y / torch.where(scale > 0, scale, 1.0)) * scale
    return (y.to(H), h.to(H)) if c["residual"] else (y.to(H),)


def _places(s):
    """Sequence and position of every new token."""
    T = s["q"].shape[0]
    t = torch.arange(T, dtype=torch.int32, device=DEV)
    seq = torch.searchsorted(s["cu_q"][1:].contiguous(), t, right=True)
    new = s["cu_q"][1:] - s["cu_q"][:-1]
    i = t - s["cu_q"][seq]
    return seq, i, s["kv_len"][seq] - new[seq] + i


def _plain_append(s):
    c = s["case"]
    seq, _, pos = _places(s)
    half, pl = c["D"] // 2, pos.long()
    cos, sin = s["rope"][pl, None, :half], s["rope"][pl, None, half:]

    def rotate(x):
        a, b = x[..., :half].float(), x[..., half:].float()
        return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1).to(H)

    page, slot = s["table"][seq, pl // c["page"]].long(), pl % c["page"]
    s["k"][page, :, slot] = rotate(s["kn"])
    s["v"][page, :, slot] = s["vn"]
    return rotate(s["q"]), s["k"], s["v"]


def _plain_attention(s):
    c = s["case"]
    S, hq, hkv, D = c["seqs"], c["hq"], c["hkv"], c["D"]
    G, Lq, T = hq // hkv, c["q"], s["q"].shape[0]
    # keys and values of every sequence in order, [S, hkv, L, D], and the queries [S, hkv, Lq*G, D]
    k = s["k"][s["table"].long()].transpose(1, 2).reshape(S, hkv, -1, D).float()
    v = s["v"][s["table"].long()].transpose(1, 2).reshape(S, hkv, -1, D).float()
    L = k.shape[2]
    at = torch.arange(L, device=DEV)
    held = at[None, :] < s["kv_len"][:, None]
    k = torch.where(held[:, None, :, None], k, 0.0)
    v = torch.where(held[:, None, :, None], v, 0.0)
    i = torch.arange(Lq, device=DEV)
    new = s["cu_q"][1:] - s["cu_q"][:-1]
    token = (s["cu_q"][:-1, None] + i[None, :]).clamp(max=T - 1).long()
    q = s["q"].float()[token].reshape(S, Lq, hkv, G, D).transpose(1, 2).reshape(S, hkv, Lq * G, D)
    x = q @ k.transpose(2, 3)
    x = x * D ** -0.5
    if c["softcap"]:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    pos = (s["kv_len"] - new)[:, None] + i[None, :]
    seen = held[:, None, :] & (at[None, None, :] <= pos[:, :, None])
    if c["window"]:
        seen = seen & (at[None, None, :] > pos[:, :, None] - c["window"])
    x = x.reshape(S, hkv, Lq, G, L).masked_fill_(~seen[:, None, :, None, :], float("-inf"))
    m = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(m > float("-inf"), m, 0.0))
    l = x.sum(-1, keepdim=True)
    o = (x.reshape(S, hkv, Lq * G, L) @ v).reshape(S, hkv, Lq, G, D)
    o = o / torch.where(l > 0, l, 1.0)
    o = o.transpose(1, 2).reshape(S, Lq, hq, D)
    seq, j, _ = _places(s)
    return (o[seq, j.long()].to(H),)


def _plain_lora(s):
    c = s["case"]
    i = s["index"].clamp(min=0).long()
    u = (s["a"][i].float() @ s["x"].float()[:, :, None])[:, :, 0]
    if s["rank"] is not None:
        u = u * (torch.arange(c["R"], device=DEV)[None, :] < s["rank"][i][:, None])
    u = u * (s["scale"][i] * (s["index"] >= 0))[:, None]
    d = (s["b"][i].float() @ u[:, :, None])[:, :, 0]
    return ((s["y"].float() + d).to(H),)


# ------------------------------------------------------------------- work ---
def _pairs(c):
    """Visible (query, key) pairs, and keys that any query of a sequence sees."""
    pairs = keys = 0
    W = c["window"]
    for q, n in zip(*_lengths(c)):
        first = n - q
        if not W or n <= W:
            pairs += q * first + q * (q + 1) // 2
            keys += n
        else:
            pairs += sum(min(W, first + j + 1) for j in range(q))
            keys += n - max(0, first + 1 - W)
    return pairs, keys


def work(case):
    c = case
    if c["op"] == "rmsnorm":
        n = c["rows"] * c["K"]
        b = 2 * n * (3 if c["residual"] else 1) + 2 * c["K"]
        b += n + 4 * c["rows"] if c["int8"] else 2 * n
        return {"bytes": b, "flops": 6 * n}
    if c["op"] == "append":
        T = _tokens(c)
        b = T * c["D"] * 2 * 2 * (c["hq"] + 2 * c["hkv"]) + 4 * T * c["D"]
        return {"bytes": b, "flops": 3 * T * c["D"] * (c["hq"] + c["hkv"])}
    if c["op"] == "attention":
        pairs, keys = _pairs(c)
        b = 2 * 2 * _tokens(c) * c["hq"] * c["D"] + 2 * 2 * keys * c["hkv"] * c["D"]
        return {"bytes": b, "flops": 4 * pairs * c["hq"] * c["D"]}
    index, ranks = _adapter_of(c), _ranks(c)
    b = 2 * c["rows"] * (c["K"] + 2 * c["N"])
    b += sum(2 * ranks[a] * (c["K"] + c["N"]) for a in set(index) if a >= 0)
    return {"bytes": b, "flops": sum(2 * ranks[a] * (c["K"] + c["N"]) for a in index if a >= 0)}


# ------------------------------------------------------------------ exact ---
def exact(case, seed):
    """The outputs from their definitions in 64 bits."""
    c, s = case, _make(case, seed)
    D64 = torch.float64
    if c["op"] == "rmsnorm":
        h = s["x"].to(D64) + (s["r"].to(D64) if c["residual"] else 0.0)
        y = h / (h.square().sum(1) / c["K"] + EPS).sqrt()[:, None] * (s["w"].to(D64) + c["bias"])
        if c["int8"]:
            step = y.abs().max(1).values / 127.0
            step[step == 0] = 1.0
            y = (y / step[:, None]).round() * step[:, None]
        return (y, h) if c["residual"] else (y,)
    qs, kvs = _lengths(c) if c["op"] != "lora" else ([], [])
    if c["op"] == "append":
        k, v, half, t = s["k"].to(D64), s["v"].to(D64), c["D"] // 2, 0
        qo = torch.empty(s["q"].shape, dtype=D64, device=DEV)
        for i, (n, L) in enumerate(zip(qs, kvs)):
            p = torch.arange(L - n, L, device=DEV)
            z = torch.complex(s["rope"][p, :half].to(D64), s["rope"][p, half:].to(D64))[:, None]
            for src, dst in ((s["q"], qo), (s["kn"], None)):
                x = src[t:t + n].to(D64)
                w = torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous()) * z
                w = torch.cat([w.real, w.imag], dim=-1)
                if dst is not None:
                    dst[t:t + n] = w
                else:
                    k[s["table"][i, p // c["page"]].long(), :, p % c["page"]] = w
            v[s["table"][i, p // c["page"]].long(), :, p % c["page"]] = s["vn"][t:t + n].to(D64)
            t += n
        return qo, k, v
    if c["op"] == "attention":
        G, t = c["hq"] // c["hkv"], 0
        out = torch.empty(s["q"].shape, dtype=D64, device=DEV)
        for i, (n, L) in enumerate(zip(qs, kvs)):
            pages = s["table"][i, :-(-L // c["page"])].long()
            p = torch.arange(L - n, L, device=DEV)[:, None]
            j = torch.arange(L, device=DEV)[None, :]
            hidden = j > p
            if c["window"]:
                hidden |= j <= p - c["window"]
            for h in range(c["hkv"]):
                k = s["k"][pages, h].reshape(-1, c["D"])[:L].to(D64)
                v = s["v"][pages, h].reshape(-1, c["D"])[:L].to(D64)
                for g in range(h * G, h * G + G):
                    x = s["q"][t:t + n, g].to(D64) @ k.T / math.sqrt(c["D"])
                    if c["softcap"]:
                        x = torch.tanh(x / c["softcap"]) * c["softcap"]
                    out[t:t + n, g] = torch.softmax(x.masked_fill(hidden, -math.inf), 1) @ v
            t += n
        return (out,)
    y, ranks = s["y"].to(D64), _ranks(c)
    for t, a in enumerate(_adapter_of(c)):
        if a >= 0 and t % c["run"] == 0:
            rows, r = slice(t, min(t + c["run"], c["rows"])), ranks[a]
            u = s["x"][rows].to(D64) @ s["a"][a, :r].to(D64).T
            y[rows] += s["scale"][a].to(D64) * (u @ s["b"][a, :, :r].to(D64).T)
    return (y,)
