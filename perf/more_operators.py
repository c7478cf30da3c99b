"""Cases of the operators around an INT8 key/value cache, and of the choice of
the next tokens.

A served step whose cache is held in INT8 rows (a code a value, a scale a row)
quantises the new keys and values as it writes them (``rope_append`` with a
``PagedKVInt8``), attends over the codes (``attention_paged``), reads rows back
in fp16 where a sequence is moved or inspected (``cache_read``), and ends with
the choice of every request's next token from its logits and one uniform random
number (``sample``).  Each case is one call, but for those of ``rope_append``,
which read the sequences back: codes and scales are compared as the values that
they stand for.

``own`` selects what ``run`` computes: False, the operators in elementary
torch operations; True, the framework's kernels.
"""
import math

import torch

own = False

DEV = "cuda"
H, F32, F64 = torch.float16, torch.float32, torch.float64
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases ---
def _append(name, seqs, q, past, hq, hkv, D, page):
    return {"name": name, "op": "append", "seqs": seqs, "q": q, "past": past, "hq": hq,
            "hkv": hkv, "D": D, "page": page}


def _read(name, seqs, held, hkv, D, page):
    return {"name": name, "op": "read", "seqs": seqs, "q": held, "past": 0, "hkv": hkv, "D": D,
            "page": page}


def _attn(name, seqs, q, past, hq, hkv, D, page, softcap=0.0, window=0):
    return {"name": name, "op": "attention", "seqs": seqs, "q": q, "past": past, "hq": hq,
            "hkv": hkv, "D": D, "page": page, "softcap": softcap, "window": window}


def _sample(name, rows, vocab, dtype="fp16", temperature=1.0, top_k=0, top_p=1.0, min_p=0.0,
            mixed=False):
    return {"name": name, "op": "sample", "rows": rows, "vocab": vocab, "dtype": dtype,
            "temperature": temperature, "top_k": top_k, "top_p": top_p, "min_p": min_p,
            "mixed": mixed}


def listed():
    return [
        # one decode step of 64 requests on the 7B-shaped stack, contexts just begun
        _append("append8_64x1_h32", 64, 1, 20, 32, 32, 128, 16),
        # packed chunks of different lengths on the 70B-shaped stack
        _append("append8_9x300_h64kv8", 9, 300, 300, 64, 8, 128, 64),
        # a short sequence read back, to be looked at or moved
        _read("read8_1x199_kv8", 1, 199, 8, 128, 16),
        # eight sequences of up to 16k tokens handed to a cache elsewhere
        _read("read8_8x16k_kv8", 8, 16384, 8, 128, 64),
        # the smallest serving step: one request, one token, a short context
        _attn("attn8_1x1_ctx200_h32kv8", 1, 1, 199, 32, 8, 128, 16),
        # a decode step of 32 requests with contexts up to 16k on the 70B-shaped stack
        _attn("attn8_32x1_ctx16k_h64kv8", 32, 1, 16383, 64, 8, 128, 64),
        # Gemma-2-9B-shaped local layer: head size 256, capped logits, a window of 4096
        _attn("attn8_8x1_ctx8k_d256_cap_win", 8, 1, 8000, 16, 8, 256, 32, softcap=50.0,
              window=4096),
        # chunks of new tokens beside long contexts (chunked prompts, verified drafts)
        _attn("attn8_4x64_ctx24k_h64kv8", 4, 64, 24000, 64, 8, 128, 64),
        # whole prompts of different lengths, packed, on the 7B-shaped stack
        _attn("attn8_4x2048_prompt_h32", 4, 2048, 0, 32, 32, 128, 64),
        # one request's next token, the usual filters
        _sample("sample_1x32000_kp", 1, 32000, temperature=0.8, top_k=50, top_p=0.9),
        # requests of many users, each with filters of its own; greedy and masked rows
        _sample("sample_16x128000_mixed", 16, 128000, "fp32", 1.0, 40, 0.9, 0.05, mixed=True),
        # 64 requests over Gemma-2-9B's vocabulary, the nucleus alone
        _sample("sample_64x256000_p", 64, 256000, top_p=0.95),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


# (heads, KV heads, head size): the stacks' own, and groups that are odd or cover every head
_HEADS = [(32, 32, 128), (64, 8, 128), (16, 8, 256), (32, 8, 128), (32, 8, 64), (12, 4, 128),
          (5, 1, 64), (16, 16, 64), (8, 1, 256), (28, 4, 128)]
_PAGES = [16, 32, 64, 128]


def draw(rng):
    op = rng.choice(["append", "read", "attention", "attention", "sample", "sample"])
    hq, hkv, D = rng.choice(_HEADS)
    if op == "append":
        return _append("", _log(rng, 1, 64), _log(rng, 1, 300), _log(rng, 1, 300), hq, hkv, D,
                       rng.choice(_PAGES))
    if op == "read":
        while True:
            c = _read("", _log(rng, 1, 64), _log(rng, 1, 16384), hkv, D, rng.choice(_PAGES))
            if c["seqs"] * c["q"] * hkv * D <= 8 * 16384 * 8 * 128:
                return c
    if op == "sample":
        while True:
            c = _sample("", _log(rng, 1, 256), _log(rng, 1, 262144), rng.choice(list(TYPES)),
                        rng.choice([1.0, 0.7, 1.5, round(rng.uniform(0.2, 3.0), 3)]),
                        rng.choice([0, 0, 1, 50, _log(rng, 2, 2000)]),
                        rng.choice([1.0, 0.9, 0.95, round(rng.uniform(0.05, 1.0), 3)]),
                        rng.choice([0.0, 0.0, 0.05, round(rng.uniform(0.0, 0.5), 3)]),
                        rng.random() < 0.3)
            if c["rows"] * c["vocab"] <= 64 * 256000:
                return c
    largest = {c["name"]: c for c in listed()}["attn8_4x64_ctx24k_h64kv8"]
    while True:
        hq, hkv, D = rng.choice(_HEADS)
        q = rng.choice([1, 1, _log(rng, 2, 64), _log(rng, 64, 2048)])
        past = _log(rng, 1, 32768) if rng.random() < 0.85 else 0
        c = _attn("", _log(rng, 1, 64), q, past, hq, hkv, D, rng.choice(_PAGES),
                  rng.choice([0.0, 0.0, 50.0]), rng.choice([0, 0, 0, 500, 4096]))
        # no larger than the largest listed, and the plain form's scores fit
        if (c["seqs"] * hq * q * (q + past) <= 4 * 64 * 64 * 24064
                and c["seqs"] * hkv * D * (q + past) <= 32 * 8 * 128 * 16384
                and work(c)["flops"] <= work(largest)["flops"]):
            return c


# ---------------------------------------------------------------- lengths ---
def _lengths(c):
    """New tokens, and tokens held with them, of every sequence: the first has
    the case's full lengths, the others 25 % to 100 % of them."""
    qs = [max(1, round(c["q"] * (1 - 0.75 * math.fmod(0.381966 * i, 1.0))))
          for i in range(c["seqs"])]
    past = [round(c["past"] * (1 - 0.75 * math.fmod(0.618034 * i, 1.0))) for i in range(c["seqs"])]
    return qs, [p + q for p, q in zip(past, qs)]


def _tokens(c):
    return sum(_lengths(c)[0])


def _sums(v):
    return [sum(v[:i]) for i in range(len(v) + 1)]


# ---------------------------------------------------------------- prepare ---
def _randn(g, *shape, scale=1.0):
    return torch.randn(shape, generator=g, device=DEV, dtype=F32).mul_(scale).to(H)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _pool(g, *shape):
    """Codes [pages, heads, slots, D] and scales [pages, heads, slots] of random
    rows, whose sizes differ by token as those of real keys and values do."""
    x = torch.randn(shape, generator=g, device=DEV, dtype=F32)
    x *= torch.exp(0.4 * torch.randn(shape[:3], generator=g, device=DEV))[..., None]
    scale = x.abs().amax(-1) / 127.0
    return torch.round(x / scale[..., None]).to(torch.int8), scale


def _paged(c, g):
    """Cache, sequence lengths and page table; pages in random order.  Slots of
    the pool that hold no token keep any codes, with scales that are NaN."""
    qs, kvs = _lengths(c)
    page, hkv, D = c["page"], c["hkv"], c["D"]
    need = [-(-n // page) for n in kvs]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    first, width = _sums(need), max(need)
    col = torch.arange(width, dtype=torch.int32, device=DEV)[None, :]
    at = torch.where(col < _i32(need)[:, None], _i32(first[:-1])[:, None] + col, 0).long()
    table = torch.where(col < _i32(need)[:, None], order[at], 0).contiguous()
    s = {"table": table, "cu_q": _i32(_sums(qs)), "kv_len": _i32(kvs), "cu_held": _i32(_sums(kvs))}
    s["n_held"] = sum(kvs)
    s["k"], s["ks"] = _pool(g, n_pages, hkv, page, D)
    s["v"], s["vs"] = _pool(g, n_pages, hkv, page, D)
    dead = torch.zeros((n_pages, page), dtype=torch.bool, device=DEV)
    last = torch.gather(table, 1, (_i32(need) - 1)[:, None].long())[:, 0].long()
    slot = torch.arange(page, device=DEV)[None, :]
    dead[last] = slot >= (_i32(kvs) - (_i32(need) - 1) * page)[:, None]
    dead[order[first[-1]:].long()] = True
    s["ks"].masked_fill_(dead[:, None, :], float("nan"))
    s["vs"].masked_fill_(dead[:, None, :], float("nan"))
    return s


def _logits(c, g):
    """Rows of logits: a wide body, a few likely tokens (more in some rows than in
    others), and one token in 50 banned (-inf)."""
    B, V = c["rows"], c["vocab"]
    x = torch.randn((B, V), generator=g, device=DEV, dtype=F32) * 2.5
    n = min(V, 40)
    at = torch.randint(0, V, (B, n), generator=g, device=DEV)
    lift = torch.randn((B, n), generator=g, device=DEV) * 3.0 + 8.0
    lift *= (torch.arange(B, device=DEV) % 3 != 2)[:, None]  # one row in three is flat
    x.scatter_add_(1, at, lift)
    banned = torch.rand((B, V), generator=g, device=DEV) < 0.02
    banned[:, V // 2] = False
    return x.masked_fill_(banned, float("-inf")).to(TYPES[c["dtype"]])


def _make(case, seed):
    c, g = case, torch.Generator(device=DEV)
    g.manual_seed(seed)
    if c["op"] == "sample":
        B, i = c["rows"], torch.arange(c["rows"], device=DEV)
        s = {"logits": _logits(c, g), "u": torch.rand((B,), generator=g, device=DEV)}
        s["temperature"], s["top_k"] = c["temperature"], c["top_k"]
        s["top_p"], s["min_p"] = c["top_p"], c["min_p"]
        if c["mixed"]:  # every fifth row greedy; filters of each row on or off; a masked row
            warm = c["temperature"] * (1.0 + 0.1 * (i % 4))
            s["temperature"] = torch.where(i % 5 == 3, 0.0, warm)
            s["top_k"] = torch.where(i % 3 == 1, 0, c["top_k"] + i).to(torch.int32)
            s["top_p"] = torch.where(i % 4 == 2, 1.0, c["top_p"] - 0.02 * (i % 3)).clamp(min=0.01)
            s["min_p"] = torch.where(i % 2 == 0, 0.0, c["min_p"])
            s["temperature"], s["top_p"], s["min_p"] = (
                s[n].to(F32) for n in ("temperature", "top_p", "min_p"))
            s["logits"][i % 8 == 7] = float("-inf")
        return s
    s, T = _paged(c, g), _tokens(c)
    if c["op"] == "append":
        qkv = _randn(g, T, c["hq"] + 2 * c["hkv"], c["D"])  # one projection's output, sliced
        s["q"], s["kn"], s["vn"] = qkv.split([c["hq"], c["hkv"], c["hkv"]], dim=1)
        pos = torch.arange(max(_lengths(c)[1]), device=DEV, dtype=F64)
        a = pos[:, None] * 10000.0 ** (-torch.arange(c["D"] // 2, device=DEV, dtype=F64)
                                       / (c["D"] // 2))[None, :]
        s["rope"] = torch.cat([a.cos(), a.sin()], dim=1).to(F32)
    if c["op"] == "attention":
        s["q"] = _randn(g, T, c["hq"], c["D"], scale=1.5)
    return s


def prepare(case, seed):
    s = _make(case, seed)
    s["case"] = dict(case)
    if own:  # the handles and workspaces that a serving program keeps
        import weight_only_quantized_dequant_gb300 as qz
        s["qz"] = qz
        if case["op"] != "sample":
            s["cache"] = qz.PagedKVInt8(s["k"], s["v"], s["ks"], s["vs"])
            s["seqs"] = qz.SeqBatch(s["cu_q"], s["kv_len"], s["table"])
            s["held"] = qz.SeqBatch(s["cu_held"], s["kv_len"], s["table"])
        if case["op"] == "attention":
            s["workspace"] = qz.attention_workspace(s["q"].shape[0], case["seqs"], case["hq"],
                                                    case["hkv"], case["D"], device=DEV)
    return s


# -------------------------------------------------------------------- run ---
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    c, qz = s["case"], s["qz"]
    if c["op"] == "append":
        q = qz.rope_append(s["q"], s["kn"], s["vn"], s["cache"], s["seqs"], s["rope"])
        return (q, *qz.cache_read(s["cache"], s["held"], s["n_held"]))
    if c["op"] == "read":
        return qz.cache_read(s["cache"], s["held"], s["n_held"])
    if c["op"] == "attention":
        return (qz.attention_paged(s["q"], s["cache"], s["seqs"], softcap=c["softcap"],
                                   window=c["window"], workspace=s["workspace"]),)
    return qz.sample(s["logits"], s["u"], s["temperature"], s["top_k"], s["top_p"], s["min_p"])


def _run_plain(s):
    return {"append": _plain_append, "read": _plain_read, "attention": _plain_attention,
            "sample": _plain_sample}[s["case"]["op"]](s)


def _places(cu, kv_len, T):
    """Sequence, place among its new tokens, and position of every one of T packed rows."""
    t = torch.arange(T, dtype=torch.int32, device=DEV)
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    i = t - cu[seq]
    return seq, i, kv_len[seq] - (cu[seq + 1] - cu[seq]) + i


def _plain_read(s):
    c = s["case"]
    seq, _, pos = _places(s["cu_held"], s["kv_len"], s["n_held"])
    pos = pos.long()
    page, slot = s["table"][seq, pos // c["page"]].long(), pos % c["page"]
    return tuple((s[x][page, :, slot].float() * s[n][page, :, slot][..., None]).to(H)
                 for x, n in (("k", "ks"), ("v", "vs")))


def _plain_append(s):
    c = s["case"]
    seq, _, pos = _places(s["cu_q"], s["kv_len"], s["q"].shape[0])
    half, pos = c["D"] // 2, pos.long()
    cos, sin = (s["rope"][pos, None, i * half:(i + 1) * half].double() for i in (0, 1))

    def rotate(x):
        a, b = x[..., :half].double(), x[..., half:].double()
        return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)

    page, slot = s["table"][seq, pos // c["page"]].long(), pos % c["page"]
    # codes next to a border: rotated in 64 bits, divided in the 32 bits that the scale has
    kn, vn = rotate(s["kn"]).float(), s["vn"].float()
    ks, vs = kn.abs().amax(-1) / 127.0, vn.abs().amax(-1) / 127.0
    s["k"][page, :, slot] = torch.round(kn / ks[..., None]).to(torch.int8)
    s["v"][page, :, slot] = torch.round(vn / vs[..., None]).to(torch.int8)
    s["ks"][page, :, slot], s["vs"][page, :, slot] = ks, vs
    return (rotate(s["q"]).to(H), *_plain_read(s))


def _plain_attention(s):
    c = s["case"]
    S, hq, hkv, D = c["seqs"], c["hq"], c["hkv"], c["D"]
    G, Lq, T = hq // hkv, c["q"], s["q"].shape[0]
    # keys and values of every sequence in order, [S, hkv, L, D], and the queries [S, hkv, Lq*G, D]
    table = s["table"].long()
    ks = s["ks"][table].transpose(1, 2).reshape(S, hkv, -1, 1)
    vs = s["vs"][table].transpose(1, 2).reshape(S, hkv, -1, 1)
    L = ks.shape[2]
    at = torch.arange(L, device=DEV)
    held = at[None, :] < s["kv_len"][:, None]
    k = s["k"][table].transpose(1, 2).reshape(S, hkv, L, D) * torch.where(
        held[:, None, :, None], ks, 0.0)
    v = s["v"][table].transpose(1, 2).reshape(S, hkv, L, D) * torch.where(
        held[:, None, :, None], vs, 0.0)
    i = torch.arange(Lq, device=DEV)
    new = s["cu_q"][1:] - s["cu_q"][:-1]
    token = (s["cu_q"][:-1, None] + i[None, :]).clamp(max=T - 1).long()
    q = s["q"].float()[token].reshape(S, Lq, hkv, G, D).transpose(1, 2).reshape(S, hkv, Lq * G, D)
    x = (q @ k.transpose(2, 3)) * D ** -0.5
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
    seq, j, _ = _places(s["cu_q"], s["kv_len"], s["q"].shape[0])
    return (o[seq, j.long()].to(H),)


def _column(v, B):
    """An option of every row, [B, 1] in 64 bits (of its 32-bit value)."""
    return torch.as_tensor(v, dtype=F32, device=DEV).double().expand(B)[:, None]


def _plain_sample(s):
    x = s["logits"].double()  # sums over a vocabulary, and borders between its tokens
    B, V = x.shape
    T, k, p, min_p = (_column(s[n], B) for n in ("temperature", "top_k", "top_p", "min_p"))
    greedy = T <= 0
    m = x.amax(1, keepdim=True)
    w = torch.where(x == m, 1.0, torch.exp((x - m) / torch.where(greedy, 1.0, T)))
    _, order = torch.sort(x, dim=1, descending=True, stable=True)
    rank = torch.arange(V, device=DEV)[None, :]
    ws = torch.gather(w, 1, order)
    keep = (rank < k) | (k <= 0)
    mass = torch.cumsum(ws * keep, 1)
    before = torch.cat([torch.zeros_like(m), mass[:, :-1]], 1)
    keep &= (p >= 1) | (rank == 0) | (before < p * mass[:, -1:])
    keep &= (min_p <= 0) | (ws >= min_p)
    keep = torch.where(greedy, rank == 0, keep)
    kept = torch.zeros_like(keep).scatter_(1, order, keep)
    sums = torch.cumsum(w * kept, 1)
    total = sums[:, -1:]
    token = (sums <= s["u"].double()[:, None] * total).sum(1, keepdim=True)
    logprob = torch.log(torch.gather(w, 1, token.clamp(max=V - 1)) / total)
    none = m == float("-inf")
    return (torch.where(none, -1, token)[:, 0].to(torch.int32),
            torch.where(none, float("-inf"), logprob)[:, 0].to(F32))


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
    if c["op"] == "sample":
        n = c["rows"] * c["vocab"]
        return {"bytes": n * (4 if c["dtype"] == "fp32" else 2) + 12 * c["rows"], "flops": 3 * n}
    row = c["hkv"] * (c["D"] + 4)  # a token's keys or values in the cache
    if c["op"] == "append":
        T, held = _tokens(c), sum(_lengths(c)[1])
        b = 2 * T * c["D"] * (2 * c["hq"] + 2 * c["hkv"]) + 4 * T * c["D"] + 2 * T * row
        b += 2 * held * (row + 2 * c["hkv"] * c["D"])  # read back
        return {"bytes": b, "flops": 5 * T * c["D"] * (c["hq"] + 2 * c["hkv"])}
    if c["op"] == "read":
        T = _tokens(c)
        return {"bytes": 2 * T * (row + 2 * c["hkv"] * c["D"]), "flops": 2 * T * c["hkv"] * c["D"]}
    pairs, keys = _pairs(c)
    return {"bytes": 2 * 2 * _tokens(c) * c["hq"] * c["D"] + 2 * keys * row,
            "flops": 4 * pairs * c["hq"] * c["D"]}


# ------------------------------------------------------------------ exact ---
def _held(s, c, i, L, codes, scales):
    """The first L rows of sequence i, [L, heads, D] in 64 bits."""
    pages = s["table"][i, :-(-L // c["page"])].long()
    x = s[codes][pages].double() * s[scales][pages].double()[..., None]
    return x.permute(0, 2, 1, 3).reshape(-1, c["hkv"], c["D"])[:L]


def _exact_sample(s, c):
    tokens, logs = [], []
    rows = {n: torch.as_tensor(s[n]).to(F32 if n != "top_k" else torch.int32).expand(c["rows"])
            .tolist() for n in ("temperature", "top_k", "top_p", "min_p", "u")}
    for r in range(c["rows"]):
        T, k, p, min_p, u = (rows[n][r] for n in ("temperature", "top_k", "top_p", "min_p", "u"))
        x = s["logits"][r].double()
        # the values that occur, largest first, with how many tokens have each
        value, which, count = torch.unique(-x, return_inverse=True, return_counts=True)
        value = -value
        if value[0] == -math.inf:
            tokens.append(-1)
            logs.append(-math.inf)
            continue
        if T <= 0:
            tokens.append(int((x == value[0]).nonzero()[0, 0]))
            logs.append(0.0)
            continue
        w = torch.exp((value - value[0]) / T)
        if k > 0:
            count = (k - (torch.cumsum(count, 0) - count)).clamp(min=0).minimum(count)
        if p < 1:
            mass = torch.cumsum(w * count, 0)
            left = p * mass[-1] - (mass - w * count)  # what is missing where a value begins
            need = torch.ceil(left / w).clamp(min=0).nan_to_num(0)
            need[0] = need[0].clamp(min=1)
            count = torch.minimum(count.double(), need).long()
        if min_p > 0:
            count = torch.where(w >= min_p, count, 0)
        kept = torch.zeros_like(x)
        cut = (count > 0).nonzero()[-1, 0]  # the last value kept, perhaps for some of its tokens
        kept[which < cut] = 1.0
        kept[(which == cut).nonzero()[:, 0][:int(count[cut])]] = 1.0
        sums = torch.cumsum(kept * w[which], 0)
        t = int((sums > u * sums[-1]).nonzero()[0, 0])
        tokens.append(t)
        logs.append(float(torch.log(w[which[t]]) - torch.log(sums[-1])))
    return (torch.tensor(tokens, dtype=torch.int32, device=DEV),
            torch.tensor(logs, dtype=F64, device=DEV))


def exact(case, seed):
    """The outputs from their definitions in 64 bits."""
    c, s = case, _make(case, seed)
    if c["op"] == "sample":
        return _exact_sample(s, c)
    qs, kvs = _lengths(c)
    if c["op"] == "read":
        return tuple(torch.cat([_held(s, c, i, L, x, n) for i, L in enumerate(kvs)])
                     for x, n in (("k", "ks"), ("v", "vs")))
    if c["op"] == "append":
        half, t = c["D"] // 2, 0
        qo, ko, vo = torch.empty(s["q"].shape, dtype=F64, device=DEV), [], []

        def turned(x, p):
            z = torch.complex(s["rope"][p, :half].double(), s["rope"][p, half:].double())[:, None]
            w = torch.complex(x[..., :half].double(), x[..., half:].double()) * z
            return torch.cat([w.real, w.imag], dim=-1)

        def held(rows):  # what an INT8 row stands for; rows and scales have 32 bits
            rows = rows.to(F32).double()
            step = (rows.abs().max(-1, keepdim=True).values / 127.0).to(F32).double()
            return (rows / step).to(F32).round().double() * step

        for i, (n, L) in enumerate(zip(qs, kvs)):
            p = torch.arange(L - n, L, device=DEV)
            qo[t:t + n] = turned(s["q"][t:t + n], p)
            ko.append(_held(s, c, i, L, "k", "ks"))
            vo.append(_held(s, c, i, L, "v", "vs"))
            ko[-1][L - n:] = held(turned(s["kn"][t:t + n], p))
            vo[-1][L - n:] = held(s["vn"][t:t + n])
            t += n
        return qo, torch.cat(ko), torch.cat(vo)
    G, t = c["hq"] // c["hkv"], 0
    out = torch.empty(s["q"].shape, dtype=F64, device=DEV)
    for i, (n, L) in enumerate(zip(qs, kvs)):
        p = torch.arange(L - n, L, device=DEV)[:, None]
        j = torch.arange(L, device=DEV)[None, :]
        hidden = j > p
        if c["window"]:
            hidden |= j <= p - c["window"]
        keys, values = _held(s, c, i, L, "k", "ks"), _held(s, c, i, L, "v", "vs")
        for g in range(c["hq"]):
            x = s["q"][t:t + n, g].double() @ keys[:, g // G].T / math.sqrt(c["D"])
            if c["softcap"]:
                x = torch.tanh(x / c["softcap"]) * c["softcap"]
            out[t:t + n, g] = torch.softmax(x.masked_fill(hidden, -math.inf), 1) @ values[:, g // G]
        t += n
    return (out,)
