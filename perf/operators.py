"""Timed cases of the 4-bit key/value cache: writing and reading it, and attention over it.

Two operators.

"store" quantises new keys and values into a paged cache and reads them back.
Each row of d values (one token, one head, K or V) is cut into groups of 32.
A group stores

    lo = min x,   s = round16((max x - lo) / 15),   u = min(15, round((x - lo) / s))

with lo and s in the cache's 16-bit type and u in 4 bits (u = 0 where s = 0);
it stands for lo + s u. Rounding is to nearest, ties to even.

"attend" is O = softmax(scale Q K^T) V and its row log-sum-exp over what such a
cache stands for: sequence b holds lengths[b] tokens, found through its row of
the page table; query head h reads key/value head h // (Hq / Hk); with
"causal" the Nq queries of a sequence are its last Nq tokens.
"""
import math

import torch

own = False

GROUP = 32
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# --------------------------------------------------------------------------- cases

def _store(name, B, Hk, n, d, page, dtype, before):
    return {"name": name, "op": "store", "B": B, "Hk": Hk, "n": n, "d": d, "page": page,
            "dtype": dtype, "before": before}


def _attend(name, B, Hq, Hk, nq, lo, hi, d, page, dtype, causal=True):
    return {"name": name, "op": "attend", "B": B, "Hq": Hq, "Hk": Hk, "nq": nq, "min_len": lo,
            "max_len": hi, "d": d, "page": page, "dtype": dtype, "causal": causal}


def listed():
    return [
        # one decoding step of eight GPT-2-small-shaped sequences: latency counts
        _store("store_decode_b8", 8, 12, 1, 64, 64, "bf16", 1023),
        # the prompt of a GPT-2-medium-shaped batch
        _store("store_prompt_4k", 4, 16, 4096, 128, 64, "bf16", 0),
        # a chunk of a prompt at an odd position, odd head count, d = 96, small pages
        _store("store_chunk_d96", 7, 5, 1537, 96, 16, "fp16", 333),
        # a long document, wide heads
        _store("store_long_d256", 1, 16, 65536, 256, 128, "bf16", 0),
        # one token after a short prompt: the smallest call
        _attend("attend_short_b1", 1, 12, 12, 1, 257, 257, 64, 64, "bf16"),
        # a decoding step of a GPT-2-small-shaped batch, every head with its own cache
        _attend("attend_gpt2_b8", 8, 12, 12, 1, 700, 1024, 64, 64, "bf16"),
        # an ordinary serving batch: ragged lengths, four query heads share a K/V head
        _attend("attend_batch_b32", 32, 32, 8, 1, 1000, 16384, 128, 64, "bf16"),
        # one user with a long context
        _attend("attend_long_b1", 1, 16, 16, 1, 65536, 65536, 128, 64, "bf16"),
        # checking five drafted tokens, eight query heads to a K/V head, small pages
        _attend("attend_draft_nq5", 16, 16, 2, 5, 5000, 8192, 128, 16, "fp16"),
        # wide heads, all query heads on one K/V head
        _attend("attend_mqa_d256", 4, 8, 1, 1, 20000, 32768, 256, 128, "bf16"),
        # odd everything: three queries, groups of three heads, d = 96, from short to long
        _attend("attend_odd_d96", 5, 15, 5, 3, 3, 9001, 96, 32, "fp16"),
        # a chunk of a long prompt against what is cached already
        _attend("attend_chunk_1k", 2, 16, 4, 1024, 9000, 16384, 128, 64, "bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    cases = listed()
    d = rng.choice([64, 96, 128, 256])
    page = rng.choice([16, 32, 48, 64, 128, 256])
    dtype = rng.choice(["bf16", "fp16"])
    top = {op: [max(work(c)[k] for c in cases if c["op"] == op) for k in ("bytes", "flops")]
           for op in ("store", "attend")}
    while True:
        if rng.random() < 0.35:
            c = _store("", _log(rng, 1, 32), _log(rng, 1, 16), _log(rng, 1, 65536), d, page,
                       dtype, rng.choice([0, rng.randrange(1, 5000)]))
        else:
            Hk = _log(rng, 1, 16)
            hi = _log(rng, 1, 65536)
            nq = rng.choice([1, 1, 1, _log(rng, 2, 16), _log(rng, 2, 1024)])
            hi = max(hi, nq)
            lo = max(nq, _log(rng, max(1, hi // 20), hi))
            c = _attend("", _log(rng, 1, 48), Hk * rng.choice([1, 1, 2, 3, 4, 5, 8, 12, 16]), Hk,
                        nq, lo, hi, d, page, dtype, rng.random() < 0.75)
        w = work(c)
        if w["bytes"] <= top[c["op"]][0] and w["flops"] <= top[c["op"]][1]:
            del c["name"]
            return c


def _lengths(case):
    """Tokens of each sequence: spread evenly from the shortest to the longest, in an order
    that puts neighbours far apart."""
    B, lo, hi = case["B"], case["min_len"], case["max_len"]
    step = next(s for s in (7, 5, 3, 1) if math.gcd(s, B) == 1)
    return [hi - (hi - lo) * ((i * step) % B) // max(B - 1, 1) for i in range(B)]


def work(case):
    d = case["d"]
    packed = d // 2 + d // GROUP * 4  # codes, s and lo of one row
    if case["op"] == "store":
        rows = 2 * case["B"] * case["Hk"] * case["n"]
        # the rows read once, the cache written and read, the rows written
        return {"bytes": rows * (2 * d * 2 + 2 * packed), "flops": rows * d * 6}
    L = sum(_lengths(case))
    q_rows = case["B"] * case["Hq"] * case["nq"]
    if case["causal"]:
        pairs = sum(n * case["nq"] - case["nq"] * (case["nq"] - 1) // 2 for n in _lengths(case))
    else:
        pairs = L * case["nq"]
    return {"bytes": 2 * L * case["Hk"] * packed + q_rows * (4 * d + 4),
            "flops": 4 * d * pairs * case["Hq"]}


# --------------------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rows(g, B, Hk, n, d, dtype):
    """Keys and values of n tokens. Keys carry an offset per channel, as those of trained
    models do."""
    k = torch.randn(B, Hk, n, d, generator=g, device="cuda", dtype=dtype)
    k += torch.randn(1, Hk, 1, d, generator=g, device="cuda", dtype=dtype)
    v = torch.randn(B, Hk, n, d, generator=g, device="cuda", dtype=dtype)
    return k, v


def _table(g, B, tokens, page):
    """A page table of B rows for `tokens` tokens each, its pages in random order, and the
    number of pages in the pool."""
    per = -(-tokens // page)
    order = torch.randperm(B * per, generator=g, device="cuda")
    return order.reshape(B, per).to(torch.int32), B * per


def _inputs(case, seed):
    """Everything random of a case: rows to store, or cached rows and queries."""
    g = _generator(seed)
    dt = DTYPES[case["dtype"]]
    if case["op"] == "store":
        k, v = _rows(g, case["B"], case["Hk"], case["n"], case["d"], dt)
        table, pages = _table(g, case["B"], case["before"] + case["n"], case["page"])
        return {"k": k, "v": v, "table": table, "pages": pages}
    k, v = _rows(g, case["B"], case["Hk"], case["max_len"], case["d"], dt)
    table, pages = _table(g, case["B"], case["max_len"], case["page"])
    q = torch.randn(case["B"], case["Hq"], case["nq"], case["d"], generator=g, device="cuda",
                    dtype=dt)
    return {"k": k, "v": v, "table": table, "pages": pages, "q": q}


def prepare(case, seed):
    x = _inputs(case, seed)
    dt = DTYPES[case["dtype"]]
    B, Hk, d, page = case["B"], case["Hk"], case["d"], case["page"]
    st = {"case": case, "table": x["table"]}
    if case["op"] == "store":
        st["k"], st["v"] = x["k"], x["v"]
        st["start"] = torch.full((B,), case["before"], dtype=torch.int32, device="cuda")
    else:
        st["q"] = x["q"]
        st["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
    if own:
        import exact_io_aware_attention_gb300 as fa
        st["cache"] = fa.KVCache4(x["pages"], Hk, d, page_size=page, dtype=dt, device="cuda")
        if case["op"] == "attend":  # what earlier steps have written
            zero = torch.zeros(B, dtype=torch.int32, device="cuda")
            fa.cache_write(st["cache"], x["k"], x["v"], x["table"], zero, st["lengths"])
    else:
        shape = (x["pages"], Hk, page)
        st["cache"] = [(torch.zeros(*shape, d, dtype=torch.uint8, device="cuda"),
                        torch.zeros(*shape, d // GROUP, dtype=dt, device="cuda"),
                        torch.zeros(*shape, d // GROUP, dtype=dt, device="cuda"))
                       for _ in "kv"]
        if case["op"] == "attend":
            zero = torch.zeros(B, dtype=torch.int32, device="cuda")
            for c, rows in zip(st["cache"], (x["k"], x["v"])):
                _plain_write(c, rows, x["table"], zero, page)
    return st


# --------------------------------------------------------------------------- the plain form

def _places(table, start, n, page):
    """[B, n] page numbers and rows within the page of n tokens from each start."""
    pos = start.long()[:, None] + torch.arange(n, device="cuda")[None]
    return torch.gather(table.long(), 1, pos // page), pos % page


def _plain_quantise(x):
    """[..., d] rows -> codes [..., d] uint8, s and lo [..., d / 32] in x's type."""
    y = x.float().unflatten(-1, (-1, GROUP))
    lo = y.amin(-1, keepdim=True)
    fifteen = torch.full_like(lo, 15.0)  # a tensor: divided by, not multiplied with a reciprocal
    s = ((y.amax(-1, keepdim=True) - lo) / fifteen).to(x.dtype)
    sf = s.float()
    u = torch.where(sf > 0, torch.round((y - lo) / sf), torch.zeros_like(y)).clamp(max=15)
    return u.to(torch.uint8).flatten(-2), s.squeeze(-1), lo.squeeze(-1).to(x.dtype)


def _plain_write(cache, rows, table, start, page):
    B, Hk, n, d = rows.shape
    at_once = max(1, min(B, int(4e9 // (16 * Hk * n * d))))  # bounds the fp32 copies
    for b in range(0, B, at_once):
        e = min(b + at_once, B)
        pg, row = _places(table[b:e], start[b:e], n, page)
        for part, val in zip(cache, _plain_quantise(rows[b:e])):
            part[pg, :, row] = val.transpose(1, 2)


def _plain_read(cache, table, start, n, page):
    """[B, Hk, n, d] fp32 values that the cache stands for."""
    pg, row = _places(table, start, n, page)
    u, s, lo = (part[pg, :, row] for part in cache)  # [B, n, Hk, ...]
    y = u.float().unflatten(-1, (-1, GROUP)) * s.float()[..., None] + lo.float()[..., None]
    return y.flatten(-2).transpose(1, 2)


def _plain_attend(st):
    case = st["case"]
    q = st["q"].float()
    B, Hq, nq, d = q.shape
    Hk, page = case["Hk"], case["page"]
    G = Hq // Hk
    o = torch.empty(B, Hq, nq, d, device="cuda")
    lse = torch.empty(B, Hq, nq, device="cuda")
    L = case["max_len"]
    at_once = max(1, min(B, int(4e9 // (4 * (Hq * nq * L * 3 + Hk * L * d * 4)))))
    j = torch.arange(L, device="cuda")
    for b in range(0, B, at_once):
        e = min(b + at_once, B)
        zero = torch.zeros(e - b, dtype=torch.int32, device="cuda")
        k, v = (_plain_read(c, st["table"][b:e], zero, L, page) for c in st["cache"])
        x = q[b:e].reshape(e - b, Hk, G * nq, d) @ k.transpose(-1, -2)
        x = x.reshape(e - b, Hk, G, nq, L) * (1.0 / math.sqrt(d))
        n = st["lengths"][b:e].long()
        last = n[:, None] - 1
        if case["causal"]:
            last = n[:, None] - nq + torch.arange(nq, device="cuda")[None]
        hidden = j > last[..., None]  # [b, nq or 1, L]
        x.masked_fill_(hidden[:, None, None], float("-inf"))
        m = x.amax(-1, keepdim=True)
        p = torch.exp(x - m)
        l = p.sum(-1, keepdim=True)
        o[b:e] = ((p / l).reshape(e - b, Hk, G * nq, L) @ v).reshape(e - b, Hq, nq, d)
        lse[b:e] = (m + torch.log(l)).reshape(e - b, Hq, nq)
    return o.to(st["q"].dtype), lse


def run(state):
    case = state["case"]
    if own:
        import exact_io_aware_attention_gb300 as fa
        if case["op"] == "store":
            fa.cache_write(state["cache"], state["k"], state["v"], state["table"], state["start"])
            return fa.cache_read(state["cache"], state["table"], state["start"], case["n"])
        return fa.cache_forward(state["q"], state["cache"], state["table"], state["lengths"],
                                causal=case["causal"])
    if case["op"] == "store":
        dt = state["k"].dtype
        for c, rows in zip(state["cache"], (state["k"], state["v"])):
            _plain_write(c, rows, state["table"], state["start"], case["page"])
        return tuple(_plain_read(c, state["table"], state["start"], case["n"],
                                 case["page"]).to(dt) for c in state["cache"])
    return _plain_attend(state)


# --------------------------------------------------------------------------- 64 bits

def _exact_values(x):
    """What the cache stands for after x was written, in 64 bits."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for g in range(0, x.shape[-1], GROUP):
        y = x[..., g:g + GROUP].double()
        lo, hi = torch.aminmax(y, dim=-1, keepdim=True)
        s = torch.div(hi - lo, torch.full_like(lo, 15.0)).to(x.dtype).double()
        u = torch.nan_to_num(torch.div(y - lo, s), nan=0.0, posinf=0.0).round()
        out[..., g:g + GROUP] = lo + s * torch.minimum(u, torch.full_like(u, 15.0))
    return out


def exact(case, seed):
    x = _inputs(case, seed)
    B, Hk, d = case["B"], case["Hk"], case["d"]
    if case["op"] == "store":
        outs = []
        for t in ("k", "v"):
            y = torch.empty(x[t].shape, dtype=torch.float64, device="cuda")
            for b in range(B):
                y[b] = _exact_values(x[t][b])
            outs.append(y)
        return tuple(outs)
    Hq, nq = case["Hq"], case["nq"]
    if work(case)["flops"] > 8e12:  # 64-bit products run at about 1 TFLOP/s
        return None
    o = torch.empty(B, Hq, nq, d, dtype=torch.float64, device="cuda")
    lse = torch.empty(B, Hq, nq, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lengths(case)):
        for h in range(Hk):
            k, v = (_exact_values(x[t][b, h, :n]) for t in ("k", "v"))
            for hq in range(h * (Hq // Hk), (h + 1) * (Hq // Hk)):
                z = torch.mm(x["q"][b, hq].double(), k.T) / math.sqrt(d)
                if case["causal"]:
                    z += torch.full_like(z, float("-inf")).triu(n - nq + 1)
                lse[b, hq] = torch.logsumexp(z, -1)
                o[b, hq] = torch.mm(torch.softmax(z, -1), v)
    return o, lse
