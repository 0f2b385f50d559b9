"""Timed cases of the paged 8-bit key/value cache: page tables and slot maps (`slots`), the write of new keys and values
(`append`) and attention over the cache (`attn`), with the plain form of each."""
import math

import torch

own = False   # False: the plain forms below; True: the calls of dequant_gemv_rtn_b200

DEV = "cuda"
TOP = {"int8": 127.0, "e4m3": 448.0}          # the largest code's magnitude
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step of a small server: one token a row, now and then a new page (latency)
        {"name": "slots 8 rows", "op": "slots", "rows": 8, "page": 16, "most": 2000, "tokens": 8, "prompt": 0, "prompts": 0, "releases": 0, "spare": 200},
        # a large server's step: decode rows, some prompts, some rows released, the pool too small for the last rows
        {"name": "slots 1500 rows mixed", "op": "slots", "rows": 1500, "page": 64, "most": 32768, "tokens": 65536, "prompt": 2048, "prompts": 3, "releases": 5,
         "spare": 60},
        # the decode step's write: one token of 64 rows, mostly into pages begun before
        {"name": "append 64 decode rows", "op": "append", "rows": 64, "new": 1, "ragged": 0, "heads": 8, "dim": 128, "page": 64, "fmt": "int8", "dtype": "bf16"},
        # a prompt chunk's write: whole pages at once, small pages
        {"name": "append 8192 prompt tokens", "op": "append", "rows": 5, "new": 1639, "ragged": 0, "heads": 8, "dim": 128, "page": 16, "fmt": "e4m3", "dtype": "f16"},
        # drafted tokens of ragged count, one wide key/value head (4 query heads, dim 256: Gemma-3-1B's)
        {"name": "append 37 drafted rows", "op": "append", "rows": 37, "new": 9, "ragged": 1, "heads": 1, "dim": 256, "page": 32, "fmt": "int8", "dtype": "f16"},
        # one request on Llama-2-7B's 32 heads, no sharing of heads (latency)
        {"name": "attn 1 row 32 heads", "op": "attn", "rows": 1, "low": 700, "high": 700, "new": 1, "ragged": 0, "heads": 32, "group": 1, "dim": 128,
         "page": 16, "fmt": "int8", "dtype": "f16", "window": 0},
        # a full decode batch on Llama-70B's 64 query and 8 key/value heads, rows of very unlike length
        {"name": "attn 64 rows to 16384", "op": "attn", "rows": 64, "low": 1, "high": 16384, "new": 1, "ragged": 0, "heads": 8, "group": 8, "dim": 128,
         "page": 64, "fmt": "e4m3", "dtype": "bf16", "window": 0},
        # one long document
        {"name": "attn 1 row 131072", "op": "attn", "rows": 1, "low": 131072, "high": 131072, "new": 1, "ragged": 0, "heads": 8, "group": 8, "dim": 128,
         "page": 128, "fmt": "int8", "dtype": "f16", "window": 0},
        # Gemma-3-1B's local layers: one key/value head of 256, a sliding window
        {"name": "attn 24 rows window 512", "op": "attn", "rows": 24, "low": 100, "high": 8191, "new": 1, "ragged": 0, "heads": 1, "group": 4, "dim": 256,
         "page": 32, "fmt": "int8", "dtype": "bf16", "window": 512},
        # drafted tokens checked in one step: ragged counts, an odd number of query heads to a key/value head
        {"name": "attn 16 rows drafted 5", "op": "attn", "rows": 16, "low": 5, "high": 6001, "new": 5, "ragged": 1, "heads": 4, "group": 7, "dim": 128,
         "page": 16, "fmt": "e4m3", "dtype": "f16", "window": 0},
        # two prompt chunks against what is cached of them
        {"name": "attn 2 chunks of 1024", "op": "attn", "rows": 2, "low": 5000, "high": 8000, "new": 1024, "ragged": 0, "heads": 8, "group": 4, "dim": 128,
         "page": 64, "fmt": "int8", "dtype": "bf16", "window": 0},
        # many short requests on small heads
        {"name": "attn 128 rows to 512", "op": "attn", "rows": 128, "low": 1, "high": 512, "new": 1, "ragged": 0, "heads": 4, "group": 8, "dim": 64,
         "page": 16, "fmt": "e4m3", "dtype": "f16", "window": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw(rng):
    kind = rng.random()
    if kind < 0.2:
        rows = _log(rng, 1, 2048)
        prompt = rng.choice([0, _log(rng, 2, 4096)])
        return {"op": "slots", "rows": rows, "page": rng.choice([16, 32, 64, 128]), "most": _log(rng, 16, 32768), "tokens": min(131072, 3 * rows + 16 * prompt),
                "prompt": prompt, "prompts": rng.randint(1, 20) if prompt else 0, "releases": rng.choice([0, 0, rng.randint(1, 30)]),
                "spare": rng.choice([100, 150, 300, rng.randint(10, 99)])}
    heads, dim = rng.choice([1, 2, 3, 4, 8, 16, 32]), rng.choice([64, 128, 128, 256])
    c = {"heads": heads, "dim": dim, "page": rng.choice([16, 32, 64, 128]), "fmt": rng.choice(["int8", "e4m3"]), "dtype": rng.choice(["f16", "bf16"])}
    if kind < 0.45:
        new = rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 16, 4096)])
        return {"op": "append", "rows": _log(rng, 1, 512), "new": new, "ragged": int(new > 1 and rng.random() < 0.5), **c}
    new = rng.choice([1, 1, 1, rng.randint(2, 8), _log(rng, 9, 1024)])
    high = max(new, _log(rng, 16, 131072))
    return {"op": "attn", "rows": _log(rng, 1, 128), "low": max(new, rng.choice([new, high // 2, high])), "high": high, "new": new,
            "ragged": int(new > 1 and rng.random() < 0.5), **c, "group": rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 8, 16]),
            "window": rng.choice([0, 0, 0, _log(rng, 1, 4096)])}


def _fits(c):
    w = work(c)
    if c["op"] == "slots":
        return c["rows"] * (c["most"] + c["prompt"]) // c["page"] <= 1 << 21
    if c["op"] == "append":
        return c["rows"] * c["new"] * c["heads"] * c["dim"] <= 1639 * 5 * 8 * 128 and c["rows"] * c["page"] * c["heads"] * c["dim"] <= 1 << 24
    return (w["bytes"] <= 1.0e9 and w["flops"] <= 2.0e11 and c["rows"] * c["high"] * c["heads"] * c["dim"] <= 1 << 29
            and c["rows"] * c["heads"] * c["group"] * c["new"] * c["high"] <= 1 << 29)


def draw(rng):
    while True:
        c = _draw(rng)
        if _fits(c):
            return c


def _news(c):
    """New tokens of each row: alike, or 1 .. new."""
    return [1 + (5 * i + 3) % c["new"] if c["ragged"] else c["new"] for i in range(c["rows"])]


def _lens(c):
    """Cached tokens of each row, the new ones among them: spread over low .. high, the extremes included."""
    lo, hi, n = c["low"], c["high"], c["rows"]
    got = [lo + int((hi - lo) * ((i * 0.6180339887498949) % 1.0)) for i in range(n)]
    if n > 1:
        got[n // 2] = hi
    return [max(g, m) for g, m in zip(got, _news(c))]


def work(case):
    c = case
    if c["op"] == "slots":
        tokens = c["rows"] + c["rows"] * c["prompts"] * c["prompt"] // 200
        return {"bytes": 16 * c["rows"] + 4 * min(tokens, c["tokens"]) + 8 * (tokens // c["page"]), "flops": 0}
    if c["op"] == "append":
        t = sum(_news(c))
        return {"bytes": 2 * t * c["heads"] * (3 * c["dim"]) + 4 * t + 16 * c["heads"] * (c["rows"] + t // c["page"]), "flops": 0}
    read = flops = 0
    for n, length in zip(_news(c), _lens(c)):
        first = max(0, length - n - c["window"] + 1) if c["window"] else 0
        read += length - first
        for_all = sum(min(length - n + t + 1, c["window"] or length) for t in ((0, n // 2, n - 1) if n > 8 else range(n)))
        flops += 4 * c["dim"] * c["heads"] * c["group"] * for_all * (n / 3 if n > 8 else 1)
    t = sum(_news(c))
    return {"bytes": 2 * read * c["heads"] * (c["dim"] + 4 / c["page"]) + 4 * t * c["heads"] * c["group"] * c["dim"], "flops": flops}


# ------------------------------------------------------------------ inputs
def _shuffled(n, g):
    return torch.randperm(n, generator=g).to(torch.int32)


def _codes(x, fmt):
    """Codes and scales of x [pages, heads, page, dim], a scale for each page and head."""
    s = x.abs().amax((2, 3)) / TOP[fmt]
    x = x / s.clamp(min=1e-30)[:, :, None, None]
    codes = (x.round_() + 128).to(torch.uint8) if fmt == "int8" else x.to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.contiguous(), s.contiguous()


def _content(c, pages, gen):
    """Keys with a few strong channels and tokens of unlike size, values without: what a cache holds."""
    shape = (pages, c["heads"], c["page"], c["dim"])
    k = torch.randn(shape, device=DEV, generator=gen)
    channel = torch.randn(c["heads"], 1, c["dim"], device=DEV, generator=gen).mul_(0.4).exp_()
    channel[:, :, :: max(1, c["dim"] // 3)] *= 4
    k *= channel * torch.randn(pages, c["heads"], c["page"], 1, device=DEV, generator=gen).mul_(0.2).exp_()
    kc, ks = _codes(k, c["fmt"])
    del k
    v = torch.randn(shape, device=DEV, generator=gen)
    v *= torch.randn(pages, c["heads"], c["page"], 1, device=DEV, generator=gen).mul_(0.2).exp_()
    vc, vs = _codes(v, c["fmt"])
    return kc, vc, ks, vs


def prepare(case, seed):
    c = case
    g = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    if c["op"] == "slots":
        rows, P = c["rows"], c["page"]
        length = torch.randint(0, c["most"] + 1, (rows,), generator=g)
        add = torch.ones(rows, dtype=torch.int64)
        pick = torch.randint(0, 100, (rows,), generator=g)
        if c["prompts"]:
            prompt = pick < c["prompts"]
            length[prompt], add[prompt] = 0, torch.randint(1, c["prompt"] + 1, (int(prompt.sum()),), generator=g)
        add[pick >= 100 - c["releases"]] = -1
        length[0], add[0] = min(5, c["most"]), 1
        n = add.clamp(min=0)
        n[torch.cumsum(n, 0) > c["tokens"]] = 0
        add = torch.where(add > 0, n, add)
        width = -(-(c["most"] + max(1, c["prompt"])) // P)
        used, need = -(-length // P), -(-(length + n) // P) - -(-length // P)
        held = int(used.sum())
        spare = int(need.sum()) * c["spare"] // 100
        pages = rows * -(-c["most"] // P) + 3 * (c["tokens"] // P + rows) + 1
        order = _shuffled(pages, g)
        table = torch.full((rows, width), -1, dtype=torch.int32)
        table[torch.arange(width)[None] < used[:, None]] = order[:held]
        free = torch.full((pages,), -1, dtype=torch.int32)
        free[:spare] = order[held:held + spare]
        i32 = lambda x: x.to(device=DEV, dtype=torch.int32)  # noqa: E731
        return {"case": c, "pages": pages, "width": width, "len": i32(length), "add": i32(add), "table": i32(table), "free": i32(free),
                "free_count": torch.tensor([spare], dtype=torch.int32, device=DEV), "len_out": i32(torch.zeros(rows)), "cu": i32(torch.zeros(rows + 1)),
                "slots": i32(torch.zeros(c["tokens"])), "free_count_out": i32(torch.zeros(1))}
    news, P = _news(c), c["page"]
    n, dtype = torch.tensor(news), TYPES[c["dtype"]]
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(n, 0)])
    tokens = int(cu[-1]) + 3                       # the batch is padded: its last three rows belong to no request
    if c["op"] == "append":
        past = torch.randint(0, 4 * P, (c["rows"],), generator=g)   # of them only the page that is being filled counts
        past[0] = 0
        begun = past % P
        need = -(-(begun + n) // P)
        pages = sum(-(-(P - 1 + m) // P) for m in news) + 5
        order = _shuffled(pages, g).to(torch.int64)
        at = torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(need, 0)])
        row = torch.repeat_interleave(torch.arange(c["rows"]), n)
        pos = begun[row] + torch.arange(int(cu[-1])) - cu[row]
        slots = torch.full((tokens,), -1, dtype=torch.int32)
        slots[:-3] = (order[at[row] + pos // P] * P + pos % P).to(torch.int32)
        kc, vc, ks, vs = _content(c, pages, gen)
        qkv = torch.randn(tokens, 2 * c["heads"] * c["dim"] + 8 * c["dim"], device=DEV, generator=gen)
        k, v = (qkv[:, (8 + i * c["heads"]) * c["dim"]:][:, :c["heads"] * c["dim"]] for i in (0, 1))
        k *= torch.randn(c["heads"] * c["dim"], device=DEV, generator=gen).mul_(0.4).exp_()
        qkv = qkv.to(dtype)
        k, v = (qkv[:, (8 + i * c["heads"]) * c["dim"]:][:, :c["heads"] * c["dim"]] for i in (0, 1))
        return {"case": c, "pages": pages, "tokens": tokens, "k": k, "v": v, "slots": slots.to(DEV), "cu": cu.to(DEV, torch.int32),
                "k_codes": kc, "v_codes": vc, "k_scales": ks, "v_scales": vs}
    length = torch.tensor(_lens(c))
    order = torch.randperm(c["rows"], generator=g)
    length, n = length[order], n[order]             # another seed: the rows in another order
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(n, 0)])
    width = -(-c["high"] // P) + 1
    used = -(-length // P)
    pages = int(used.sum()) + 2
    table = torch.full((c["rows"], width), -1, dtype=torch.int32)
    table[torch.arange(width)[None] < used[:, None]] = _shuffled(pages, g)[:int(used.sum())]
    kc, vc, ks, vs = _content(c, pages, gen)
    heads = c["heads"] * c["group"]
    qkv = torch.randn(tokens, (heads + 2 * c["heads"]) * c["dim"], device=DEV, generator=gen).to(dtype)
    return {"case": c, "pages": pages, "tokens": tokens, "width": width, "q": qkv[:, :heads * c["dim"]], "len": length.to(DEV, torch.int32),
            "cu": cu.to(DEV, torch.int32), "table": table.to(DEV), "k_codes": kc, "v_codes": vc, "k_scales": ks, "v_scales": vs,
            "y": torch.zeros(tokens, heads * c["dim"], dtype=dtype, device=DEV)}


# ------------------------------------------------------------------ the library's calls
def _own(s):
    from dequant_gemv_rtn_b200 import qnt as Q
    c = s["case"]
    xdtype = Q.QNT_BF16 if c.get("dtype") == "bf16" else Q.QNT_F16
    if "desc" not in s:   # what a program keeps beside its cache
        s["desc"] = Q.kv_desc(Q.QNT_KV_E4M3 if c.get("fmt") == "e4m3" else Q.QNT_KV_INT8, c["page"], s["pages"], c.get("heads", 1), c.get("dim", 128))
    d = s["desc"]
    if c["op"] == "slots":
        Q.qnt_kv_slots(d, s["len"], s["add"], s["table"], s["free"], s["free_count"], s["len_out"], s["cu"], s["slots"], s["free_count_out"],
                       c["rows"], s["width"], c["tokens"])
        return {k: s[k] for k in ("table", "free", "len_out", "cu", "slots", "free_count_out")}
    if c["op"] == "append":
        Q.qnt_kv_append(d, s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"], s["k"], s["v"], s["k"].stride(0), s["slots"], s["tokens"], xdtype)
        return _cache(s)
    heads = c["heads"] * c["group"]
    if "work" not in s:
        s["work"] = torch.zeros(Q.qnt_kv_attn_work_bytes(d, heads, c["new"]), dtype=torch.uint8, device=DEV)
    Q.qnt_kv_attn(d, s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"], s["q"], s["q"].stride(0), s["y"], s["y"].stride(0), heads, s["cu"], s["len"],
                  s["table"], c["rows"], s["width"], s["tokens"], c["new"], 1 / math.sqrt(c["dim"]), c["window"], s["work"], xdtype)
    return s["y"]


def _cache(s):
    """The cache as it stands: INT8 codes are whole numbers (plus 128), E4M3 codes their values."""
    got = {k: s[k] if s["case"]["fmt"] == "int8" else s[k].view(torch.float8_e4m3fn) for k in ("k_codes", "v_codes")}
    return {**got, "k_scales": s["k_scales"], "v_scales": s["v_scales"]}


# ------------------------------------------------------------------ the plain forms
def _up(a, b):
    return -(-a // b)


def _plain_slots(s):
    c, P, dev = s["case"], s["case"]["page"], s["len"].device
    length, add, table, free, count = (s[k].long() for k in ("len", "add", "table", "free", "free_count"))
    width, tokens, pages = s["width"], c["tokens"], s["pages"]
    used, n = _up(length, P), add.clamp(min=0)
    out = torch.where(add < 0, used, 0)
    out_end = out.cumsum(0)
    ends = n.cumsum(0)
    fits = (length + n <= width * P) & (ends <= tokens)
    need = torch.where(fits, _up(length + n, P) - used, 0)
    end = need.cumsum(0)
    have = count + out_end[-1]
    ok = (add >= 0) & fits & ((need == 0) | (end <= have))
    taken = torch.where(ok, end, 0).amax()
    left = have - taken
    col = torch.arange(width, device=dev)[None]
    at = torch.where(col < out[:, None], (out_end - out)[:, None] + col, pages)
    released = torch.zeros(pages + 1, dtype=torch.int64, device=dev).scatter_(0, at.reshape(-1), table.reshape(-1))

    def stack(i):
        return torch.where(i < count, free[i.clamp(0, pages - 1)], released[(i - count).clamp(0, pages)])

    new = ok[:, None] & (col >= used[:, None]) & (col < (used + need)[:, None])
    table = torch.where(new, stack(have - 1 - ((end - need - used)[:, None] + col)), table)
    i = torch.arange(pages, device=dev)
    free = torch.where((i >= count) & (i < left), stack(i), free)
    cu = torch.cat([torch.zeros_like(ends[:1]), ends.clamp(max=tokens)])
    t = torch.arange(tokens, device=dev)
    row = torch.searchsorted(ends, t, right=True).clamp(max=c["rows"] - 1)
    pos = length[row] + t - (ends - n)[row]
    slot = table[row, (pos // P).clamp(0, width - 1)] * P + pos % P
    slot = torch.where((t < ends[-1]) & ok[row], slot, -1)
    i32 = torch.int32
    return {"table": table.to(i32), "free": free.to(i32), "len_out": torch.where(add < 0, 0, torch.where(ok, length + n, length)).to(i32), "cu": cu.to(i32),
            "slots": slot.to(i32), "free_count_out": left.to(i32)}


def _nearest(x, s, fmt):
    """Nearest code values of x / s, ties to even, in 64 bits (a quotient next to a tie decides a code); 0 where s is 0."""
    y = torch.where(s > 0, x.double() / s.double().clamp(min=1e-300), 0.0)
    if fmt == "int8":
        return y.round().clamp(-127, 127)
    step = torch.exp2((torch.frexp(y.abs())[1] - 1).clamp(min=-6) - 3.0)
    return ((y / step).round() * step).clamp(-448, 448)


def _byte(v, fmt):
    return (v + 128).to(torch.uint8) if fmt == "int8" else v.float().to(torch.float8_e4m3fn).view(torch.uint8)


def _value(b, fmt):
    return b.double() - 128 if fmt == "int8" else b.view(torch.float8_e4m3fn).double()


def _plain_append(s):
    c, fmt, P, H, D = s["case"], s["case"]["fmt"], s["case"]["page"], s["case"]["heads"], s["case"]["dim"]
    slots = s["slots"].long()
    live = (slots >= 0).nonzero()[:, 0]
    page, off = slots[live] // P, slots[live] % P
    start = torch.full((s["pages"],), P, device=DEV).scatter_reduce_(0, page, off, "amin")     # where the run begins in its page
    first = s["cu"][:-1].long()                       # only a request's first token can fall inside a page begun before
    mid = slots[first] // P
    for x, codes, scales in ((s["k"], s["k_codes"], s["k_scales"]), (s["v"], s["v_codes"], s["v_scales"])):
        x = x[live].float().view(-1, H, D)
        top = torch.zeros(s["pages"], H, device=DEV).scatter_reduce_(0, page[:, None].expand(-1, H), x.abs().amax(2), "amax")
        new = torch.maximum((top.double() / TOP[fmt]).float(), torch.where((start > 0)[:, None], scales, 0.0))
        new = torch.where((start < P)[:, None], new, scales)
        old = _value(codes[mid], fmt) * scales[mid].double()[:, :, None, None]
        old = _byte(_nearest(old, new[mid][:, :, None, None], fmt), fmt)
        kept = (torch.arange(P, device=DEV)[None] < start[mid][:, None])[:, None, :, None] & (new[mid] > scales[mid])[:, :, None, None]
        codes[mid] = torch.where(kept, old, codes[mid])
        codes[page, :, off] = _byte(_nearest(x, new[page][:, :, None], fmt), fmt)
        scales.copy_(new)
    return _cache(s)


def _plain_attn(s):
    c, P, H, D, G, N = s["case"], s["case"]["page"], s["case"]["heads"], s["case"]["dim"], s["case"]["group"], s["case"]["new"]
    B, dev = c["rows"], s["q"].device
    length, cu = s["len"].long(), s["cu"].long()
    n = cu[1:] - cu[:-1]
    t = torch.arange(N, device=dev)
    at = (cu[:-1, None] + t[None]).clamp(max=s["tokens"] - 1)
    table = s["table"].long().clamp(min=0)
    W = table.shape[1]

    def values(codes, scales):
        x = codes[table]                                                       # [B, W, H, P, D]
        x = x.float() - 128 if c["fmt"] == "int8" else x.view(torch.float8_e4m3fn).float()
        x *= scales[table][..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(B, H, W * P, D)

    q = s["q"].view(-1, H, G, D)[at].float().permute(0, 2, 3, 1, 4).reshape(B, H, G * N, D)
    score = (q @ values(s["k_codes"], s["k_scales"]).transpose(2, 3)).view(B, H, G, N, W * P)
    score *= 1 / math.sqrt(D)
    pos = (length - n)[:, None] + t[None]                                      # [B, N]
    j = torch.arange(W * P, device=dev)
    seen = (j <= pos[..., None]) & (j > pos[..., None] - (c["window"] or W * P))
    score.masked_fill_(~seen[:, None, None], -math.inf)
    score -= score.amax(-1, keepdim=True).clamp(min=-1e30)
    score.exp_()
    total = score.sum(-1, keepdim=True)
    o = score.view(B, H, G * N, W * P) @ values(s["v_codes"], s["v_scales"])
    o = (o.view(B, H, G, N, D) / total.clamp(min=1e-30)).permute(0, 3, 1, 2, 4).reshape(B, N, -1)
    live = t[None] < n[:, None]
    y = s["y"]
    y[at[live]] = o[live].to(y.dtype)
    return y


def run(state):
    if own:
        return _own(state)
    return {"slots": _plain_slots, "append": _plain_append, "attn": _plain_attn}[state["case"]["op"]](state)


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    c = case
    if c["op"] == "slots":
        return None
    s = prepare(case, seed)
    P, D, H = c["page"], c["dim"], c["heads"]
    cu, wide = s["cu"].tolist(), torch.float64
    if c["op"] == "append":
        slots = s["slots"].tolist()
        got = {}
        for name in ("k", "v"):
            x, scales = s[name].to(wide).view(-1, H, D), s[name + "_scales"].to(wide)
            limit = {}
            runs = {}
            for t, slot in enumerate(slots):
                if slot >= 0:
                    runs.setdefault(slot // P, []).append(t)
            for page, ts in runs.items():
                top = x[ts[0]:ts[-1] + 1].abs().amax((0, 2)) / TOP[c["fmt"]]
                limit[page] = torch.maximum(top, scales[page]) if slots[ts[0]] % P else top
            pages = torch.tensor(list(limit), device=DEV)
            scales[pages] = torch.stack(list(limit.values()))
            got[name + "_codes"], got[name + "_scales"] = None, scales
        return got
    length, table = s["len"].tolist(), s["table"].long()
    G = c["group"]
    y = torch.zeros(s["y"].shape, dtype=wide, device=DEV)
    for b in range(c["rows"]):
        n = cu[b + 1] - cu[b]
        begin = max(0, length[b] - n + 1 - c["window"]) // P * P if c["window"] else 0
        ids = table[b, begin // P:-(-length[b] // P)]
        both = []
        for name in ("k", "v"):
            code = s[name + "_codes"][ids]
            code = code.to(wide) - 128 if c["fmt"] == "int8" else code.view(torch.float8_e4m3fn).to(wide)
            both.append((code * s[name + "_scales"][ids].to(wide)[..., None, None]).transpose(0, 1).reshape(H, -1, D))
        q = s["q"][cu[b]:cu[b + 1]].to(wide).view(n, H, G, D).permute(1, 0, 2, 3).reshape(H, n * G, D)
        j = begin + torch.arange(both[0].shape[1], device=DEV)[None]
        pos = (length[b] - n + torch.arange(n, device=DEV)).repeat_interleave(G)[:, None]
        hide = (j > pos) | (j <= pos - c["window"]) if c["window"] else j > pos
        a = torch.einsum("hrd,hjd->hrj", q, both[0]) / math.sqrt(D)
        p = torch.softmax(a.masked_fill_(hide, -math.inf), -1)
        y[cu[b]:cu[b + 1]] = torch.einsum("hrj,hjd->hrd", p, both[1]).view(H, n, G, D).permute(1, 0, 2, 3).reshape(n, -1)
    return y
