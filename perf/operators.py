"""The operators of a paged key/value cache, as cases that can be timed and compared.

Four operators: new keys and values appended to the pages (in BF16, or quantised to E4M3 as they are written),
cached tokens read back as BF16, attention of a chunk of new tokens over the pages, and attention of single
tokens over them, the last two with an optional sliding window and a few first tokens that stay visible.
With ``own`` false ``run`` computes them with elementary torch operations in FP32, with ``own`` true through
``bf16_gemm_skinny_gb300``.

The cache.  ``pages[block, slot, kv_head, d]``; position p of sequence s lies in block ``tables[s, p // page]``,
slot ``p % page``.  In E4M3 every row (token, kv_head) has one scale 2^e, held as the byte e + 127 (E8M0):
e is the least integer with max|x| <= 448 * 2^e, kept within [-117, 120]; the codes are x / 2^e rounded to
nearest even.  (The scale is a power of two, so the codes stand for values that BF16 holds exactly.)

Attention.  The new tokens of a sequence are its last ones; the query at position p sees the positions t <= p
with t > p - window or t < sinks (window 0: all t <= p); out = softmax(scale * q K^T) V over those, and zeros where
there are none.
"""
import math
import random

import torch

own = False

NAMES = ("op", "type", "heads", "group", "dim", "page", "seqs", "new_lo", "new_hi", "old_lo", "old_hi", "window", "sinks")


def _case(name, *values):
    return dict(zip(NAMES, values), name=name)


def listed():
    return [
        # one decode step of a small batch writes its 16 new tokens: pure latency
        _case("append_decode_step", "append", "e4m3", 4, 4, 256, 784, 16, 1, 1, 100, 3000, 0, 0),
        # prompts of three requests are quantised into 784-token pages
        _case("append_prompts", "append", "e4m3", 4, 4, 256, 784, 3, 1500, 9000, 0, 700, 0, 0),
        # the same without quantisation, small pages, ragged prompts
        _case("append_bf16", "append", "bf16", 8, 4, 128, 16, 5, 100, 7000, 0, 100, 0, 0),
        # two long sequences leave the cache in BF16 (to be moved, or read by a kernel that takes no pages)
        _case("gather_long", "gather", "e4m3", 4, 4, 256, 784, 2, 12000, 16384, 0, 0, 0, 0),
        # the last tokens of a few short sequences, in pages of an odd size
        _case("gather_short", "gather", "e4m3", 4, 8, 64, 31, 4, 20, 200, 0, 50, 0, 0),
        # a prompt's last chunk of 2048 tokens, the context filled up to 32768: the largest
        _case("chunk_long", "chunk", "bf16", 4, 4, 256, 784, 1, 2048, 2048, 30720, 30720, 0, 0),
        # chunks of four requests over a quantised cache with small pages, ragged
        _case("chunk_ragged_e4m3", "chunk", "e4m3", 8, 4, 128, 16, 4, 300, 1000, 0, 7000, 0, 0),
        # a few drafted tokens of eight requests are verified at once
        _case("chunk_few_tokens", "chunk", "e4m3", 4, 4, 256, 784, 8, 1, 6, 2000, 9000, 0, 0),
        # a whole prompt of odd length with a sliding window and four sinks
        _case("chunk_window", "chunk", "bf16", 4, 8, 64, 64, 1, 4097, 4097, 0, 0, 1024, 4),
        # one user's long context, quantised: the stream of the cache
        _case("decode_long_e4m3", "decode", "e4m3", 4, 4, 256, 784, 1, 1, 1, 32767, 32767, 0, 0),
        # a batch with a sliding window and sinks over longer sequences
        _case("decode_window", "decode", "bf16", 4, 4, 256, 784, 8, 1, 1, 3000, 32000, 4096, 4),
        # a large batch of ordinary lengths, quantised, small pages
        _case("decode_batch_e4m3", "decode", "e4m3", 8, 8, 128, 16, 64, 1, 1, 100, 8000, 0, 0),
    ]


def draw(rng: random.Random):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("append", "gather", "chunk", "chunk", "decode", "decode"))
    c = {"op": op, "type": rng.choice(("bf16", "e4m3")), "heads": rng.choice((1, 2, 4, 8)), "group": rng.choice((1, 2, 4, 8)),
         "dim": rng.choice((64, 128, 256)), "page": rng.choice((8, 16, 31, 64, 784)), "window": 0, "sinks": 0}
    c["seqs"] = log(1, 64)
    if op in ("append", "gather"):
        tokens = log(c["seqs"], 16384)
        c["new_hi"] = max(1, tokens // c["seqs"])
        c["new_lo"] = rng.randint(1, c["new_hi"])
        c["old_lo"], c["old_hi"] = 0, log(1, 500)
    else:
        total = log(c["seqs"] * 8, 131072)
        c["old_hi"] = max(4, total // c["seqs"])
        c["old_lo"] = rng.randint(1, c["old_hi"])
        c["new_lo"], c["new_hi"] = 1, 1
        if op == "chunk":
            # pairs of query rows and keys stay under those of the largest listed case
            rows = 2048 * 16 * 32768 * 256 // (c["heads"] * c["group"] * c["dim"] * c["seqs"] * (c["old_hi"] + 1000) * 2)
            c["new_hi"] = log(1, max(1, min(2048, rows, 16384 // c["seqs"])))
            c["new_lo"] = rng.randint(1, c["new_hi"])
        if rng.random() < 0.4:
            c["window"], c["sinks"] = log(16, 4096), rng.choice((0, 1, 4, 64))
    return {k: c[k] for k in NAMES}


def _spread(lo, hi, n, turn):
    """n whole numbers from lo to hi, hi among them, the same for a case every time."""
    return [hi - int((hi - lo) * ((i * turn) % 1.0)) for i in range(n)]


def _lengths(c):
    """(new tokens, tokens in the cache after them) of each sequence."""
    new = _spread(c["new_lo"], c["new_hi"], c["seqs"], 0.6180339887)
    old = _spread(c["old_lo"], c["old_hi"], c["seqs"], 0.7548776662)
    return new, [a + b for a, b in zip(new, old)]


def _round_up_scale(amax):
    """The biased exponent (E8M0) of each row's scale, from max|x| in FP32."""
    m, e = torch.frexp(amax)                       # amax = m * 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = e - 9 + (m > 0.875).to(e.dtype)
    return torch.where(amax > 0, e.clamp(-117, 120), torch.full_like(e, -117)) + 127


def _power(e):
    """2^(e - 127) in FP32, 1 <= e <= 254."""
    return (e.int() << 23).view(torch.float32)


def _quantise(x):
    """Rows of BF16 values -> E4M3 codes and their scales' bytes."""
    x = x.float()
    e = _round_up_scale(x.abs().amax(-1))
    return (x * _power(254 - e).unsqueeze(-1)).to(torch.float8_e4m3fn), e.to(torch.uint8)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    new, lens = _lengths(c)
    page, heads, dim, hq = c["page"], c["heads"], c["dim"], c["heads"] * c["group"]
    blocks = [-(-n // page) for n in lens]
    num_blocks, max_blocks, tokens = sum(blocks) + 3, max(blocks), sum(new)
    order = torch.randperm(num_blocks, generator=g, device="cuda").to(torch.int32)
    tables = torch.zeros(c["seqs"], max_blocks, dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(blocks):
        tables[s, :n] = order[at:at + n]
        at += n

    def rows(*shape, spread=0.0):
        """Normal values; each channel with a size of its own."""
        x = torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)
        return x * torch.exp(spread * torch.randn(shape[-1], generator=g, device="cuda")).bfloat16() if spread else x

    st = {"case": c, "tables": tables, "num_blocks": num_blocks, "max_blocks": max_blocks, "tokens": tokens,
          "max_new": max(new), "max_len": max(lens), "scale": 1.0 / math.sqrt(dim),
          "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
          "cu": torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device="cuda")}
    k, v = rows(num_blocks, page, heads, dim, spread=0.4), rows(num_blocks, page, heads, dim, spread=0.2)
    if c["type"] == "e4m3":
        (st["k"], st["ks"]), (st["v"], st["vs"]) = _quantise(k), _quantise(v)
    else:
        st["k"], st["v"], st["ks"], st["vs"] = k, v, None, None
    # q, k and v of the new tokens lie side by side, as a fused projection leaves them
    fused = rows(tokens, (hq + 2 * heads) * dim)
    st["qkv"], st["stride"] = fused, fused.shape[1]
    st["q"] = fused[:, :hq * dim].mul_(1.5).view(tokens, hq, dim)
    st["new_k"] = fused[:, hq * dim:(hq + heads) * dim].view(tokens, heads, dim)
    st["new_v"] = fused[:, (hq + heads) * dim:].view(tokens, heads, dim)
    if c["op"] == "gather":
        st["out"] = [torch.empty(tokens, heads, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    elif c["op"] != "append":
        st["out"] = torch.empty(tokens, hq, dim, dtype=torch.bfloat16, device="cuda")
    return st


def _slots(st):
    """Row of the cache, and sequence and position, of each new token."""
    i = torch.arange(st["tokens"], device="cuda")
    s = torch.searchsorted(st["cu"], i.to(torch.int32), right=True) - 1
    p = st["lens"].long()[s] - (st["cu"].long()[s + 1] - i)
    page = st["case"]["page"]
    return st["tables"].long()[s, p // page] * page + p % page, s, p


def _plain_append(st):
    at = _slots(st)[0]
    out = []
    for name in ("k", "v"):
        x, cache, scales = st["new_" + name], st[name], st[name + "s"]
        if scales is not None:
            x, e = _quantise(x)
            scales.view(-1, scales.shape[-1])[at] = e
            cache.view(torch.uint8).view(-1, *cache.shape[2:])[at] = x.view(torch.uint8)
        else:
            cache.view(-1, *cache.shape[2:])[at] = x
        out += [cache] if scales is None else [cache, scales]
    return out


def _values(st, name, at):
    """FP32 values of the cache's rows `at`."""
    cache, scales = st[name], st[name + "s"]
    if scales is None:
        return cache.view(-1, *cache.shape[2:])[at].float()
    x = cache.view(torch.uint8).view(-1, *cache.shape[2:])[at].view(torch.float8_e4m3fn).float()
    return x * _power(scales.view(-1, scales.shape[-1])[at]).unsqueeze(-1)


def _plain_gather(st):
    at = _slots(st)[0]
    return [_values(st, name, at).bfloat16() for name in ("k", "v")]


def _plain_attention(st):
    c = st["case"]
    seqs, n, length, heads, group, dim = c["seqs"], st["max_new"], st["max_len"], c["heads"], c["group"], c["dim"]
    lens = st["lens"].long()
    t = torch.arange(length, device="cuda")
    there = t < lens[:, None]
    at = st["tables"].long().gather(1, (t // c["page"]).expand(seqs, length)) * c["page"] + t % c["page"]
    k, v = (_values(st, name, torch.where(there, at, 0)).masked_fill(~there[..., None, None], 0).transpose(1, 2) for name in ("k", "v"))
    _, s, p = _slots(st)
    row = torch.arange(st["tokens"], device="cuda") - st["cu"].long()[s]
    q = torch.zeros(seqs, n, heads * group, dim, device="cuda")
    q[s, row] = st["q"].float()
    q = q.view(seqs, n, heads, group, dim).permute(0, 2, 3, 1, 4).reshape(seqs, heads, group * n, dim)
    pos = torch.full((seqs, n), -1, device="cuda")
    pos[s, row] = p
    seen = (t <= pos[..., None]) & there[:, None]
    if c["window"]:
        seen &= (t > pos[..., None] - c["window"]) | (t < c["sinks"])
    x = (q @ k.transpose(-1, -2)).view(seqs, heads, group, n, length).mul_(st["scale"])
    x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp_(min=-3e38)
    x = x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x.view(seqs, heads, group * n, length) @ v).view(seqs, heads, group, n, dim) / total.clamp_(min=1e-37)
    return o.permute(0, 3, 1, 2, 4).reshape(seqs, n, heads * group, dim)[s, row].bfloat16()


def _own(st):
    import bf16_gemm_skinny_gb300 as bsk

    c = st["case"]
    kind = bsk.CACHE_E4M3 if c["type"] == "e4m3" else bsk.CACHE_BF16
    cache = (kind, st["k"], st["v"], st["ks"], st["vs"])
    shape = (c["heads"], c["dim"], c["page"], st["max_blocks"], st["num_blocks"])
    if c["op"] == "append":
        bsk.kv_cache_append_enqueue(*cache, st["new_k"], st["stride"], st["new_v"], st["stride"], st["cu"], st["tables"], st["lens"],
                                    c["seqs"], st["tokens"], *shape)
        return [st["k"], st["v"]] if st["ks"] is None else [st["k"], st["ks"], st["v"], st["vs"]]
    if c["op"] == "gather":
        bsk.kv_cache_gather_enqueue(*cache, *st["out"], st["cu"], st["tables"], st["lens"], c["seqs"], st["tokens"], *shape)
        return st["out"]
    width = c["heads"] * c["group"] * c["dim"]
    if c["op"] == "chunk":
        bsk.chunk_attention_enqueue(*cache, st["q"], st["stride"], st["out"], width, st["cu"], st["tables"], st["lens"], c["seqs"],
                                    st["tokens"], st["max_new"], c["heads"] * c["group"], *shape, st["max_len"], st["scale"],
                                    c["window"], c["sinks"])
    else:
        bsk.decode_attention_enqueue(*cache, st["q"], st["stride"], st["out"], width, st["tables"], st["lens"], c["seqs"],
                                     c["heads"] * c["group"], *shape, st["max_len"], st["scale"], c["window"], c["sinks"])
    return st["out"]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _plain_append(state) if op == "append" else _plain_gather(state) if op == "gather" else _plain_attention(state)


def _seen(c, new, length):
    """(pairs of a query and a visible key, keys that some query sees) of one sequence."""
    window, sinks = c["window"] or length + 1, c["sinks"]
    pairs = 0
    for p in range(length - new, length):
        low = max(0, p - window + 1)
        pairs += p + 1 - low + min(sinks, low)
    low = max(0, length - new - window + 1)
    return pairs, length - low + min(sinks, low)


def work(case):
    c = case
    new, lens = _lengths(c)
    tokens, row = sum(new), c["heads"] * c["dim"]
    cached = 2 * row * 2 if c["type"] == "bf16" else 2 * (row + c["heads"])   # a token's K and V in the cache
    where = 4 * (2 * c["seqs"] + 1) + 4 * sum(-(-n // c["page"]) for n in lens)
    if c["op"] in ("append", "gather"):
        return {"bytes": tokens * (cached + 2 * row * 2) + where, "flops": 0}
    seen = [_seen(c, a, b) for a, b in zip(new, lens)]
    return {"bytes": sum(k for _, k in seen) * cached + 2 * tokens * row * c["group"] * 2 + where,
            "flops": 4 * sum(p for p, _ in seen) * row * c["group"]}


def _exact_codes(x):
    """E4M3 values (as multiples of the scale) and exponent bytes of rows x, in 64 bits."""
    x = x.double()
    top = x.abs().amax(-1)
    e = torch.ceil(torch.log2((top / 448).clamp(min=2.0 ** -200)))
    e = torch.where(top > 448 * torch.exp2(e), e + 1, torch.where(top <= 448 * torch.exp2(e - 1), e - 1, e)).clamp(-117, 120)
    y = x / torch.exp2(e)[..., None]
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step, e + 127


def exact(case, seed):
    st = prepare(case, seed)
    c, page = case, case["page"]
    new, lens = _lengths(c)
    tables = st["tables"].tolist()

    def places(s, first, last):
        return torch.tensor([tables[s][p // page] * page + p % page for p in range(first, last)], device="cuda")

    def wide(name, at):
        x = st[name].view(-1, *st[name].shape[2:])
        if st["ks"] is None:
            return x[at].double()
        x = x.view(torch.uint8)[at].view(torch.float8_e4m3fn).double()
        return x * torch.exp2(st[name + "s"].view(-1, c["heads"])[at].double() - 127)[..., None]

    if c["op"] == "append":
        at = torch.cat([places(s, b - a, b) for s, (a, b) in enumerate(zip(new, lens))])
        out = []
        for name in ("k", "v"):
            cache = st[name].double()
            if st["ks"] is None:
                cache.view(-1, *cache.shape[2:])[at] = st["new_" + name].double()
                out.append(cache)
            else:
                y, _ = _exact_codes(st["new_" + name])
                cache.view(-1, *cache.shape[2:])[at] = y
                out += [cache, None]
        return out
    if c["op"] == "gather":
        at = torch.cat([places(s, b - a, b) for s, (a, b) in enumerate(zip(new, lens))])
        return [wide("k", at), wide("v", at)]
    if work(case)["flops"] > 2e12:
        return None
    out, first = [], 0
    for s, (a, b) in enumerate(zip(new, lens)):
        at = places(s, 0, b)
        k, v = wide("k", at), wide("v", at)
        part = torch.empty(a, c["heads"] * c["group"], c["dim"], dtype=torch.float64, device="cuda")
        t = torch.arange(b, device="cuda")
        for lo in range(0, a, 256):
            hi = min(a, lo + 256)
            p = torch.arange(b - a + lo, b - a + hi, device="cuda")[:, None]
            hidden = t > p
            if c["window"]:
                hidden = hidden | ((t <= p - c["window"]) & (t >= c["sinks"]))
            for h in range(c["heads"] * c["group"]):
                j = h // c["group"]
                x = st["q"][first + lo:first + hi, h].double() @ k[:, j].T * st["scale"]
                part[lo:hi, h] = torch.softmax(x.masked_fill(hidden, -math.inf), -1) @ v[:, j]
        out.append(part)
        first += a
    return torch.cat(out)
