"""The operators between the projections of a layer that is served from 4-bit
codes: keys and values rotated and appended to a paged 4-bit cache, the cache's
rows read back, attention over that cache (one or many new tokens of each
sequence, with a sliding window and first tokens that stay visible), and the
low-rank adapters of many requests beside a shared projection.  Cases, inputs,
plain forms and 64-bit results of each."""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
BLOCK = 32           # tokens whose values share the words of a page


def listed():
    return [
        # one sequence's next token: 40 query heads of a 5120-wide model, 8 key/value heads
        {"name": "append-1x1-after-1000", "op": "append", "B": 1, "new": 1, "ctx": 1000, "H": 8, "R": 5, "D": 128,
         "g": 64, "page": 64, "rot": 128, "inter": False, "given": False, "dtype": "fp16"},
        # a prefill batch of three ragged prompts, 6147 tokens, behind prefixes that the cache holds already
        {"name": "append-3x2731-ragged", "op": "append", "B": 3, "new": 2731, "ctx": 333, "H": 8, "R": 5, "D": 128,
         "g": 64, "page": 64, "rot": 128, "inter": False, "given": False, "dtype": "bf16"},
        # a short sequence's rows back out of the cache (to hand it to another worker)
        {"name": "read-1x777", "op": "read", "B": 1, "len": 777, "H": 8, "D": 128, "g": 64, "page": 64, "dtype": "fp16"},
        # a whole batch's prefixes read back in one call
        {"name": "read-8x16000-ragged", "op": "read", "B": 8, "len": 16000, "H": 8, "D": 128, "g": 64, "page": 64,
         "dtype": "bf16"},
        # decode: one sequence with a short context, where latency counts
        {"name": "attend-1x1-of-1000", "op": "attend", "B": 1, "new": 1, "len": 1000, "ragged": False, "H": 8, "R": 5,
         "D": 128, "g": 64, "page": 64, "window": 0, "sinks": 0, "dtype": "fp16"},
        # decode: a batch of 16 ragged sequences up to 8191 tokens
        {"name": "attend-16x1-of-8191", "op": "attend", "B": 16, "new": 1, "len": 8191, "ragged": True, "H": 8, "R": 5,
         "D": 128, "g": 64, "page": 64, "window": 0, "sinks": 0, "dtype": "bf16"},
        # decode: one very long context, the work split along it
        {"name": "attend-1x1-of-131072", "op": "attend", "B": 1, "new": 1, "len": 131072, "ragged": False, "H": 8,
         "R": 8, "D": 128, "g": 128, "page": 64, "window": 0, "sinks": 0, "dtype": "bf16"},
        # decode: a large batch through a windowed layer with four first tokens kept
        {"name": "attend-64x1-window1000", "op": "attend", "B": 64, "new": 1, "len": 5000, "ragged": True, "H": 8,
         "R": 4, "D": 128, "g": 32, "page": 32, "window": 1000, "sinks": 4, "dtype": "fp16"},
        # chunked prefill: two prompts' next chunks over what is cached of them
        {"name": "attend-2x2048-of-6100", "op": "attend", "B": 2, "new": 2048, "len": 6100, "ragged": True, "H": 8,
         "R": 5, "D": 128, "g": 64, "page": 64, "window": 0, "sinks": 0, "dtype": "bf16"},
        # adapters: one token at decode
        {"name": "lora-1-of-8-rank16", "op": "lora", "T": 1, "L": 8, "rank": 16, "K": 5120, "N": 5120, "none": 0.0,
         "dtype": "fp16"},
        # adapters: a decode batch of 64 requests over 32 adapters at the MLP's width, some without one
        {"name": "lora-64-of-32-rank16", "op": "lora", "T": 64, "L": 32, "rank": 16, "K": 5120, "N": 17408,
         "none": 0.1, "dtype": "bf16"},
        # adapters: a prefill batch, odd token count
        {"name": "lora-4093-of-8-rank64", "op": "lora", "T": 4093, "L": 8, "rank": 64, "K": 5120, "N": 17408,
         "none": 0.0, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "attend", "attend", "attend", "lora"])
    dtype = rng.choice(["fp16", "bf16"])
    D = rng.choice([64, 128, 128, 256])
    g = rng.choice([n for n in (32, 64, 128) if n <= D])
    H = rng.choice([1, 2, 4, 8])
    heads = {"H": H, "D": D, "g": g, "page": rng.choice([32, 64, 128, 256])}
    if op == "append":
        B = _log_int(rng, 1, 64)
        new = rng.choice([1, _log_int(rng, 1, max(2, 3000 // B))])
        return {"op": op, "B": B, "new": new, "ctx": rng.randint(0, 700), **heads,
                "R": rng.randint(1, max(1, 2560 // (H * D))), "rot": rng.choice([0, D // 2, D, D]),
                "inter": rng.random() < 0.4, "given": rng.random() < 0.3, "dtype": dtype}
    if op == "read":
        B = _log_int(rng, 1, 32)
        return {"op": op, "B": B, "len": _log_int(rng, 1, 60000 // B), **heads, "dtype": dtype}
    if op == "attend":
        R = rng.randint(1, 10)
        window = rng.choice([0, 0, _log_int(rng, 1, 4000)])
        kind = rng.choice(["one", "one", "few", "many"])
        if kind == "many":
            B = rng.randint(1, 3)
            new = _log_int(rng, 100, 1200)
            length = new + _log_int(rng, 1, 3000)
            R = rng.randint(1, max(1, 4096 // (H * D)))
        else:
            B = _log_int(rng, 1, 64)
            new = 1 if kind == "one" else rng.randint(2, 9)
            length = new + _log_int(rng, 1, 130000 // B)
        return {"op": op, "B": B, "new": new, "len": length, "ragged": rng.random() < 0.7, **heads, "R": R,
                "window": window, "sinks": rng.choice([0, 1, 4, 40]) if window else 0, "dtype": dtype}
    rank = rng.choice([8, 16, 32, 64, 128])
    return {"op": op, "T": _log_int(rng, 1, 3500), "L": rng.randint(1, 1024 // rank), "rank": rank,
            "K": 8 * _log_int(rng, 32, 1000), "N": 8 * _log_int(rng, 32, 1500),
            "none": rng.choice([0.0, 0.0, 0.2]), "dtype": dtype}


# ---- a batch of sequences in a paged cache ----
# k, v    [pages, H, page, D/8] int32, eight codes a word
# k_sz    [pages, H, D/g, page, 2] fp16: scale and zero of each token's groups (v_sz the same)
# A key's words: of a token [4][D/32]: word (q, 2i + l) holds in nibble 4a + 2b + c the channel
#   32 (i + c D/64) + 8 q + 4 l + 2 b + a.
# A value's words: of 32 tokens [D/64][4][16][4]: word (u, q, m, j) holds in nibble 4a + 2b + c the
#   channel 64 u + 16 j + m of the token 16 c + 4 q + 2 b + a.

def _lengths(B, n, ragged=True):
    """n and, ragged, less down to a half, spread evenly over the batch."""
    return [n - (n // 2) * b // max(B - 1, 1) if ragged else n for b in range(B)]


def _shifts(device):
    return 4 * torch.arange(8, dtype=torch.int32, device=device)


def _pack_k(codes):
    D = codes.shape[-1]
    c = codes.unflatten(-1, (2, D // 64, 4, 2, 2, 2))                # c, i, q, l, b, a
    n = c.dim() - 6
    c = c.permute(*range(n), n + 2, n + 1, n + 3, n + 5, n + 4, n).flatten(n + 3)
    return (c << _shifts(codes.device)).sum(-1, dtype=torch.int32).flatten(n)


def _unpack_k(words, D):
    c = (words[..., None] >> _shifts(words.device)) & 15
    n = words.dim() - 1
    c = c.flatten(n).unflatten(n, (4, D // 64, 2, 2, 2, 2))          # q, i, l, a, b, c
    return c.permute(*range(n), n + 5, n + 1, n, n + 2, n + 4, n + 3).flatten(n)


def _pack_v(codes):
    """codes [..., tokens, D], whole blocks of 32 tokens."""
    T, D = codes.shape[-2:]
    n = codes.dim() - 2
    c = codes.unflatten(-1, (D // 64, 4, 16)).unflatten(n, (T // BLOCK, 2, 4, 2, 2))   # block, c, q, b, a, u, j, m
    c = c.permute(*range(n + 1), n + 5, n + 2, n + 7, n + 6, n + 4, n + 3, n + 1).flatten(n + 5)
    return (c << _shifts(codes.device)).sum(-1, dtype=torch.int32).flatten(n).unflatten(n, (T, D // 8))


def _unpack_v(words):
    T, D = words.shape[-2], words.shape[-1] * 8
    n = words.dim() - 2
    w = words.flatten(n).unflatten(n, (T // BLOCK, D // 64, 4, 16, 4))                 # block, u, q, m, j
    c = ((w[..., None] >> _shifts(words.device)) & 15).unflatten(-1, (2, 2, 2))        # a, b, c
    c = c.permute(*range(n + 1), n + 7, n + 2, n + 6, n + 5, n + 1, n + 4, n + 3)      # block, c, q, b, a, u, j, m
    return c.flatten(n + 5).flatten(n, n + 4)


def _group_codes(x, g):
    """Codes and (scale, zero) of fp32 rows [..., D], one pair for each g channels."""
    p = x.unflatten(-1, (-1, g))
    lo, hi = p.amin(-1, keepdim=True), p.amax(-1, keepdim=True)
    # true quotients: a plain number would be multiplied by its inverse
    s = ((hi - lo) / torch.full_like(lo, 15.0)).half()
    z = lo.half()
    q = torch.round((p - z.float()) / s.float()).nan_to_num(0.0).clamp(0, 15)
    return q.to(torch.int32).flatten(-2), torch.cat([s, z], -1)


def _cache(rows, c, gen):
    """A cache of `rows` pages whose tokens are normal values with a few large key channels."""
    H, D, g, page = c["H"], c["D"], c["g"], c["page"]
    made = {}
    for name in ("k", "v"):
        x = torch.randn((rows, H, page, D), device="cuda", generator=gen)
        if name == "k":
            x *= torch.where(torch.rand((H, 1, D), device="cuda", generator=gen) < 0.03, 4.0, 1.0)
        codes, sz = _group_codes(x, g)
        made[name] = (_pack_k if name == "k" else _pack_v)(codes).contiguous()
        made[name + "_sz"] = sz.transpose(2, 3).contiguous()
    return made


def _batch(c, lens, news, gen):
    """Lengths, offsets of the new rows and a page table, its pages in any order."""
    width = -(-max(lens) // c["page"]) + 1
    counts = [-(-n // c["page"]) for n in lens]
    pages = sum(counts) + 3
    order = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = order[at:at + n]
        at += n
    off = [0]
    for n in news:
        off.append(off[-1] + n)
    return {"lens": torch.tensor(lens, dtype=torch.int32, device="cuda"), "table": table, "T": off[-1],
            "off": torch.tensor(off, dtype=torch.int32, device="cuda"), "pages": pages}


def _sequences(c):
    """(lengths, new rows) of the batch's sequences."""
    if c["op"] == "append":
        news = _lengths(c["B"], c["new"])
        return [n + m for n, m in zip(news, _lengths(c["B"], c["ctx"]))], news
    lens = _lengths(c["B"], c["len"], c.get("ragged", True))
    if c["op"] == "read":
        return lens, lens
    news = [min(n, m) for n, m in zip(_lengths(c["B"], c["new"], c["ragged"]), lens)]
    return lens, [max(n, 1) for n in news]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    c, s, op = case, {"case": case}, case["op"]
    dt = DTYPES[c["dtype"]]
    if op == "lora":
        T, L, rank, K, N = (c[n] for n in ("T", "L", "rank", "K", "N"))
        x = torch.randn((T, K), device="cuda", generator=gen)
        s["x"] = (x * torch.where(torch.rand(K, device="cuda", generator=gen) < 0.01, 8.0, 1.0)).to(dt)
        s["a"] = (torch.randn((L, rank, K), device="cuda", generator=gen) / math.sqrt(K)).to(dt)
        s["b"] = (torch.randn((L, N, rank), device="cuda", generator=gen) * 0.05).to(dt)
        s["scaling"] = torch.rand(L, device="cuda", generator=gen) + 0.5
        s["y"] = torch.randn((T, N), device="cuda", generator=gen).to(dt)
        ids = torch.randint(0, L, (T,), device="cuda", generator=gen)
        ids = torch.where(torch.rand(T, device="cuda", generator=gen) < c["none"], L, ids)
        # the plan of the batch: its rows by adapter, those without one behind
        by, order = torch.sort(ids, stable=True)
        s["off"] = torch.searchsorted(by, torch.arange(L + 1, device="cuda")).to(torch.int32)
        s["rows"] = torch.where(by < L, order, -1).to(torch.int32)
        place = torch.where(by < L, torch.arange(T, device="cuda"), -1)
        s["slots"] = torch.empty_like(place).scatter_(0, order, place).to(torch.int32)[:, None].contiguous()
        s["ids"] = ids
        return s
    H, D = c["H"], c["D"]
    lens, news = _sequences(c)
    s.update(_batch(c, lens, news, gen))
    T = s["T"]
    s["cache"] = _cache(s["pages"], c, gen)
    s["news"] = max(news)
    if op == "append":
        R, rot = c["R"], c["rot"]
        # a projection's output: each token's queries, keys and values side by side
        qkv = torch.randn((T, (R + 2) * H * D), device="cuda", generator=gen).to(dt)
        s["q"], s["k"], s["v"] = (t.unflatten(1, (-1, D)) for t in qkv.split([R * H * D, H * D, H * D], 1))
        s["q_out"] = torch.empty((T, R * H, D), dtype=dt, device="cuda")
        s["k_out"], s["v_out"] = (torch.empty((T, H, D), dtype=dt, device="cuda") for _ in range(2))
        first = 100000 if c["given"] else 0
        s["positions"] = (first + _index(s["off"], s["lens"], T)[1]).to(torch.int32) if c["given"] else None
        if rot:
            # angles in 64 bits: those of far positions lose their digits in 32
            at = torch.arange(first + max(lens) + 1, device="cuda", dtype=torch.float64)
            by = 1e6 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
            angle = at[:, None] * by
            s["cos_sin"] = torch.cat([torch.cos(angle), torch.sin(angle)], 1).float()
        else:
            s["cos_sin"] = None
    elif op == "read":
        s["k_out"], s["v_out"] = (torch.empty((T, H, D), dtype=dt, device="cuda") for _ in range(2))
    else:
        s["q"] = torch.randn((T, H * c["R"], D), device="cuda", generator=gen).to(dt)
        s["out"] = torch.empty_like(s["q"])
        s["scale"] = 1.0 / math.sqrt(D)
    return s


def _index(off, lens, T):
    """The sequence of each row and its place in it."""
    row = torch.arange(T, device=off.device)
    b = torch.searchsorted(off.long(), row, right=True) - 1
    return b, row - off.long()[b + 1] + lens.long()[b]


def _places(s):
    """Page and place in the page of each row."""
    b, at = _index(s["off"], s["lens"], s["T"])
    page = s["case"]["page"]
    return s["table"][b, at // page].long(), at % page


def _rotate(x, cos_sin, at, rot, inter):
    if not rot:
        return x
    cos, sin = cos_sin[at][:, None].chunk(2, -1)
    part, rest = x[..., :rot], x[..., rot:]
    a, b = (part[..., 0::2], part[..., 1::2]) if inter else part.chunk(2, -1)
    y = (a * cos - b * sin, b * cos + a * sin)
    y = torch.stack(y, -1).flatten(-2) if inter else torch.cat(y, -1)
    return torch.cat([y, rest], -1)


def _read_plain(s):
    c, cache = s["case"], s["cache"]
    page, slot = _places(s)
    D, g, H = c["D"], c["g"], c["H"]
    k = _unpack_k(cache["k"][page, :, slot], D)                               # [T, H, D]
    # a value's code: the word of its block, place and channel, and the nibble
    d = torch.arange(D, device=page.device)
    at, nib = _value_word(slot, d, D)
    flat = cache["v"].flatten(2)
    head = torch.arange(H, device=page.device)
    w = flat[page[:, None, None], head[None, :, None], at[:, None, :]]
    v = (w >> nib[:, None, None]) & 15
    outs = []
    for codes, name in ((k, "k_sz"), (v, "v_sz")):
        sz = cache[name][page, :, :, slot].float()                            # [T, H, D/g, 2]
        outs.append((codes.unflatten(-1, (-1, g)).float() * sz[..., :1] + sz[..., 1:]).flatten(-2))
    dt = DTYPES[c["dtype"]]
    return outs[0].to(dt), outs[1].to(dt)


def _value_word(slot, d, D):
    """Index of the word (in a head's page) of each token's channels, and the shift of the token's nibble."""
    t = slot % BLOCK
    hi, q, b, a = t // 16, t // 4 % 4, t // 2 % 2, t % 2
    at = (slot // BLOCK * (BLOCK * D // 8))[:, None] + ((d // 64 * 4 + q[:, None]) * 16 + d % 16) * 4 + d // 16 % 4
    return at, (4 * (4 * a + 2 * b + hi)).to(torch.int32)


def _append_plain(s):
    c, cache = s["case"], s["cache"]
    b, place = _index(s["off"], s["lens"], s["T"])
    at = s["positions"].long() if s["positions"] is not None else place
    page, slot = _places(s)
    k = _rotate(s["k"].float(), s["cos_sin"], at, c["rot"], c["inter"])
    q = _rotate(s["q"].float(), s["cos_sin"], at, c["rot"], c["inter"]).to(s["q"].dtype)
    codes, sz = _group_codes(k, c["g"])
    cache["k"][page, :, slot] = _pack_k(codes)
    cache["k_sz"][page, :, :, slot] = sz
    codes, sz = _group_codes(s["v"].float(), c["g"])
    cache["v_sz"][page, :, :, slot] = sz
    # a word is shared by eight tokens: each adds what its nibble changes by
    d = torch.arange(c["D"], device=page.device)
    word, nib = _value_word(slot, d, c["D"])
    flat = cache["v"].view(-1)
    head = torch.arange(c["H"], device=page.device)
    word = (page[:, None, None] * c["H"] + head[None, :, None]) * (c["page"] * c["D"] // 8) + word[:, None, :]
    old = (flat[word] >> nib[:, None, None]) & 15
    flat.index_add_(0, word.flatten(), ((codes - old) << nib[:, None, None]).flatten())
    return (q, *_read_plain(s))


def _dense(s):
    """The batch's keys and values [B, H, tokens, D] in 32 bits, padded to the table's width."""
    c, cache = s["case"], s["cache"]
    pages = s["table"].clamp_min(0).long()
    outs = []
    for name in ("k", "v"):
        w = cache[name][pages].transpose(1, 2).flatten(2, 3)                  # [B, H, tokens, D/8]
        codes = _unpack_k(w, c["D"]) if name == "k" else _unpack_v(w)
        sz = cache[name + "_sz"][pages].permute(0, 2, 1, 4, 3, 5).flatten(2, 3).float()
        outs.append((codes.unflatten(-1, (-1, c["g"])).float() * sz[..., :1] + sz[..., 1:]).flatten(-2))
    return outs


def _attend_plain(s):
    c = s["case"]
    k, v = _dense(s)
    B, H, L, D = k.shape
    n, R = s["news"], c["R"]
    off, lens = s["off"].long(), s["lens"].long()
    i = torch.arange(n, device=k.device)
    live = i < (off[1:] - off[:-1])[:, None]                                  # [B, n]
    rows = torch.where(live, off[:-1, None] + i, 0)
    q = s["q"].float()[rows].view(B, n, H, R, D).permute(0, 2, 1, 3, 4).reshape(B, H, n * R, D)
    score = torch.matmul(q, k.transpose(2, 3).contiguous()) * s["scale"]
    pos = (lens - off[1:] + off[:-1])[:, None] + i
    t = torch.arange(L, device=k.device)
    seen = t <= pos[..., None]
    if c["window"]:
        seen &= (t > pos[..., None] - c["window"]) | (t < c["sinks"])
    seen = seen[:, None, :, None, :].expand(B, 1, n, R, L).reshape(B, 1, n * R, L)
    score = torch.where(seen, score, -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    o = torch.matmul(p, v).view(B, H, n, R, D).permute(0, 2, 1, 3, 4).reshape(B, n, H * R, D)
    b, _ = _index(s["off"], s["lens"], s["T"])
    return o[b, torch.arange(s["T"], device=k.device) - off[b]].to(s["q"].dtype)


def _lora_plain(s):
    c = s["case"]
    L, rank = c["L"], c["rank"]
    h = torch.matmul(s["x"].float(), s["a"].float().view(L * rank, -1).t())
    mine = (s["ids"][:, None] == torch.arange(L, device=h.device)) * s["scaling"]
    h = (h.view(-1, L, rank) * mine[..., None]).flatten(1)
    b = s["b"].float().transpose(1, 2).reshape(L * rank, -1)
    s["y"].copy_(s["y"].float() + torch.matmul(h, b))
    return s["y"]


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        import int4_weight_only_uint32_amd as qg
        if op == "lora":
            return qg.lora(s["x"], s["a"], s["b"], (s["off"], s["rows"], s["slots"]), s["y"], scaling=s["scaling"])
        cache = qg.KV4Cache(**s["cache"])
        if op == "append":
            qg.kv4_append(cache, s["k"], s["v"], s["lens"], s["table"], seq_offsets=s["off"],
                          positions=s["positions"], cos_sin=s["cos_sin"], interleaved=c["inter"], q=s["q"],
                          q_out=s["q_out"])
            # the codes come back as the values that they stand for
            return (s["q_out"], *qg.kv4_read(cache, s["lens"], s["table"], seq_offsets=s["off"], k_out=s["k_out"],
                                             v_out=s["v_out"]))
        if op == "read":
            return qg.kv4_read(cache, s["lens"], s["table"], seq_offsets=s["off"], k_out=s["k_out"], v_out=s["v_out"])
        return qg.kv4_attend(s["q"], cache, s["lens"], s["table"], seq_offsets=s["off"], max_new=s["news"],
                             scale=s["scale"], window=c["window"], sinks=c["sinks"], out=s["out"])
    if op == "lora":
        return _lora_plain(s)
    if op == "append":
        return _append_plain(s)
    if op == "read":
        return _read_plain(s)
    return _attend_plain(s)


def _token_bytes(c):
    """A token's codes, scales and zeros, of keys and values, in all heads."""
    return c["H"] * (c["D"] + 8 * (c["D"] // c["g"]))


def work(case):
    c, op = case, case["op"]
    if op == "lora":
        T, L, rank, K, N = (c[n] for n in ("T", "L", "rank", "K", "N"))
        T = T * (1 - c["none"])
        used = L * (1 - (1 - 1 / L) ** T)
        return {"bytes": 2 * (T * K + used * rank * (K + N) + 2 * T * N) + 4 * (3 * T + 2 * L),
                "flops": 2 * T * rank * (K + N)}
    lens, news = _sequences(c)
    T, H, D = sum(news), c["H"], c["D"]
    if op == "append":
        # the call and the reading of what it wrote
        return {"bytes": T * (2 * D * H * (2 * c["R"] + 2) + 4 * c["rot"] + 2 * _token_bytes(c) + 4 * D * H),
                "flops": T * D * H * (3 * c["R"] + 14)}
    if op == "read":
        return {"bytes": T * (_token_bytes(c) + 4 * D * H), "flops": 4 * T * D * H}
    pairs = reach = 0
    for n, m in zip(lens, news):
        w, k = c["window"], c["sinks"]
        first = n - m
        if not w:
            pairs += m * first + m * (m + 1) // 2
            reach += n
            continue
        pairs += sum(min(p + 1, w) + min(k, max(0, p + 1 - w)) for p in range(first, n))
        reach += min(n, m - 1 + w + k)
    return {"bytes": reach * _token_bytes(c) + 4 * T * H * c["R"] * D, "flops": 4 * D * H * c["R"] * pairs}


# ---- the definitions in 64 bits ----

def _exact_group(x, g):
    """The values that the codes of 64-bit rows stand for."""
    out = torch.empty_like(x)
    for u in range(0, x.shape[-1], g):
        p = x[..., u:u + g]
        lo, hi = p.min(-1, keepdim=True).values, p.max(-1, keepdim=True).values
        s = ((hi - lo) / 15).half().to(torch.float64)
        z = lo.half().to(torch.float64)
        code = torch.where(s > 0, ((p - z) / s).round().clamp(0, 15), 0)
        out[..., u:u + g] = code * s + z
    return out


def _exact_rotated(x, table, at, rot, inter):
    y = x.to(torch.float64).clone()
    for j in range(rot // 2):
        a, b = (2 * j, 2 * j + 1) if inter else (j, j + rot // 2)
        cos, sin = (table[at, i].to(torch.float64)[:, None] for i in (j, j + rot // 2))
        u, w = x[..., a].to(torch.float64), x[..., b].to(torch.float64)
        y[..., a], y[..., b] = u * cos - w * sin, w * cos + u * sin
    return y


def _exact_rows(s, b, n):
    """Keys and values [n, H, D] of sequence b in 64 bits, nibble by nibble."""
    c, cache = s["case"], s["cache"]
    H, D, g, page = c["H"], c["D"], c["g"], c["page"]
    pages = s["table"][b, :-(-n // page)].long()
    kw, vw = cache["k"][pages].long(), cache["v"][pages].long()               # [P, H, page, D/8]
    k, v = (torch.empty((pages.numel(), H, page, D), dtype=torch.float64, device=kw.device) for _ in range(2))
    word = torch.arange(D // 8, device=kw.device)
    vword = torch.arange(page * D // 8, device=kw.device)
    block, r = vword // (4 * D), vword % (4 * D)
    u, q, m, j = r // 256, r // 64 % 4, r // 4 % 16, r % 4
    for nib in range(8):
        a, bb, hi = nib // 4, nib // 2 % 2, nib % 2
        i, lo = word % (D // 32) // 2, word % 2
        k[..., 32 * (i + hi * D // 64) + 8 * (word // (D // 32)) + 4 * lo + 2 * bb + a] = \
            (kw >> (4 * nib) & 15).to(torch.float64)
        v[:, :, block * 32 + 16 * hi + 4 * q + 2 * bb + a, 64 * u + 16 * j + m] = \
            (vw.flatten(2) >> (4 * nib) & 15).to(torch.float64)
    for x, name in ((k, "k_sz"), (v, "v_sz")):
        for i in range(D // g):
            sz = cache[name][pages][:, :, i].to(torch.float64)
            x[..., i * g:(i + 1) * g] = x[..., i * g:(i + 1) * g] * sz[..., 0, None] + sz[..., 1, None]
    return tuple(x.transpose(1, 2).flatten(0, 1)[:n] for x in (k, v))


def _exact_attend(s):
    c = s["case"]
    off, lens = s["off"].tolist(), s["lens"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    R, H = c["R"], c["H"]
    for b, n in enumerate(lens):
        k, v = _exact_rows(s, b, n)
        q = s["q"][off[b]:off[b + 1]].to(torch.float64)
        pos = torch.arange(n - q.shape[0], n, device="cuda")[:, None]
        t = torch.arange(n, device="cuda")
        hidden = t > pos
        if c["window"]:
            hidden |= (t <= pos - c["window"]) & (t >= c["sinks"])
        for h in range(H):
            for r in range(R):
                x = (q[:, h * R + r] @ k[:, h].t() * s["scale"]).masked_fill(hidden, -math.inf)
                out[off[b]:off[b + 1], h * R + r] = torch.softmax(x, 1) @ v[:, h]
    return out


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "lora":
        y = s["y"].to(torch.float64)
        for e in range(c["L"]):
            mine = (s["ids"] == e).nonzero()[:, 0]
            h = s["x"][mine].to(torch.float64) @ s["a"][e].to(torch.float64).t()
            y[mine] += s["scaling"][e].to(torch.float64) * (h @ s["b"][e].to(torch.float64).t())
        return y
    if c["op"] == "attend":
        return _exact_attend(s)
    if c["op"] == "read":
        rows = [_exact_rows(s, b, n) for b, n in enumerate(s["lens"].tolist())]
        return torch.cat([r[0] for r in rows]), torch.cat([r[1] for r in rows])
    off, lens = s["off"].tolist(), s["lens"].tolist()
    at = torch.cat([torch.arange(n - off[b + 1] + off[b], n, device="cuda") for b, n in enumerate(lens)])
    at = s["positions"].long() if s["positions"] is not None else at
    q, k = (_exact_rotated(x, s["cos_sin"], at, c["rot"], c["inter"]) for x in (s["q"], s["k"]))
    return q, _exact_group(k, c["g"]), _exact_group(s["v"].to(torch.float64), c["g"])
