"""Plain forms of the paged 4-bit cache for the tests: its layout by the header's
formulas, word by word, and attention in 64 bits."""
import math
import random

import torch

import int4_weight_only_uint32_amd as qg


def key_place(d, D):
    """(word of the token, nibble) of a key's channel."""
    step, q, slot = d // 32, d // 8 % 4, d % 8
    c, i = divmod(step, D // 64)
    l, b, a = slot // 4, slot // 2 % 2, slot % 2
    return q * (D // 32) + 2 * i + l, 4 * a + 2 * b + c


def value_place(t, d, D):
    """(word of the 32-token block, nibble) of channel d of token t (0 .. 31)."""
    u, j, m = d // 64, d // 16 % 4, d % 16
    c, q, b, a = t // 16, t // 4 % 4, t // 2 % 2, t % 2
    return ((u * 4 + q) * 16 + m) * 4 + j, 4 * a + 2 * b + c


def codes_of(cache):
    """Codes of all keys and values, int64 [pages, heads, page_size, D], on the CPU."""
    D, page = cache.head_dim, cache.page_size
    kw, vw = cache.k.cpu().long(), cache.v.cpu().long()
    k, v = (torch.empty(kw.shape[:3] + (D,), dtype=torch.int64) for _ in range(2))
    for d in range(D):
        w, n = key_place(d, D)
        k[..., d] = kw[..., w] >> (4 * n) & 15
    flat = vw.flatten(2)
    for t in range(page):
        at = [value_place(t % 32, d, D) for d in range(D)]
        w = torch.tensor([x[0] for x in at]) + t // 32 * (32 * D // 8)
        v[:, :, t] = flat[..., w] >> (4 * torch.tensor([x[1] for x in at])) & 15
    return k, v


def values_of(cache, dtype=torch.float64):
    """What the cache stands for, [pages, heads, page_size, D]."""
    out = []
    for c, sz in zip(codes_of(cache), (cache.k_sz, cache.v_sz)):
        s = sz.cpu().to(dtype).transpose(2, 3)
        out.append((c.to(dtype).unflatten(-1, (-1, cache.group)) * s[..., :1] + s[..., 1:]).flatten(-2))
    return out


def random_cache(gen, pages, heads, D, page, g, spread=1.0):
    """A cache of random codes, with scales and zeros of normal values, a few of them large."""
    c = qg.kv4_cache(pages, heads, D, page, g, device="cpu")
    c.k.random_(-2**31, 2**31, generator=gen)
    c.v.random_(-2**31, 2**31, generator=gen)
    for sz in (c.k_sz, c.v_sz):
        s = (0.1 + 0.3 * torch.rand(sz.shape[:-1], generator=gen)) * spread
        sz[..., 0] = s.half()
        sz[..., 1] = (-7.5 * s + 0.3 * spread * torch.randn(s.shape, generator=gen)).half()
    return c


def to_gpu(c):
    return qg.KV4Cache(*(t.cuda() for t in (c.k, c.v, c.k_sz, c.v_sz)))


def batch(rnd, lens, news, page, spare=2, width=None):
    """(lens, offsets, table, pages): the sequences' pages in any order, unused entries -1."""
    counts = [-(-n // page) for n in lens]
    pages = sum(counts) + spare
    order = list(range(pages))
    rnd.shuffle(order)
    width = width or max(counts + [1])
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    off = [0]
    for n in news:
        off.append(off[-1] + n)
    return (torch.tensor(lens, dtype=torch.int32), torch.tensor(off, dtype=torch.int32), table, pages)


def rows_of(values, table, b, n, page):
    """Rows [n, heads, D] of a sequence, and whether each has a place."""
    H, D = values.shape[1], values.shape[3]
    out = torch.zeros((n, H, D), dtype=values.dtype)
    has = torch.zeros(n, dtype=torch.bool)
    for i in range(-(-n // page)):
        p = int(table[b, i]) if i < table.shape[1] else -1
        if 0 <= p < values.shape[0]:
            m = min(page, n - i * page)
            out[i * page:i * page + m] = values[p, :, :m].transpose(0, 1)
            has[i * page:i * page + m] = True
    return out, has


def attend(q, cache, lens, off, table, scale, window=0, sinks=0):
    """(out, tolerance) [T, q_heads, D] in 64 bits, of fp16 or bf16 q on the CPU.

    The tolerance adds up, for each value:
      * its rounding to q's type: half a step, eps / 2 of it;
      * with V = s c + z written as s (c - 8) + m, m = z + 8 s: p_t s_t rounded to fp16 (2^-11 of it,
        2^-25 where it is subnormal) against c - 8, and p_t rounded to fp16 against m and in
        its sum (the same again, of the sum of p |m| and of the value);
      * p_t in 32 bits: the score's sum of D products (2^-24 of their sizes for each of
        the D/32 + 8 additions in a row), its product with the scale, and 2^-22 for
        the exponential; the same for their sum;
      * the sum of a group's queries as two 16-bit values, and codes that enter as 64 + code: within
        2^-16 times 2 max |q| times |z| for each group (zeros are 7.5 scales and more here);
      * products and sums in 32 bits, 2^-20 of their sizes.
    """
    kd, vd = values_of(cache)
    vc = codes_of(cache)[1].double()
    page, H, D, g = cache.page_size, cache.heads, cache.head_dim, cache.group
    vs = cache.v_sz[..., 0].cpu().double().transpose(2, 3).repeat_interleave(g, -1)
    vz = cache.v_sz[..., 1].cpu().double().transpose(2, 3).repeat_interleave(g, -1)
    kz = cache.k_sz[..., 1].cpu().double().abs().amax(2)[..., None]      # [pages, heads, page, 1]: a token's largest
    codep, mid = (vc - 8).abs() * vs, (vz + 8 * vs).abs()
    R = q.shape[1] // H
    out = torch.zeros(q.shape, dtype=torch.float64)
    tol = torch.zeros(q.shape, dtype=torch.float64)
    half = torch.finfo(q.dtype).eps / 2
    for b in range(len(lens)):
        n, r0, r1 = int(lens[b]), int(off[b]), int(off[b + 1])
        if n <= 0:
            continue
        k, has = rows_of(kd, table, b, n, page)
        v, _ = rows_of(vd, table, b, n, page)
        c, _ = rows_of(codep, table, b, n, page)
        mm, _ = rows_of(mid, table, b, n, page)
        zz, _ = rows_of(kz, table, b, n, page)
        t = torch.arange(n)
        for i in range(r0, r1):
            pos = n - (r1 - r0) + (i - r0)
            seen = (t <= pos) & has
            if window:
                seen &= (t > pos - window) | (t < sinks)
            if not bool(seen.any()):
                continue
            for h in range(H):
                kk, vv, cc, md = k[seen, h], v[seen, h], c[seen, h], mm[seen, h]
                for r in range(R):
                    qq = q[i, h * R + r].double()
                    x = kk @ qq * scale
                    p = torch.softmax(x, 0)
                    o = p @ vv
                    out[i, h * R + r] = o
                    size = kk.abs() @ qq.abs() * scale
                    e = size.max() * (D / 32 + 8) * 2.0**-24 + x.abs().max() * 2.0**-23 + 2.0**-22
                    e = e + zz[seen, h].max() * 2 * qq.abs().max() * 2.0**-16 * (D // g) * scale
                    flat = 2.0**-25 * len(x) / torch.exp(x - x.max()).sum() * (8 + md.amax(0) + o.abs())
                    tol[i, h * R + r] = (half * o.abs() + 2.0**-11 * (p @ cc + p @ md + o.abs()) + flat +
                                         2 * e * (p @ vv.abs() + o.abs()) + 2.0**-20 * (p @ vv.abs()))
    return out, tol * 1.01 + 1e-30


def quantized(x, g):
    """(codes, scale and zero) of fp32 rows [..., D] by the header's formulas, on the CPU."""
    p = x.unflatten(-1, (-1, g))
    lo, hi = p.amin(-1, keepdim=True), p.amax(-1, keepdim=True)
    z = lo.half()
    bad = ~torch.isfinite(z) | ~torch.isfinite(hi.half())
    s = torch.where(bad, math.nan, ((hi - lo) / torch.full_like(lo, 15.0)).half().float()).half()
    q = torch.where(s > 0, torch.round((p - z.float()) / s.float()), 0.0).clamp(0, 15)
    z = torch.where(bad, math.nan, z.float()).half()
    return q.long().flatten(-2), torch.cat([s, z], -1)


def rotated(x, cos_sin, at, interleaved):
    """fp32 rows [T, heads, D] rotated by the header's formulas, on the CPU."""
    x = x.float().clone()
    if cos_sin is None:
        return x
    rot = cos_sin.shape[1]
    ok = (at >= 0) & (at < cos_sin.shape[0])
    row = cos_sin[torch.where(ok, at, 0).long()][:, None]
    c, s = row[..., :rot // 2], row[..., rot // 2:]
    ia = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    a, b = x[..., ia], x[..., ib]
    x[..., ia] = a * c - b * s
    x[..., ib] = b * c + a * s
    x[~ok, :, :rot] = math.nan
    return x


def angles(n, rot, base=1e4):
    at = torch.arange(n, dtype=torch.float64)[:, None]
    w = at * base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    return torch.cat([torch.cos(w), torch.sin(w)], 1).float()


def store(cache, k, v, lens, off, table):
    """What kv4_append of fp32 rows makes of a cache on the CPU (in place): each nibble by itself."""
    D, page, g = cache.head_dim, cache.page_size, cache.group
    kq, ksz = quantized(k, g)
    vq, vsz = quantized(v, g)
    kplace = [key_place(d, D) for d in range(D)]
    kw = torch.tensor([x[0] for x in kplace])
    for b in range(len(lens)):
        n, r0, r1 = int(lens[b]), int(off[b]), int(off[b + 1])
        for i in range(r0, r1):
            t = n - (r1 - r0) + (i - r0)
            if t < 0 or t // page >= table.shape[1]:
                continue
            p = int(table[b, t // page])
            if not 0 <= p < cache.pages:
                continue
            slot = t % page
            for h in range(cache.heads):
                words = torch.zeros(D // 8, dtype=torch.int64)
                words.index_add_(0, kw, kq[i, h] << (4 * torch.tensor([x[1] for x in kplace])))
                cache.k[p, h, slot] = words.to(torch.int32)
                vplace = [value_place(slot % 32, d, D) for d in range(D)]
                w = torch.tensor([x[0] for x in vplace]) + slot // 32 * (4 * D)
                nib = 4 * torch.tensor([x[1] for x in vplace])
                flat = cache.v[p, h].view(-1)
                old = flat[w].long() & 0xFFFFFFFF
                flat[w] = ((old & ~(15 << nib)) | (vq[i, h] << nib)).to(torch.int32)
                cache.k_sz[p, h, :, slot] = ksz[i, h]
                cache.v_sz[p, h, :, slot] = vsz[i, h]


def rng(seed):
    return random.Random(seed), torch.Generator().manual_seed(seed)
