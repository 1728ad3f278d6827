"""The paged 4-bit cache on the GPU: rows appended bit for bit as the formulas make them,
rows read back, attention against 64 bits (tolerances: kv4_util.attend), at the lengths,
masks and page tables where it can go wrong, and a layer's run of the calls."""
import math

import pytest
import torch

import int4_weight_only_uint32_amd as qg
from tests.gpu_util import note
from tests.kv4_util import angles, attend, batch, quantized, random_cache, rng, rotated, rows_of, store, to_gpu, values_of

pytestmark = pytest.mark.gpu

HALF = {"fp16": torch.float16, "bf16": torch.bfloat16}


def _same_cache(got, want):
    for n in ("k", "v", "k_sz", "v_sz"):
        a, b = getattr(got, n).cpu(), getattr(want, n)
        a, b = (a, b) if a.dtype == torch.int32 else (a.view(torch.int16), b.view(torch.int16))
        assert torch.equal(a, b), (n, (a != b).nonzero()[:4].tolist())


def _rows(gen, T, heads, D, dtype, scale=1.0):
    x = torch.randn((T, heads, D), generator=gen) * scale
    return (x * torch.where(torch.rand(D, generator=gen) < 0.05, 6.0, 1.0)).to(dtype)


APPEND = [
    # D, g, page, H, q heads, lens, news, rot, interleaved, type
    (128, 64, 64, 2, 6, [1], [1], 128, False, "fp16"),
    (128, 32, 32, 1, 4, [33], [1], 128, True, "bf16"),
    (128, 128, 64, 3, 3, [70, 1, 200, 64, 65], [70, 1, 37, 64, 2], 64, False, "fp16"),
    (64, 32, 32, 2, 16, [31, 32, 33, 95], [31, 1, 32, 64], 64, True, "bf16"),
    (64, 64, 128, 1, 1, [129, 300], [9, 300], 32, False, "fp16"),
    (256, 64, 256, 1, 10, [257, 5], [100, 5], 256, False, "bf16"),
    (256, 128, 64, 2, 2, [40, 41, 42], [3, 2, 1], 128, True, "fp16"),
    (256, 32, 1024, 1, 9, [1025], [60], 0, False, "bf16"),
]


@pytest.mark.parametrize("D,g,page,H,Hq,lens,news,rot,inter,dtype", APPEND)
def test_append_is_bit_exact(D, g, page, H, Hq, lens, news, rot, inter, dtype):
    rnd, gen = rng(D + g + page)
    note(f"append D={D} g={g} page={page} H={H} lens={lens} news={news} rot={rot} {inter} {dtype}")
    lens_t, off, table, pages = batch(rnd, lens, news, page)
    T, dt = int(off[-1]), HALF[dtype]
    want = random_cache(gen, pages, H, D, page, g)
    got = to_gpu(want)
    # parts of one wider tensor, as a projection leaves them
    qkv = torch.cat([_rows(gen, T, n, D, dt).flatten(1) for n in (Hq, H, H)], 1)
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([Hq * D, H * D, H * D], 1))
    dev = [t.unflatten(1, (-1, D)) for t in qkv.cuda().split([Hq * D, H * D, H * D], 1)]
    cs = angles(max(lens) + 1, rot) if rot else None
    at = torch.cat([torch.arange(n - m, n) for n, m in zip(lens, news)])
    out = qg.kv4_append(got, dev[1], dev[2], lens_t.cuda(), table.cuda(), seq_offsets=off.cuda(),
                        cos_sin=cs.cuda() if rot else None, interleaved=inter, q=dev[0])
    torch.cuda.synchronize()
    store(want, rotated(k, cs, at, inter), v.float(), lens_t, off, table)
    _same_cache(got, want)
    assert torch.equal(out.cpu(), rotated(q, cs, at, inter).to(dt))


def test_append_without_offsets_positions_and_far_angles():
    """One row a sequence; positions of their own, those without angles NaN."""
    rnd, gen = rng(3)
    lens_t, off, table, pages = batch(rnd, [5, 64, 100], [1, 1, 1], 64)
    want = random_cache(gen, pages, 2, 128, 64, 64)
    got = to_gpu(want)
    k, v, q = (_rows(gen, 3, n, 128, torch.float16) for n in (2, 2, 4))
    cs = angles(50, 64)
    at = torch.tensor([49, 50, -1], dtype=torch.int32)
    q_out = torch.empty((3, 4, 128), dtype=torch.float16, device="cuda")
    got_q = qg.kv4_append(got, k.cuda(), v.cuda(), lens_t.cuda(), table.cuda(), positions=at.cuda(), cos_sin=cs.cuda(),
                          q=q.cuda(), q_out=q_out)
    assert got_q is q_out
    store(want, rotated(k, cs, at, False), v.float(), lens_t, off, table)
    _same_cache(got, want)
    ref = rotated(q, cs, at, False).half()
    assert torch.equal(torch.isnan(q_out.cpu()), torch.isnan(ref)) and bool(torch.isnan(ref).any())
    assert torch.equal(q_out.cpu().nan_to_num(7.0), ref.nan_to_num(7.0))
    assert qg.kv4_append(got, k.cuda(), v.cuda(), lens_t.cuda(), table.cuda()) is None


def test_append_keeps_what_has_no_place():
    """Pages outside the cache, tokens past the table, more rows than tokens, empty sequences, rows
    behind the last sequence: nothing of the cache or of q_out but what belongs there changes."""
    rnd, gen = rng(4)
    lens_t = torch.tensor([70, 3, 0, 200, 64, -5], dtype=torch.int32)
    off = torch.tensor([2, 42, 47, 50, 60, 60, 62], dtype=torch.int32)
    table = torch.tensor([[0, -1], [1, 0], [2, 2], [2, 3], [9, 9], [3, 3]], dtype=torch.int32)
    table[0, 1] = 1 << 30
    T = 66
    want = random_cache(gen, 5, 2, 128, 64, 32)
    got = to_gpu(want)
    k, v, q = (_rows(gen, T, n, 128, torch.bfloat16) for n in (2, 2, 5))
    cs = angles(300, 128)
    q_out = torch.full((T, 5, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    qg.kv4_append(got, k.cuda(), v.cuda(), lens_t.cuda(), table.cuda(), seq_offsets=off.cuda(), cos_sin=cs.cuda(),
                  q=q.cuda(), q_out=q_out)
    at = torch.full((T,), -1)
    for b in range(6):
        n = int(off[b + 1] - off[b])
        at[int(off[b]):int(off[b + 1])] = max(int(lens_t[b]), 0) - n + torch.arange(n)
    store(want, rotated(k, cs, at, False), v.float(), lens_t.clamp_min(0), off, table)
    _same_cache(got, want)
    ref = rotated(q, cs, at, False).bfloat16()
    o = q_out.cpu()
    assert bool((o[:2] == 3.0).all()) and bool((o[62:] == 3.0).all())
    assert torch.equal(o[2:62].nan_to_num(7.0), ref[2:62].nan_to_num(7.0))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_append_odd_groups(dtype):
    """Constant groups, zeros of both signs, subnormal ranges, NaN, infinities and values past fp16."""
    dt = HALF[dtype]
    gen = torch.Generator().manual_seed(5)
    x = torch.randn((8, 1, 128), generator=gen).to(dt)
    x[0] = 0.0
    x[1, 0, :64] = -0.0
    x[1, 0, 64:] = 3.25
    x[2] *= 1e-6
    x[3, 0, 5] = math.nan
    x[4, 0, 70] = math.inf
    x[5, 0, 3] = -math.inf
    x[6, 0, 9] = 65504.0
    x[6, 0, 10] = -65504.0
    x[6, 0, 80] = 1e5 if dtype == "bf16" else 60000.0
    x[7, 0, 64:] = torch.arange(64) / 64.0
    lens, off, table = torch.tensor([8], dtype=torch.int32), torch.tensor([0, 8], dtype=torch.int32), torch.zeros(
        (1, 1), dtype=torch.int32)
    want = qg.kv4_cache(1, 1, 128, 32, 64, device="cpu")
    got = to_gpu(want)
    qg.kv4_append(got, x.cuda(), x.cuda(), lens.cuda(), table.cuda(), seq_offsets=off.cuda())
    store(want, x.float(), x.float(), lens, off, table)
    for n in ("k", "v"):
        assert torch.equal(getattr(got, n).cpu(), getattr(want, n))
    for n in ("k_sz", "v_sz"):
        a, b = getattr(got, n).cpu(), getattr(want, n)
        assert torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(9.0), b.nan_to_num(9.0))
    assert bool(torch.isnan(quantized(x.float(), 64)[1]).any())


@pytest.mark.parametrize("D,g,page,H,lens,news,dtype", [
    (128, 64, 64, 2, [1], [1], torch.float32), (128, 32, 32, 3, [33, 200], [33, 77], torch.float16),
    (64, 64, 128, 1, [300, 31], [300, 31], torch.bfloat16), (256, 128, 64, 2, [65, 64], [2, 64], torch.float16),
    (64, 32, 32, 1, [70], [70], torch.float32), (256, 32, 1024, 1, [1100], [90], torch.bfloat16),
    (128, 128, 256, 1, [500], [257], torch.float32),
])
def test_read(D, g, page, H, lens, news, dtype):
    """fp32: the sum rounded once (the product of a code and a scale is exact); 16 bits: rounded
    from that."""
    rnd, gen = rng(D + page)
    note(f"read D={D} g={g} page={page} lens={lens} news={news} {dtype}")
    lens_t, off, table, pages = batch(rnd, lens, news, page)
    c = random_cache(gen, pages, H, D, page, g)
    k, v = qg.kv4_read(to_gpu(c), lens_t.cuda(), table.cuda(), seq_offsets=off.cuda(), rows=int(off[-1]), dtype=dtype)
    for got, all_rows in zip((k, v), values_of(c)):
        ref = torch.cat([rows_of(all_rows, table, b, n, page)[0][n - m:] for b, (n, m) in enumerate(zip(lens, news))])
        assert torch.equal(got.cpu(), ref.float().to(dtype))


def test_read_without_place_and_rows_behind():
    rnd, gen = rng(6)
    lens_t, _, table, pages = batch(rnd, [100, 40], [0, 0], 32)
    table[0, 1] = 77
    off = torch.tensor([1, 101, 145], dtype=torch.int32)
    c = random_cache(gen, pages, 2, 64, 32, 32)
    outs = [torch.full((150, 2, 64), 5.0, device="cuda") for _ in range(2)]
    qg.kv4_read(to_gpu(c), lens_t.cuda(), table.cuda(), seq_offsets=off.cuda(), k_out=outs[0], v_out=outs[1])
    for got, all_rows in zip(outs, values_of(c)):
        got = got.cpu()
        assert bool((got[:1] == 5.0).all()) and bool((got[145:] == 5.0).all())
        assert torch.equal(got[1:101], rows_of(all_rows, table, 0, 100, 32)[0].float())
        assert not bool(got[33:65].any())
        assert not bool(got[101:105].any())                       # 44 rows of 40 tokens: the first four have none
        assert torch.equal(got[105:145], rows_of(all_rows, table, 1, 40, 32)[0].float())


def _check(q, c, lens, off, table, window=0, sinks=0, scale=None, max_new=None, offsets=True, **kw):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    out = qg.kv4_attend(q.cuda(), to_gpu(c), lens.cuda(), table.cuda(), seq_offsets=off.cuda() if offsets else None,
                        max_new=max_new, scale=scale, window=window, sinks=sinks, **kw)
    torch.cuda.synchronize()
    ref, tol = attend(q, c, lens, off, table, scale, window, sinks)
    err = (out.cpu().double() - ref).abs()
    assert torch.isfinite(out).all()
    assert bool((err <= tol).all()), (float((err / tol).max()), (err > tol).nonzero()[:5].tolist())
    return out


ATTEND = [
    # D, g, page, H, R, lens, news, window, sinks, type
    (128, 64, 64, 2, 5, [1], [1], 0, 0, "fp16"),
    (128, 64, 64, 1, 1, [31, 32, 33], [1, 1, 1], 0, 0, "bf16"),
    (128, 128, 32, 1, 16, [700, 129, 1, 64], [1, 1, 1, 1], 0, 0, "fp16"),
    (128, 32, 128, 2, 4, [515, 260], [1, 1], 0, 0, "bf16"),
    (64, 32, 32, 2, 7, [333, 65], [1, 1], 0, 0, "fp16"),
    (64, 64, 64, 1, 8, [90, 1000], [2, 1], 0, 0, "bf16"),
    (256, 64, 64, 1, 3, [200, 31], [1, 1], 0, 0, "fp16"),
    (256, 128, 32, 1, 2, [150], [5], 0, 0, "bf16"),
    (256, 32, 256, 1, 1, [300], [1], 0, 0, "fp16"),
    # more rows of a head than a workgroup shares: several tokens, wide groups of heads
    (128, 64, 64, 1, 17, [100], [1], 0, 0, "fp16"),
    (128, 64, 32, 2, 5, [170, 40, 3], [130, 40, 2], 0, 0, "bf16"),
    (128, 128, 64, 1, 3, [300], [200], 0, 0, "fp16"),
    (128, 32, 64, 1, 2, [100, 100], [33, 64], 0, 0, "bf16"),
    (64, 32, 64, 1, 4, [260, 70], [90, 70], 0, 0, "fp16"),
    (64, 64, 32, 2, 1, [200], [129], 0, 0, "bf16"),
    (256, 64, 64, 1, 2, [150, 40], [70, 40], 0, 0, "fp16"),
    (256, 128, 64, 1, 1, [100], [65], 0, 0, "bf16"),
    (256, 32, 32, 1, 4, [90], [20], 0, 0, "fp16"),
    # windows and first tokens
    (128, 64, 64, 2, 5, [500, 30, 100], [1, 1, 1], 64, 4, "bf16"),
    (128, 64, 32, 1, 4, [700], [1], 1, 0, "fp16"),
    (128, 64, 32, 1, 4, [700], [1], 1, 1, "fp16"),
    (128, 64, 64, 1, 4, [700], [1], 100, 40, "bf16"),
    (128, 64, 64, 1, 4, [700], [1], 33, 680, "bf16"),
    (128, 32, 64, 1, 2, [400, 90], [150, 90], 50, 3, "fp16"),
    (64, 32, 32, 1, 3, [400], [150], 32, 33, "bf16"),
    (256, 64, 32, 1, 1, [300], [150], 7, 5, "fp16"),
]


@pytest.mark.parametrize("D,g,page,H,R,lens,news,window,sinks,dtype", ATTEND)
def test_attend(D, g, page, H, R, lens, news, window, sinks, dtype):
    rnd, gen = rng(D + g + page + len(lens) + lens[0])
    note(f"attend D={D} g={g} page={page} H={H} R={R} lens={lens} news={news} window={window} sinks={sinks} {dtype}")
    lens_t, off, table, pages = batch(rnd, lens, news, page)
    c = random_cache(gen, pages, H, D, page, g)
    q = _rows(gen, int(off[-1]), H * R, D, HALF[dtype])
    out = _check(q, c, lens_t, off, table, window, sinks, max_new=max(news))
    # a wrong hint of the rows picks another kernel, not another result: within twice the tolerance
    _check(q, c, lens_t, off, table, window, sinks, max_new=1 if max(news) > 1 else 100)
    if all(n == 1 for n in news):
        same = qg.kv4_attend(q.cuda(), to_gpu(c), lens_t.cuda(), table.cuda(), window=window, sinks=sinks)
        assert torch.equal(same, out)


def test_attend_rows_that_see_nothing():
    """Empty sequences, more rows than tokens, pages that are none: zeros; rows of no sequence stay."""
    rnd, gen = rng(8)
    lens_t = torch.tensor([0, 3, 40, 64, -7], dtype=torch.int32)
    off = torch.tensor([1, 3, 9, 10, 12, 13], dtype=torch.int32)
    table = torch.tensor([[0, 1], [1, -1], [-1, 2], [99, 3], [0, 0]], dtype=torch.int32)
    c = random_cache(gen, 5, 2, 128, 32, 64)
    q = _rows(gen, 15, 6, 128, torch.bfloat16)
    out = torch.full((15, 6, 128), 2.0, dtype=torch.bfloat16, device="cuda")
    for max_new in (1, 6):
        out.fill_(2.0)
        qg.kv4_attend(q.cuda(), to_gpu(c), lens_t.cuda(), table.cuda(), seq_offsets=off.cuda(), max_new=max_new, out=out)
        ref, tol = attend(q, c, lens_t, off, table, 128 ** -0.5)
        got = out.cpu().double()
        assert bool((got[:1] == 2.0).all()) and bool((got[13:] == 2.0).all())
        assert not bool(got[1:6].any()) and not bool(got[12].any())
        assert bool(((got - ref).abs() <= tol)[1:13].all())


@pytest.mark.parametrize("max_new", [1, 50])
def test_attend_ignores_what_is_not_seen(max_new):
    """NaN scales and zeros of tokens behind the sequence, outside the window or on other pages."""
    rnd, gen = rng(9)
    lens_t, off, table, pages = batch(rnd, [75], [2], 64)
    c = random_cache(gen, pages, 1, 128, 64, 64)
    hidden = to_gpu(c)
    seen = torch.zeros((pages, 64), dtype=torch.bool)
    for t in list(range(3)) + list(range(75 - 2 - 20 + 1, 75)):
        seen[int(table[0, t // 64]), t % 64] = True
    for sz in (hidden.k_sz, hidden.v_sz):
        sz.masked_fill_(~seen[:, None, None, :, None].cuda(), math.nan)
    q = _rows(gen, 2, 4, 128, torch.float16)
    want = qg.kv4_attend(q.cuda(), to_gpu(c), lens_t.cuda(), table.cuda(), seq_offsets=off.cuda(), window=20, sinks=3,
                         max_new=max_new)
    got = qg.kv4_attend(q.cuda(), hidden, lens_t.cuda(), table.cuda(), seq_offsets=off.cuda(), window=20, sinks=3,
                        max_new=max_new)
    assert bool(torch.isfinite(got).all()) and torch.equal(got, want)
    # what is seen and no number makes the rows that see it none
    p, s = int(table[0, 1]), 74 % 64
    hidden.v_sz[p, 0, 0, s] = math.nan
    got = qg.kv4_attend(q.cuda(), hidden, lens_t.cuda(), table.cuda(), seq_offsets=off.cuda(), window=20, sinks=3,
                        max_new=max_new)
    assert bool(torch.isnan(got[1, :, :64]).all()) and torch.equal(got[0], want[0])
    assert torch.equal(got[1, :, 64:], want[1, :, 64:])


@pytest.mark.parametrize("dtype,size", [("bf16", 1e-30), ("bf16", 1e20), ("fp16", 6e-8), ("fp16", 1.0), ("bf16", 0.0)])
def test_attend_query_sizes(dtype, size):
    """Tiny, large and zero queries (with a scale that brings the scores back into range)."""
    rnd, gen = rng(10)
    lens_t, off, table, pages = batch(rnd, [100], [3], 64)
    c = random_cache(gen, pages, 1, 128, 64, 64)
    q = (torch.randn((3, 4, 128), generator=gen) * size).to(HALF[dtype])
    _check(q, c, lens_t, off, table, scale=128 ** -0.5 / size if size else 0.1, max_new=3)


def test_attend_infinite_queries_are_no_numbers():
    rnd, gen = rng(11)
    lens_t, off, table, pages = batch(rnd, [100, 50], [1, 1], 64)
    c = random_cache(gen, pages, 1, 128, 64, 64)
    for bad in (math.inf, -math.inf, math.nan):
        q = _rows(gen, 2, 3, 128, torch.float16)
        q[0, 1, 17] = bad
        for max_new in (1, 40):
            out = qg.kv4_attend(q.cuda(), to_gpu(c), lens_t.cuda(), table.cuda(), seq_offsets=off.cuda(), max_new=max_new)
            nan = torch.isnan(out).cpu()
            assert bool(nan[0, 1].all()) and int(nan.sum()) == 128


def test_attend_sharp_and_flat_scores():
    """A running maximum that rises all along, falls all along, or stays."""
    rnd, gen = rng(12)
    lens_t, off, table, pages = batch(rnd, [600], [1], 64)
    for order in (1.0, -1.0, 0.0):
        c = random_cache(gen, pages, 1, 128, 64, 64)
        for t in range(600):
            c.k_sz[int(table[0, t // 64]), 0, :, t % 64, 1] = order * t * 0.01
            c.k_sz[int(table[0, t // 64]), 0, :, t % 64, 0] = 0.02
        q = torch.ones((1, 4, 128), dtype=torch.float16)
        _check(q, c, lens_t, off, table, scale=0.3)
        _check(q, c, lens_t, off, table, scale=0.3, max_new=64)


def test_attend_long_split_and_repeatable():
    """A long context over many workgroups, bit for bit the same again, also beside itself on
    two streams; strided queries."""
    rnd, gen = rng(13)
    lens_t, off, table, pages = batch(rnd, [9001, 1, 4500], [1, 1, 1], 64)
    c = random_cache(gen, pages, 2, 128, 64, 64)
    wide = _rows(gen, 3, 14, 128, torch.bfloat16)
    q = wide[:, 2:12]
    out = _check(q, c, lens_t, off, table)
    g, args = to_gpu(c), (lens_t.cuda(), table.cuda())
    qd = wide.cuda()[:, 2:12]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            outs.append(qg.kv4_attend(qd, g, *args, seq_offsets=off.cuda()))
    torch.cuda.synchronize()
    assert all(torch.equal(o, out) for o in outs)


def test_pages_past_32_bits():
    """A cache whose codes need more than 2^32 bytes and more than 2^31 words of offsets."""
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("not enough memory")
    pages, H, page, D, g = 36000, 8, 256, 128, 128
    assert pages * H * page * (D // 8) * 4 > 2**32 and pages * H * page * D // 2 > 2**32
    gen = torch.Generator().manual_seed(14)
    cache = qg.kv4_cache(pages, H, D, page, g)
    table = torch.tensor([[pages - 1, 3, pages - 2]], dtype=torch.int32)
    lens, off = torch.tensor([600], dtype=torch.int32), torch.tensor([0, 600], dtype=torch.int32)
    k, v = (_rows(gen, 600, H, D, torch.bfloat16) for _ in range(2))
    qg.kv4_append(cache, k.cuda(), v.cuda(), lens.cuda(), table.cuda(), seq_offsets=off.cuda())
    small = qg.kv4_cache(3, H, D, page, g, device="cpu")
    moved = torch.tensor([[0, 1, 2]], dtype=torch.int32)
    store(small, k.float(), v.float(), lens, off, moved)
    for n in ("k", "v", "k_sz", "v_sz"):
        assert torch.equal(getattr(cache, n)[table[0].long().cuda()].cpu(), getattr(small, n)), n
    q = _rows(gen, 1, H * 2, D, torch.bfloat16)
    got = qg.kv4_attend(q.cuda(), cache, lens.cuda(), table.cuda())
    want = qg.kv4_attend(q.cuda(), to_gpu(small), lens.cuda(), moved.cuda())
    assert torch.equal(got, want)
    a = qg.kv4_read(cache, lens.cuda(), table.cuda(), seq_offsets=off.cuda(), rows=600)
    b = qg.kv4_read(to_gpu(small), lens.cuda(), moved.cuda(), seq_offsets=off.cuda(), rows=600)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("H,R,D,g,dtype", [(2, 3, 64, 64, "bf16"), (1, 8, 128, 32, "fp16")])
def test_attend_parts_of_many_ragged_sequences(H, R, D, g, dtype):
    """More sequences than lanes, one far longer than the others, some empty: parts of one size."""
    rnd, gen = rng(11)
    lens = [rnd.choice((0, 1, 5, 33, 64, 70)) for _ in range(100)]
    lens[70], lens[3] = 5000, 900
    note(f"attend parts H={H} R={R} D={D} g={g} {dtype}")
    lens_t, off, table, pages = batch(rnd, lens, [1] * 100, 64)
    c = random_cache(gen, pages, H, D, 64, g)
    q = _rows(gen, 100, H * R, D, HALF[dtype])
    out = _check(q, c, lens_t, off, table, max_new=1)
    for _ in range(3):
        again = qg.kv4_attend(q.cuda(), to_gpu(c), lens_t.cuda(), table.cuda())
        assert torch.equal(again, out)


@pytest.mark.parametrize("D,g,R,lens,news", [(128, 64, 5, [1500, 300], [1, 1]), (128, 32, 4, [300], [100]),
                                             (64, 64, 8, [2500], [1]), (256, 32, 2, [400], [1])])
def test_attend_scales_of_all_sizes(D, g, R, lens, news):
    """Scales from 1e-4 to 3000 and constant groups, the large ones late: the reference of p moves."""
    rnd, gen = rng(12 + D + g)
    note(f"attend scales D={D} g={g} R={R} lens={lens} news={news}")
    lens_t, off, table, pages = batch(rnd, lens, news, 64)
    c = random_cache(gen, pages, 1, D, 64, g)
    for b, n in enumerate(lens):
        for i in range(-(-n // 64)):
            p = int(table[b, i])
            size = (1e-4, 0.02, 1.0, 0.0, 40.0, 3000.0)[min(5, 6 * i * 64 // n)]
            s = (size * (0.5 + 0.5 * torch.rand(c.v_sz[p, ..., 0].shape, generator=gen))).half()
            c.v_sz[p, ..., 0], c.v_sz[p, ..., 1] = s, (-7.5 * s.float()).half()
    q = _rows(gen, int(off[-1]), R, D, torch.float16)
    _check(q, c, lens_t, off, table, max_new=max(news))
    _check(q, c, lens_t, off, table, max_new=max(news), window=200, sinks=3)


@pytest.mark.parametrize("D,g", [(64, 64), (128, 128), (256, 128)])
def test_attend_largest_query_sums(D, g):
    """Queries whose channels are all the largest of a power of two: 64 times their sum is the largest binary16."""
    rnd, gen = rng(13 + D)
    lens_t, off, table, pages = batch(rnd, [100], [1], 64)
    c = random_cache(gen, pages, 1, D, 64, g)
    q = torch.full((1, 2, D), 2047 / 2048, dtype=torch.float16)
    q[:, 1] = -q[:, 1]
    _check(q, c, lens_t, off, table, max_new=1, scale=1e-3)
