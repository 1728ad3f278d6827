"""Groups of the 4-bit cache that are no numbers, in blocks that all rows see and in blocks
that some do: a value group makes its own channels of the rows that see it no numbers and
no others, a key group all channels of those rows."""
import math

import pytest
import torch

import int4_weight_only_uint32_amd as qg
from tests.gpu_util import note
from tests.kv4_util import attend, batch, random_cache, rng, to_gpu

pytestmark = pytest.mark.gpu

HALF = {"fp16": torch.float16, "bf16": torch.bfloat16}

CASES = [
    # D, g, R, len, new rows, hints of the rows
    (64, 64, 4, 200, 1, (1, 100)), (64, 32, 3, 200, 1, (1, 100)), (128, 128, 2, 200, 1, (1, 100)),
    (128, 64, 5, 200, 1, (1, 100)), (128, 32, 4, 200, 1, (1, 100)), (256, 128, 2, 200, 1, (1, 100)),
    (256, 64, 2, 200, 1, (1, 100)), (256, 32, 2, 200, 1, (1, 100)),
    # many rows, the first of which come before the token
    (64, 64, 4, 200, 195, (195, 1)), (64, 32, 2, 200, 195, (195, 1)), (128, 64, 2, 200, 195, (195, 1)),
    (128, 32, 1, 200, 195, (195, 1)), (256, 64, 1, 200, 195, (195, 1)), (256, 32, 1, 200, 195, (195, 1)),
    # parts along the tokens, which meet in a second kernel
    (128, 64, 2, 2500, 1, (1, 100)), (256, 32, 1, 2500, 1, (1, 100)),
]


def _run(q, c, lens, off, table, max_new, **kw):
    return qg.kv4_attend(q.cuda(), to_gpu(c), lens.cuda(), table.cuda(), seq_offsets=off.cuda(), max_new=max_new, **kw)


@pytest.mark.parametrize("D,g,R,n,new,hints", CASES)
def test_value_group_spoils_its_own_channels_only(D, g, R, n, new, hints):
    """Token 10: in a block that every row behind token 31 sees entirely.  The other channels are
    held to the tolerance of a cache whose group there is a number."""
    rnd, gen = rng(D + g + n + new)
    dtype = "fp16" if g == 64 else "bf16"
    lens, off, table, pages = batch(rnd, [n], [new], 64)
    c = random_cache(gen, pages, 1, D, 64, g)
    q = torch.randn((new, R, D), generator=gen).to(HALF[dtype])
    ref, tol = attend(q, c, lens, off, table, D ** -0.5)
    sees = torch.arange(n - new, n) >= 10
    for group in {0, D // g - 1}:
        bad = qg.KV4Cache(c.k, c.v, c.k_sz, c.v_sz.clone())
        bad.v_sz[int(table[0, 0]), 0, group, 10] = math.nan
        own = torch.zeros(D, dtype=torch.bool)
        own[group * g:(group + 1) * g] = True
        for hint in hints:
            note(f"value group {group} D={D} g={g} R={R} n={n} new={new} max_new={hint}")
            out = _run(q, bad, lens, off, table, hint).cpu()
            assert bool(torch.isnan(out[sees][..., own]).all())
            err = (out.double() - ref).abs()
            assert bool((err <= tol)[..., ~own].all()) and bool((err <= tol)[~sees].all())


@pytest.mark.parametrize("D,g,R,n,new,hints", CASES)
def test_key_group_spoils_the_rows_that_see_it(D, g, R, n, new, hints):
    rnd, gen = rng(D + g + n + new + 1)
    lens, off, table, pages = batch(rnd, [n], [new], 64)
    c = random_cache(gen, pages, 1, D, 64, g)
    q = torch.randn((new, R, D), generator=gen).half()
    ref, tol = attend(q, c, lens, off, table, D ** -0.5)
    c.k_sz[int(table[0, 0]), 0, D // g - 1, 10] = math.nan
    sees = torch.arange(n - new, n) >= 10
    for hint in hints:
        note(f"key group D={D} g={g} R={R} n={n} new={new} max_new={hint}")
        out = _run(q, c, lens, off, table, hint).cpu()
        assert bool(torch.isnan(out[sees]).all())
        assert bool(((out.double() - ref).abs() <= tol)[~sees].all())


def test_appended_values_past_fp16():
    """The way such a group comes about: a bf16 value past 65504, appended and attended to."""
    rnd, gen = rng(31)
    lens, off, table, pages = batch(rnd, [300], [300], 64)
    k, v = (torch.randn((300, 2, 128), generator=gen).bfloat16() for _ in range(2))
    v[7, 1, 70] = 7e4
    cache = qg.kv4_cache(pages, 2, 128, 64, 64)
    qg.kv4_append(cache, k.cuda(), v.cuda(), lens.cuda(), table.cuda(), seq_offsets=off.cuda())
    q = torch.randn((1, 6, 128), generator=gen).bfloat16()
    for hint in (1, 100):
        out = qg.kv4_attend(q.cuda(), cache, lens.cuda(), table.cuda(), seq_offsets=torch.tensor([0, 1]).int().cuda(),
                            max_new=hint).cpu()
        nan = torch.isnan(out)
        assert bool(nan[0, 3:, 64:].all()) and int(nan.sum()) == 3 * 64


@pytest.mark.parametrize("D,g,n", [(128, 64, 6000), (64, 64, 2500), (256, 32, 2500), (128, 64, 700)])
def test_a_weight_of_nothing_does_not_hide_it(D, g, n):
    """A seen group is no number however small its weight is: here 2^-400 and less of another
    part's, beside which it comes to 0 in 32 bits."""
    rnd, gen = rng(D + n)
    lens, off, table, pages = batch(rnd, [n], [1], 64)
    c = random_cache(gen, pages, 1, D, 64, g, spread=0.01)
    p, t = int(table[0, (n - 10) // 64]), (n - 10) % 64
    c.k_sz[p, 0, :, t] = torch.tensor([0.0, 8.0]).half()
    q = torch.ones((1, 2, D), dtype=torch.float16)
    ref, tol = attend(q, c, lens, off, table, 0.6)
    bad = qg.KV4Cache(c.k, c.v, c.k_sz, c.v_sz.clone())
    bad.v_sz[int(table[0, 0]), 0, 0, 5] = math.nan
    for hint in (1, 100):
        note(f"no weight D={D} g={g} n={n} max_new={hint}")
        clean = _run(q, c, lens, off, table, hint, scale=0.6).cpu()
        assert bool(((clean.double() - ref).abs() <= tol).all())
        out = _run(q, bad, lens, off, table, hint, scale=0.6).cpu()
        assert bool(torch.isnan(out[..., :g]).all()) and torch.equal(out[..., g:], clean[..., g:])
