"""The cache's layout by the header's formulas: every channel of every token has a nibble
of its own, and the plain forms of the tests write and read the same ones.  On the CPU."""
import pytest
import torch

import int4_weight_only_uint32_amd as qg
from tests.kv4_util import batch, codes_of, key_place, quantized, random_cache, rng, store, value_place, values_of


@pytest.mark.parametrize("D", [64, 128, 256])
def test_each_nibble_has_one_channel(D):
    assert len({key_place(d, D) for d in range(D)}) == D
    assert max(w for w, _ in (key_place(d, D) for d in range(D))) == D // 8 - 1
    assert len({value_place(t, d, D) for t in range(32) for d in range(D)}) == 32 * D


@pytest.mark.parametrize("D,g", [(64, 32), (64, 64), (128, 32), (128, 128), (256, 64)])
def test_stored_rows_read_back(D, g):
    rnd, gen = rng(D + g)
    lens, off, table, pages = batch(rnd, [5, 70], [5, 40], 32)
    c = random_cache(gen, pages, 2, D, 32, g)
    before = [t.clone() for t in values_of(c)]
    k, v = (torch.randn((45, 2, D), generator=gen) for _ in range(2))
    store(c, k, v, lens, off, table)
    kc, vc = codes_of(c)
    kq, vq = quantized(k, g)[0], quantized(v, g)[0]
    touched = torch.zeros(kc.shape[:1] + kc.shape[2:3], dtype=torch.bool)
    for b, (n, m) in enumerate(((5, 5), (70, 40))):
        for i in range(m):
            t = n - m + i
            p = int(table[b, t // 32])
            touched[p, t % 32] = True
            assert torch.equal(kc[p, :, t % 32], kq[int(off[b]) + i]) and torch.equal(vc[p, :, t % 32], vq[int(off[b]) + i])
    for x, y in zip(before, values_of(c)):
        assert torch.equal(x.transpose(1, 2)[~touched], y.transpose(1, 2)[~touched])


def test_group_codes_are_half_a_step_off_at_most():
    # z and s are rounded to fp16 before the codes are taken: (15.5 steps of it cover the range)
    x = torch.randn((50, 1, 128), generator=torch.Generator().manual_seed(1))
    q, sz = quantized(x, 64)
    s, z = sz.float()[..., :1], sz.float()[..., 1:]
    y = (q.unflatten(-1, (-1, 64)).float() * s + z).flatten(-2)
    step = s.expand(-1, -1, -1, 64).flatten(-2)
    assert bool(((x - y).abs() <= 0.52 * step).all())


def test_empty_cache_and_its_shape():
    c = qg.kv4_cache(3, 2, 128, 64, 32, device="cpu")
    assert (c.pages, c.heads, c.page_size, c.head_dim, c.group) == (3, 2, 64, 128, 32)
    assert not any(bool(x.any()) for x in values_of(c))
    for kw in (dict(head_dim=96), dict(group=48), dict(head_dim=64, group=128), dict(page_size=16),
               dict(page_size=96), dict(page_size=2048)):
        with pytest.raises(ValueError):
            qg.kv4_cache(**{**dict(pages=1, heads=1, head_dim=128, device="cpu"), **kw})
