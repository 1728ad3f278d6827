"""Attention over the 4-bit cache where single tokens have value scales far above the others':
p times the scale must not leave fp16's range, whichever token of a block it is."""
import pytest
import torch

import int4_weight_only_uint32_amd as qg
from tests.gpu_util import note
from tests.kv4_util import attend, batch, random_cache, rng, to_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,g,R,new,hints", [
    (64, 64, 4, 1, (1, 100)), (64, 32, 3, 1, (1, 100)), (128, 128, 2, 1, (1, 100)), (128, 64, 5, 1, (1, 100)),
    (128, 32, 4, 1, (1, 100)), (256, 128, 2, 1, (1, 100)), (256, 32, 1, 1, (1, 100)), (128, 64, 2, 40, (40, 1)),
    (128, 32, 1, 40, (40, 1)), (256, 64, 1, 40, (40, 1)),
])
@pytest.mark.parametrize("size", [8.0, 300.0, 60000.0])
def test_single_tokens(D, g, R, new, hints, size):
    """One token each of the blocks' eight places in a lane (32 i + 4 j + r, j and r 0 .. 3), in its
    last group; queries of zeros (every p the largest) and random ones."""
    rnd, gen = rng(D + g + new)
    n = 32 * 18 + 5
    lens, off, table, pages = batch(rnd, [n], [new], 64)
    c = random_cache(gen, pages, 1, D, 64, g)
    for i in range(16):
        t = 32 * i + 4 * (i // 4) + i % 4 + (16 if i % 3 else 0)
        c.v_sz[int(table[0, t // 64]), 0, -1, t % 64] = torch.tensor([size / 8, -size / 2]).half()
    q = torch.randn((new, 2 * R, D), generator=gen).bfloat16()
    q[:, :R] = 0.0
    # one key/value head, 2 R query heads
    ref, tol = attend(q, c, lens, off, table, D ** -0.5)
    for hint in hints:
        note(f"single large scales D={D} g={g} R={R} new={new} size={size} max_new={hint}")
        out = qg.kv4_attend(q.cuda(), to_gpu(c), lens.cuda(), table.cuda(), seq_offsets=off.cuda(), max_new=hint).cpu()
        err = (out.double() - ref).abs()
        assert bool((err <= tol).all()), float((err / tol).max())
