"""Attention over the 4-bit cache with the largest and smallest softmax scales that are allowed."""
import pytest
import torch

import int4_weight_only_uint32_amd as qg
from tests.gpu_util import note
from tests.kv4_util import attend, batch, random_cache, rng, to_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale,size", [(3.4e38, 1e-38), (2.9e38, 2e-38), (2.4e38, 1e-37), (2.0e38, 1e-37), (1.2e-38, 1e37), (3e-42, 1e37)])
@pytest.mark.parametrize("max_new", [1, 100])
def test_softmax_scale(scale, size, max_new):
    rnd, gen = rng(41)
    lens, off, table, pages = batch(rnd, [150], [3], 64)
    c = random_cache(gen, pages, 1, 128, 64, 64, spread=0.05)
    q = (torch.randn((3, 4, 128), generator=gen) * size).bfloat16()
    note(f"softmax scale {scale} queries {size} max_new={max_new}")
    out = qg.kv4_attend(q.cuda(), to_gpu(c), lens.cuda(), table.cuda(), seq_offsets=off.cuda(), max_new=max_new,
                        scale=scale).cpu()
    ref, tol = attend(q, c, lens, off, table, float(torch.tensor(scale, dtype=torch.float32)))
    err = (out.double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
