"""The 4-bit cache where indices into its words pass 32 bits, not only byte offsets."""
import pytest
import torch

import int4_weight_only_uint32_amd as qg
from tests.gpu_util import note
from tests.kv4_util import codes_of, rng, store

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,g,page", [(64, 32, 1024), (256, 128, 256)])
def test_words_past_32_bits(D, g, page):
    """Pages whose first word is number 2^31, 2^32 - (a page) and 2^32 and more, of codes; scales
    pass 2^30 words (2^32 bytes).  The rows are held against a small cache."""
    H = 8
    words = H * page * D // 8                                  # a page's
    pages = 2**32 // words + 3
    assert (pages - 1) * words >= 2**32 and pages * H < 2**31
    if D == 64:
        assert (pages - 1) * H * (D // g) * page >= 2**30
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("not enough memory")
    rnd, gen = rng(D)
    note(f"words past 32 bits D={D} g={g} page={page} pages={pages}")
    cache = qg.kv4_cache(pages, H, D, page, g)
    names = ("k", "v", "k_sz", "v_sz")
    at = [pages - 1, 2**31 // words, 2**32 // words - 1, 2**32 // words]
    # what a number cut to 32 bits would meet: the pages 2^31 and 2^32 words before
    near = [p - 2**32 // words for p in at if p >= 2**32 // words] + [p - 2**31 // words for p in at]
    n = 3 * page + 77
    lens, off = torch.tensor([n], dtype=torch.int32), torch.tensor([0, n], dtype=torch.int32)
    table = torch.tensor([at], dtype=torch.int32)
    k, v = (torch.randn((n, H, D), generator=gen).bfloat16() for _ in range(2))
    qg.kv4_append(cache, k.cuda(), v.cuda(), lens.cuda(), table.cuda(), seq_offsets=off.cuda())
    for name in names:
        for p in set(near) - set(at):
            assert not bool(getattr(cache, name)[p].any()), (name, p)
    small = qg.kv4_cache(4, H, D, page, g, device="cpu")
    moved = torch.tensor([[0, 1, 2, 3]], dtype=torch.int32)
    # all rows against a small cache on the GPU, the last five against the CPU's form
    onto = qg.kv4_cache(4, H, D, page, g)
    qg.kv4_append(onto, k.cuda(), v.cuda(), lens.cuda(), moved.cuda(), seq_offsets=off.cuda())
    for name in names:
        for i, p in enumerate(at):
            assert torch.equal(getattr(cache, name)[p], getattr(onto, name)[i]), (name, p)
    store(small, k[-5:].float(), v[-5:].float(), lens, torch.tensor([0, 5]), moved)
    for a, b in zip(codes_of(qg.KV4Cache(*(getattr(cache, name)[at[3]:at[3] + 1] for name in names))), codes_of(small)):
        assert torch.equal(a[0, :, 72:77], b[3, :, 72:77])
    q = torch.randn((2, 2 * H, D), generator=gen).bfloat16()
    off = torch.tensor([0, 2], dtype=torch.int32)
    for hint in (1, 100):
        got = qg.kv4_attend(q.cuda(), cache, lens.cuda(), table.cuda(), seq_offsets=off.cuda(), max_new=hint)
        want = qg.kv4_attend(q.cuda(), onto, lens.cuda(), moved.cuda(), seq_offsets=off.cuda(), max_new=hint)
        assert torch.equal(got, want) and bool(torch.isfinite(got).all())
    rows = qg.kv4_read(cache, lens.cuda(), table.cuda(), seq_offsets=torch.tensor([0, n]).int().cuda(), rows=n)
    same = qg.kv4_read(onto, lens.cuda(), moved.cuda(), seq_offsets=torch.tensor([0, n]).int().cuda(), rows=n)
    assert all(torch.equal(a, b) for a, b in zip(rows, same))
    del cache
    torch.cuda.empty_cache()
