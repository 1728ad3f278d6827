"""Race check of the 4-bit cache's and the adapters' kernels: the library and its build whose
pipeline stages wait for every outstanding memory operation give the same bits."""
import pytest
import torch

import int4_weight_only_uint32_amd as qg
from tests.gpu_util import note
from tests.kv4_util import batch, random_cache, to_gpu
from tests.test_gpu_fp8_debug_sync import both
from tests.test_gpu_kv4 import rng

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available()
    assert qg.qg_device_supported(0), "GPU visible but not gfx950"
    torch.cuda.set_device(0)


@pytest.mark.parametrize("D,g,R,lens,news,window", [
    (128, 64, 5, [4000, 1, 777, 31], [1, 1, 1, 1], 0),            # parts of one size
    (128, 128, 8, [1000], [1], 0), (64, 32, 4, [1200, 64], [1, 1], 0),  # eight waves
    (128, 32, 4, [900] * 40, [1] * 40, 200), (256, 32, 3, [700, 2000], [1, 1], 0), (256, 128, 2, [1500], [1], 0),
    (128, 64, 5, [900, 333], [300, 333], 0), (128, 32, 2, [1300], [500], 100), (64, 64, 1, [700], [600], 0),
    (256, 64, 2, [500, 70], [200, 70], 0),
])
def test_attend(D, g, R, lens, news, window, monkeypatch):
    rnd, gen = rng(D + g + sum(lens))
    note(f"attend debug-sync D={D} g={g} R={R} lens={lens[:4]} news={news[:4]} window={window}")
    lens_t, off, table, pages = batch(rnd, lens, news, 64)
    c, table = to_gpu(random_cache(gen, pages, 8, D, 64, g)), table.cuda()
    lens_t, off = lens_t.cuda(), off.cuda()
    q = torch.randn((sum(news), 8 * R, D), generator=gen).half().cuda()
    for _ in range(3):
        both(monkeypatch, lambda: [qg.kv4_attend(q, c, lens_t, table, seq_offsets=off, max_new=max(news),
                                                 window=window)])


@pytest.mark.parametrize("T,L,R,K,N", [(1, 3, 16, 2048, 4096), (64, 32, 16, 5120, 5128), (50, 2, 24, 520, 1000),
                                       (300, 3, 64, 2048, 2048), (1000, 4, 128, 1032, 3000), (900, 2, 200, 512, 512)])
def test_adapters(T, L, R, K, N, monkeypatch):
    note(f"lora debug-sync T={T} L={L} R={R} K={K} N={N}")
    gen = torch.Generator().manual_seed(T + K)
    x, A, B, y = (torch.randn(s, generator=gen).bfloat16().cuda() for s in ((T, K), (L, R, K), (L, N, R), (T, N)))
    plan = qg.sort_rows(torch.randint(-1, L, (T, 1), generator=gen, dtype=torch.int32).cuda(), L)
    for _ in range(3):
        both(monkeypatch, lambda: [qg.lora(x, A, B, plan, y.clone())])


@pytest.mark.parametrize("D,g,H", [(128, 64, 8), (64, 32, 3), (256, 128, 2)])
def test_append_and_read(D, g, H, monkeypatch):
    rnd, gen = rng(D + H)
    note(f"append and read debug-sync D={D} g={g} H={H}")
    lens_t, off, table, pages = batch(rnd, [500, 40, 3], [200, 40, 1], 64)
    k, v = (torch.randn((241, H, D), generator=gen).half().cuda() for _ in range(2))
    lens_t, off, table = lens_t.cuda(), off.cuda(), table.cuda()

    def call():
        c = qg.kv4_cache(pages, H, D, 64, g)
        for t in (c.k, c.v, c.k_sz, c.v_sz):
            t.zero_()
        qg.kv4_append(c, k, v, lens_t, table, seq_offsets=off)
        return [c.k, c.v, c.k_sz, c.v_sz, *qg.kv4_read(c, lens_t, table, seq_offsets=off, rows=241)]

    both(monkeypatch, call)
