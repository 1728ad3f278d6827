"""Race check of the routing, sorting and tiled fp8 kernels: the same bits from the library
and from the build that waits after each load to LDS and where lanes meet in LDS.  The
quantizers and the weighted sum, which stage nothing, are the same code in both: for them
this is a repeat on a second copy of the library."""
import pytest
import torch

import int4_weight_only_uint32_amd as qg
from tests.gpu_util import note
from tests.test_gpu_fp8 import codes, kb, offsets_of, scales
from tests.test_gpu_fp8_debug_sync import both

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available()
    assert qg.qg_device_supported(0), "GPU visible but not gfx950"
    torch.cuda.set_device(0)


@pytest.mark.parametrize("swiglu,dtype,M,K", [(True, torch.bfloat16, 3000, 2064), (True, torch.float16, 33, 5120),
                                              (False, torch.float16, 1000, 1040)])
def test_quantizer(swiglu, dtype, M, K, monkeypatch):
    note(f"debug-sync quantize_fp8 swiglu={swiglu} {dtype} M={M} K={K}")
    x = torch.randn(M, K * (1 + swiglu), device="cuda").to(dtype)
    both(monkeypatch, lambda: qg.quantize_fp8(x, swiglu=swiglu))


# experts of each width; groups on whole runs of lanes and (60 of 6, 1000 of 10) out of LDS
@pytest.mark.parametrize("E,g,kg,k", [(60, 6, 2, 4), (64, 8, 3, 8), (128, 1, 1, 6), (256, 8, 4, 8), (500, 5, 2, 9),
                                      (1000, 10, 4, 20)])
@pytest.mark.parametrize("biased", [False, True])
def test_route(E, g, kg, k, biased, monkeypatch):
    note(f"debug-sync route E={E} groups {kg}/{g} bias={biased}")
    x = torch.randn(3000, E, device="cuda")
    x[::7] = (x[::7] * 8).round() / 8                # (ties, which go to 64 bits)
    bias = (torch.randn(E, device="cuda") * 8).round() / 64 if biased else None
    for gs in ("max", "top2"):
        for _ in range(3):
            both(monkeypatch, lambda: qg.route(x, k, bias=bias, score="sigmoid", n_group=g, topk_group=kg, group_score=gs))


# one workgroup of 8 waves and of 16, two launches
@pytest.mark.parametrize("T,k,E", [(100, 8, 64), (1000, 2, 800), (500, 8, 64), (9000, 8, 256), (5000, 6, 1024)])
def test_sort(T, k, E, monkeypatch):
    note(f"debug-sync sort T={T} k={k} E={E}")
    ids = torch.randint(-1, E, (T, k), dtype=torch.int32, device="cuda")
    for _ in range(3):
        row = torch.zeros(T * k, dtype=torch.int32, device="cuda")
        both(monkeypatch, lambda: qg.sort_rows(ids, E, row_token=row))


# each tile: 64 x 64, 64 x 128 (one and two groups over k), 128 x 128, 128 x 256 with four and
# eight waves, 256 x 256, and 256 x 256 with each of its small ones
@pytest.mark.parametrize("M,N,K", [
    (300, 3000, 1104), (200, 9000, 528), (256, 8192, 2064), (64, 40000, 656), (256, 17408, 4624), (256, 17408, 1040),
    (600, 21000, 1552), (1024, 17408, 784), (1024, 19500, 272), (1024, 21900, 400)])
def test_tiles(M, N, K, monkeypatch):
    note(f"debug-sync fp8_gemm M={M} N={N} K={K}")
    a, w = codes((M, K), 1), codes((N, K), 2)
    sa, sw = scales((M, kb(K)), 3), scales((kb(N), kb(K)), 4)
    for _ in range(3):
        both(monkeypatch, lambda: [qg.fp8_gemm(a, sa, w, sw)])


def test_experts_with_waves_that_have_no_rows(monkeypatch):
    note("debug-sync fp8_gemm partial row blocks of 12 experts")
    counts, N, K = [1, 70, 0, 200, 257, 300, 129, 64, 500, 3, 90, 256], 7300, 2064
    E, M = len(counts), sum(counts)
    a, w = codes((M, K), 1), codes((E, N, K), 2)
    sa, sw = scales((M, kb(K)), 3), scales((E, kb(N), kb(K)), 4)
    off = offsets_of(counts)
    rows = torch.randperm(M, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    for idx in (None, rows):
        for _ in range(3):
            both(monkeypatch, lambda: [qg.fp8_gemm(a, sa, w, sw, expert_offsets=off, a_rows=idx)])
