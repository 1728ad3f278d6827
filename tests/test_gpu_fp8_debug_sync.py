"""Race check of the fp8 and expert-routing kernels: the library and its build
whose pipeline stages wait for every outstanding memory operation give the same
bits, over every kernel of the fp8 GEMM and the multi-launch sort."""
import pytest
import torch

import int4_weight_only_uint32_amd as qg
from tests.gpu_util import note
from tests.test_gpu_fp8 import codes, kb, offsets_of, scales

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available()
    assert qg.qg_device_supported(0), "GPU visible but not gfx950"
    torch.cuda.set_device(0)


def both(monkeypatch, call):
    """call() with the library and with the waiting build."""
    outs = []
    for load in (qg.lib, qg.debug_sync_lib):
        L = load()
        with monkeypatch.context() as m:
            m.setattr(qg, "_lib", L)
            outs.append([t.clone() for t in call()])
            torch.cuda.synchronize()
    for a, b in zip(*outs):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("M,N,K", [
    (1, 5120, 2064), (16, 65600, 2064), (9, 2048, 2048), (20, 5120, 2064), (32, 65600, 1040), (64, 5120, 4240),
    (100, 4100, 4240), (300, 3000, 2000), (40, 33500, 656), (256, 8192, 2064), (128, 17408, 1296), (512, 9000, 1040),
    (1024, 17408, 784)])
def test_gemm(M, N, K, monkeypatch):
    note(f"fp8_gemm debug-sync M={M} N={N} K={K}")
    a, w = codes((M, K), 1), codes((N, K), 2)
    sa, sw = scales((M, kb(K)), 3), scales((kb(N), kb(K)), 4)
    for _ in range(3):
        both(monkeypatch, lambda: [qg.fp8_gemm(a, sa, w, sw)])


@pytest.mark.parametrize("counts", [[1, 0, 3, 2] * 12, [40, 17, 0, 70, 300, 1, 129, 250] * 2, [700, 260, 900, 129]])
def test_grouped(counts, monkeypatch):
    E, N, K, M = len(counts), 4100, 656, sum(counts)
    a, w = codes((M, K), 1), codes((E, N, K), 2)
    sa, sw = scales((M, kb(K)), 3), scales((E, kb(N), kb(K)), 4)
    off = offsets_of(counts)
    rows = torch.randperm(M, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    for _ in range(3):
        both(monkeypatch, lambda: [qg.fp8_gemm(a, sa, w, sw, expert_offsets=off, a_rows=rows)])


def test_the_other_steps(monkeypatch):
    x = torch.randn(3000, 2064, device="cuda").bfloat16()
    logits, bias = torch.randn(5000, 160, device="cuda"), 0.1 * torch.randn(160, device="cuda")
    both(monkeypatch, lambda: qg.quantize_fp8(x))
    both(monkeypatch, lambda: qg.quantize_fp8(x, swiglu=False))
    both(monkeypatch, lambda: qg.route(logits, 6, bias=bias, n_group=8, topk_group=3, group_score="top2"))
    ids, weights = qg.route(logits, 6, bias=bias, score="sigmoid")
    row = torch.empty(30000, dtype=torch.int32, device="cuda")
    both(monkeypatch, lambda: qg.sort_rows(ids, 160, row_token=row))
    off, _, slot = qg.sort_rows(ids, 160)
    y = torch.randn(30000, 520, device="cuda").half()
    both(monkeypatch, lambda: [qg.combine_rows(y, slot, weights)])
