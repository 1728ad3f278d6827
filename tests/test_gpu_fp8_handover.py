"""The columns where the fp8 product's large tiles hand over to small ones."""
import pytest
import torch

import int4_weight_only_uint32_amd as qg
from tests.gpu_util import note
from tests.test_gpu_fp8 import check, codes, kb, scales

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available()
    assert qg.qg_device_supported(0), "GPU visible but not gfx950"
    torch.cuda.set_device(0)


# 4 row blocks of 256 rows: rounds of 256 large tiles end at column 16384, 65 row blocks (one
# round holds 3 column blocks) at 768; the rest goes to 64 x 128, 128 x 128 or 128 x 256 tiles
@pytest.mark.parametrize("M,N,K,at", [
    (1000, 17500, 272, 16384), (1024, 17408, 144, 16384), (1000, 19500, 272, 16384), (1024, 21900, 144, 16384),
    (1024, 26000, 144, 16384), (16500, 1000, 144, 768), (1024, 16640, 272, 16384), (1001, 16385, 400, 16384)])
def test_columns_around_the_handover(M, N, K, at):
    note(f"fp8_gemm handover M={M} N={N} K={K}")
    a, w = codes((M, K), 1), codes((N, K), 2)
    sa, sw = scales((M, kb(K)), 3), scales((kb(N), kb(K)), 4)
    C = torch.full((M, N), float("nan"), dtype=torch.float16, device="cuda")
    qg.fp8_gemm(a, sa, w, sw, C=C)
    torch.cuda.synchronize()
    assert bool(C.isfinite().all())
    cols = torch.arange(max(0, at - 270), min(N, at + 270))
    part, cols = (cols // 128).cuda(), cols.cuda()
    fa = sa.double().repeat_interleave(128, 1)[:, :K]
    fw = sw[part].double().repeat_interleave(128, 1)[:, :K]
    av, wv = a.double(), w[cols].double()
    up = lambda v: torch.where(v != 0, v.abs().clamp_min(2.0**-6), 0.0)
    check(C[:, cols], (av * fa).cpu(), (wv * fw).cpu(), (up(av) * fa).float(), (up(wv) * fw).float(), torch.float16)
