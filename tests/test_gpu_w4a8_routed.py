"""Routed rows through the int4 experts with tokens that no expert takes: the gather of codes
and token scales by a row_token that was zero-filled before the sort."""
import numpy as np
import pytest
import torch

import int4_weight_only_uint32_amd as qg
import oracle
import synth
from tests.gpu_util import dev, note
from tests.test_gpu_moe import INF, logits_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available()
    assert qg.qg_device_supported(0), "GPU visible but not gfx950"
    torch.cuda.set_device(0)


@pytest.mark.parametrize("T", [1, 30, 200])
def test_dropped_slots(T):
    note(f"w4a8 routed rows T={T}")
    E, K, N, k = 4, 256, 256, 2
    c = synth.w4a8_case(E, 16, K, N, 128, stream=7, case_id=1)
    packs = [qg.pack(dev(c.q[e]), dev(c.s[e]), None, 128, fold=True) for e in range(E)]
    W = torch.stack([p.w for p in packs]).contiguous()
    S = torch.stack([p.scale for p in packs]).contiguous()
    x = torch.randn(T, K, generator=torch.Generator().manual_seed(5)).half().cuda()
    logits = logits_of(T, E, torch.float16, 6)
    logits[::5] = -INF                                   # padded tokens (T = 1: the only one)
    logits[1::5, 1:] = -INF                              # one expert left for two slots
    ids, w = qg.route(logits, k)
    tok = torch.zeros(T * k, dtype=torch.int32, device="cuda")
    off, tok, slot = qg.sort_rows(ids, E, row_token=tok)
    q, s = qg.quantize_rows(x)
    rows = tok.long()
    y = qg.w4a8(q[rows], s[rows], W, S, off, E, T, N, 128)
    out = qg.combine_rows(y, slot, w)
    torch.cuda.synchronize()
    assert int(off[E]) == int((ids >= 0).sum()) < T * k
    assert not bool(out[::5].any())
    if T == 1:
        return
    ref8, _ = oracle.w4a8(q[rows].cpu().numpy(), s[rows].cpu().numpy(), c.q, c.s, off.cpu().numpy(), 128)
    y64 = torch.from_numpy(np.asarray(ref8, dtype=np.float64))
    sl, w = slot.cpu().long(), w.cpu().double()
    ref = (torch.where(sl[..., None] >= 0, y64[sl.clamp_min(0)], 0.0) * w[..., None]).sum(1)
    err = out.cpu().double() - ref
    # each row of the product in fp32, then an fp16 rounding of it and of the sum (2^-11 each of
    # a row's or the result's size; two rows of a result may cancel, which 2^-8 leaves room for)
    assert float(err.norm() / ref.norm()) <= 2.0**-8
