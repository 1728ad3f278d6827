"""Codes of blocks without a scale: the byte 0, whatever the signs."""
import pytest
import torch

import int4_weight_only_uint32_amd as qg
from tests.gpu_util import note
from tests.test_gpu_fp8 import ref_quant

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available()
    assert qg.qg_device_supported(0), "GPU visible but not gfx950"
    torch.cuda.set_device(0)


def bytes_and_scales(x, swiglu=False):
    q, s = qg.quantize_fp8(x.cuda(), swiglu=swiglu)
    torch.cuda.synchronize()
    return q.view(torch.uint8).cpu(), s.cpu()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_blocks_of_negative_zeros(dtype):
    """Alone, mixed with +0, in a partial block; a live block keeps the sign of its zeros."""
    note(f"quantize_fp8 negative zeros {dtype}")
    x = torch.zeros(4, 272, dtype=dtype)
    x[0] = -0.0
    x[1, ::3] = -0.0
    x[2, 256:] = -0.0
    x[3] = -0.0
    x[3, 130] = -2.0
    q, s = bytes_and_scales(x)
    want = torch.zeros(4, 272, dtype=torch.uint8)
    want[3, 128:256] = 0x80
    want[3, 130] = 0xFE                      # -448
    assert torch.equal(q, want)
    assert int(s.count_nonzero()) == 1 and float(s[3, 1]) == float(torch.tensor(2.0) / 448)


def test_swiglu_zeros_with_a_sign():
    """A gate of 0 with negative up values, of -0, and gates whose silu or whose
    product 32 bits round to -0."""
    note("quantize_fp8 swiglu zeros with a sign")
    x = torch.zeros(6, 256)
    x[0, 128:] = -3.0
    x[1, :128] = -0.0
    x[1, 128:] = 2.0
    x[2, :128] = -1000.0
    x[2, 128:] = 1.0
    x[3, :128] = -30.0
    x[3, 128:] = 1e-38                       # -2.8e-12 * 1e-38: below the least value
    x[4, :128] = 1e-30
    x[4, 128:] = -1e-30
    x[5, :128] = -1e-40                      # (a subnormal) / 448 rounds to 0
    x[5, 128:] = 1e-3
    q, s = bytes_and_scales(x.bfloat16(), swiglu=True)
    assert not bool(s.any()) and not bool(q.any())
    x = torch.zeros(2, 256)
    x[:, 128:] = -3.0
    x[1, :128] = -1000.0
    q, s = bytes_and_scales(x.half(), swiglu=True)
    assert not bool(s.any()) and not bool(q.any())


def test_swiglu_products_just_inside_the_range():
    """16 sigmoid(16) 2^124 is 2^128 (1 - 2^-23.08), which binary32 holds."""
    note("quantize_fp8 swiglu largest product")
    x = torch.zeros(2, 256)
    x[0, 5], x[0, 128 + 5] = 16.0, 2.0**124
    x[1, 9], x[1, 128 + 9] = 16.0, -2.0**124
    x = x.bfloat16()
    q, s = qg.quantize_fp8(x.cuda(), swiglu=True)
    torch.cuda.synchronize()
    gate, up = x.double().chunk(2, 1)
    rq, rs = ref_quant(gate / (1.0 + torch.exp(-gate)) * up)
    assert torch.equal(s.cpu(), rs) and torch.equal(q.cpu().double(), rq)
