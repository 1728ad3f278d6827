"""CPU checks of the 4-bit cache's calls: which softmax scales are taken.  No kernel runs here."""
import ctypes
import math

import pytest
import torch

import int4_weight_only_uint32_amd as qg

P = ctypes.c_void_p
FAKE = P(0x10000)     # never dereferenced

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake pointers: only where no kernel can start")


@no_gpu
@pytest.mark.parametrize("scale,rc", [(3.4028234e38, qg.QG_ERR_DEVICE), (1e-45, qg.QG_ERR_DEVICE), (0.1, qg.QG_ERR_DEVICE),
                                      (math.inf, qg.QG_ERR_INVALID_ARG), (math.nan, qg.QG_ERR_INVALID_ARG),
                                      (-math.inf, qg.QG_ERR_INVALID_ARG), (-0.0, qg.QG_ERR_INVALID_ARG)])
def test_softmax_scales(scale, rc):
    """Every finite one above zero."""
    assert qg.lib().kv4_attend(FAKE, qg.QG_DTYPE_BF16, 2, 1024, 8, 1, None, FAKE, FAKE, 2, 4, FAKE, FAKE, FAKE, FAKE, 9, 2, 64,
                               128, 64, scale, 0, 0, FAKE, None, 0, 0, None) == rc
