"""Rows so wide that their count of 128-column blocks passes 32 bits on the way: no GPU."""
import ctypes

import pytest
import torch

import int4_weight_only_uint32_amd as qg

P = ctypes.c_void_p
FAKE = P(0x10000)     # never dereferenced


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake pointers: only where no kernel can start")
@pytest.mark.parametrize("K", [2**31 - 128, 2**31 - 112, 2**31 - 16])
def test_blocks_of_the_widest_rows_are_counted(K):
    """2^24 blocks a row, of 2^28 - 16 in one launch."""
    def call(M):
        return qg.lib().quantize_rows_fp8(FAKE, qg.QG_DTYPE_F16, M, K, 0, FAKE, FAKE, None)
    assert call(1) == qg.QG_ERR_DEVICE
    assert call(15) == qg.QG_ERR_DEVICE
    for M in (16, 17, 1000, 2**31 - 1):
        assert call(M) == qg.QG_ERR_UNSUPPORTED, M
        assert b"too large" in qg.lib().qg_last_error()
