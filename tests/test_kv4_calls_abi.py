"""CPU checks of the 4-bit cache's calls: which softmax scales are taken, what the binding expects
of a batch's rows.  No kernel runs here."""
import ctypes
import math

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

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


@pytest.mark.skipif(torch.cuda.is_available(), reason="tensors without storage: only where no kernel can start")
@pytest.mark.filterwarnings("ignore:Accessing the data pointer of FakeTensor")
@pytest.mark.parametrize("T,B,given,want", [(64, 64, None, 1), (65, 64, None, 2), (3, 64, None, 1), (0, 4, None, 1),
                                            (0, 0, None, 1), (5, 1, None, 5), (700, 3, None, 234), (700, 3, 8, 8)])
def test_expected_rows_of_a_sequence(T, B, given, want, monkeypatch):
    """Without max_new a decode batch that comes with offsets is taken for one: the rows' mean."""
    seen = []
    monkeypatch.setattr(qg, "_call", lambda fn, dev, *args: seen.append(args))
    with FakeTensorMode():
        t = lambda *shape, dtype=torch.int32: torch.empty(shape, dtype=dtype, device="cuda:0")  # noqa: E731
        words, sz = (9, 2, 64, 16), (9, 2, 2, 64, 2)
        c = qg.KV4Cache(t(*words), t(*words), t(*sz, dtype=torch.float16), t(*sz, dtype=torch.float16))
        qg.kv4_attend(t(T, 8, 128, dtype=torch.float16), c, t(B), t(B, 4), seq_offsets=t(B + 1), max_new=given)
    # (q, type, T, row distance, query heads, max_new, ...)
    assert seen[0][2] == T and seen[0][5] == want
