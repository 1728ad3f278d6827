"""A workspace on another GPU than the call's tensors is refused by the binding
(tensors without storage stand in for two GPUs, no kernel can start)."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import int4_weight_only_uint32_amd as qg

pytestmark = [pytest.mark.skipif(torch.cuda.is_available(), reason="tensors without storage: only where no kernel can start"),
              pytest.mark.filterwarnings("ignore:Accessing the data pointer of FakeTensor")]


def test_workspace_of_another_gpu():
    with FakeTensorMode():
        def t(*shape, dtype=torch.int32, dev="cuda:0"):
            return torch.empty(shape, dtype=dtype, device=dev)

        f8, f32, u8 = torch.float8_e4m3fn, torch.float32, torch.uint8
        ws = t(1 << 20, dtype=u8, dev="cuda:1")
        with pytest.raises(ValueError, match="workspace is on cuda:1, not on GPU 0"):
            qg.moe_sort_rows(t(9000, 8), 9000, 8, 256, t(257), t(72000), t(9000, 8), ws)
        with pytest.raises(ValueError, match="workspace is on cuda:1, not on GPU 0"):
            qg.qgemm_fp8(t(4, 128, dtype=f8), t(4, 1, dtype=f32), None, 4, t(64, 128, dtype=f8), t(1, 1, dtype=f32), None,
                         1, 4, 64, 128, t(4, 64, dtype=torch.float16), ws)
        with pytest.raises(ValueError, match="ids is on cuda:1|expert_offsets is on cuda:0"):
            qg.moe_sort_rows(t(9000, 8, dev="cuda:1"), 9000, 8, 256, t(257), t(72000), t(9000, 8), ws)
        with pytest.raises(ValueError, match="contiguous"):
            qg.moe_sort_rows(t(9000, 8), 9000, 8, 256, t(257), t(72000), t(9000, 8), t(1 << 20, 2, dtype=u8)[:, 0])
