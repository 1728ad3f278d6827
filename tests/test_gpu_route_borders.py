"""Routing where 32 bits run out: biases whose sums overflow them."""
import pytest
import torch

import int4_weight_only_uint32_amd as qg
from tests.gpu_util import note
from tests.test_gpu_moe import INF, logits_of, ref_route

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available()
    assert qg.qg_device_supported(0), "GPU visible but not gfx950"
    torch.cuda.set_device(0)


def same_ids(x, k, **kw):
    ids, _ = qg.route(x, k, **kw)
    torch.cuda.synchronize()
    assert (ids.cpu().numpy() == ref_route(x, k, **kw)[0]).all()


def test_group_sums_beyond_32_bits():
    """Finite biases whose two largest of each group sum to more than 32 bits hold:
    groups of {3.3e38, 0.2e38} and {3.0e38, 3.0e38}, the second of which wins."""
    note("route group sums beyond 32 bits")
    bias = torch.tensor([3.3e38, 0.2e38, 3.0e38, 3.0e38], device="cuda")
    for score in ("softmax", "sigmoid"):
        ids, _ = qg.route(logits_of(3, 4, torch.float32, 1), 1, bias=bias, score=score, n_group=2, topk_group=1,
                          group_score="top2")
        torch.cuda.synchronize()
        assert ids.flatten().tolist() == [2, 2, 2]


@pytest.mark.parametrize("n_group,E", [(8, 64), (4, 96), (6, 60), (2, 1024)])
@pytest.mark.parametrize("topk_group", [1, 2])
@pytest.mark.parametrize("least", [-3.4e38, 0.0, 2.5e38])
def test_biases_near_the_largest_value(n_group, E, topk_group, least):
    """Sums that overflow in some groups, in all (least 2.5e38) and to both sides."""
    note(f"route biases near the largest value E={E} groups {topk_group}/{n_group} from {least}")
    for seed in range(6):
        g = torch.Generator().manual_seed(seed)
        bias = (least + (3.4e38 - least) * torch.rand(E, generator=g, dtype=torch.float64)).float().cuda()
        x = logits_of(5, E, torch.float32, seed)
        for score in ("softmax", "sigmoid"):
            for gs in ("max", "top2"):
                for k in (1, 3):
                    same_ids(x, k, bias=bias, score=score, n_group=n_group, topk_group=topk_group, group_score=gs)


def test_infinite_biases():
    """An infinite choice is a choice: the first of each group, of all of them or of
    the last two groups only."""
    note("route infinite biases")
    x = logits_of(4, 64, torch.float32, 2)
    for groups in (slice(0, 8), slice(6, 8)):
        bias = torch.zeros(8, 8)
        bias[groups, 0] = INF
        for gs in ("max", "top2"):
            for k in (1, 2, 9):
                same_ids(x, k, bias=bias.flatten().cuda(), n_group=8, topk_group=2, group_score=gs)
