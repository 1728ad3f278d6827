"""The weights of masked, infinite and far rows, each token held to its own bound.

In units of 2^-24 of a weight.  An exponential is off by 4 (2^-22) and by its argument's
rounding, |l - max| of them, at most 150: terms further below the largest are less than
2^-149 of it and are taken in 64 bits where they are weights.  softmax: that for the
weight and, on average, for the sum, whose terms meet in up to 7 additions at 72 experts,
a reciprocal (2) and two products: 19 + 2 |l - max|.  Sigmoid: exponential 4, the sum with
1, the reciprocal 2, and the same for the sum they are divided by, with its 6
additions, the division and the scaling: 22.  24 covers both.  Weights down to and below
the least value: half a step of it, 2^-150, rounded up."""
import math

import numpy as np
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


def rows_of_extremes(E):
    x = logits_of(14, E, torch.float32, 1)
    x[0] = -INF
    x[1, 3:] = -INF
    x[2, ::2] = float("nan")
    x[3, 10] = INF
    x[4, 10:13] = INF
    x[5] = 300 * torch.randn(E, generator=torch.Generator().manual_seed(2)).cuda()
    x[6] = torch.finfo(torch.float32).min
    x[6, 5] = 0
    x[7, 9:] = -INF
    x[8, 9:] = -INF
    x[8, 40] = -50
    x[9] = float("nan")
    x[10] = torch.finfo(torch.float32).max
    x[11] = torch.finfo(torch.float32).min
    x[12] = INF
    x[12, ::2] = float("nan")
    x[13, 7:] = torch.finfo(torch.float32).min
    return x


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("biased", [False, True])
def test_weights_of_masks_and_extremes(score, renormalize, biased):
    note(f"route weights of extremes {score} renormalize={renormalize} bias={biased}")
    E = 72
    x = rows_of_extremes(E)
    bias = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(3)).cuda() if biased else None
    if biased:
        bias[7], bias[8] = -INF, float("nan")
    for kw in (dict(), dict(n_group=8, topk_group=3), dict(n_group=8, topk_group=3, group_score="top2")):
        ids, w = qg.route(x, 6, bias=bias, score=score, renormalize=renormalize, scaling=2.5, **kw)
        torch.cuda.synchronize()
        ri, rw = ref_route(x, 6, bias=bias, score=score, renormalize=renormalize, scaling=2.5, **kw)
        assert (ids.cpu().numpy() == ri).all()
        w = w.cpu().double().numpy()
        for t in range(x.shape[0]):
            l = x[t].double().cpu().numpy()
            l = l[np.isfinite(l)]
            span = min(150.0, float(l.max() - l.min())) if l.size else 0.0
            units = 24 + (2 * span if score == "softmax" else 0)
            tol = units * 2.0**-24 * np.abs(rw[t]) + 2.5 * 2.0**-149
            assert (np.abs(w[t] - rw[t]) <= tol).all(), (t, w[t], rw[t])


def test_weights_of_equal_shares():
    """Named values, apart from any computation: +infinity and the largest finite logit share
    equally, a token with nothing left weighs nothing."""
    note("route weights of equal shares")
    x = rows_of_extremes(72)
    ids, w = qg.route(x, 6, scaling=2.5)
    one = qg.route(x, 6, renormalize=False)[1]
    torch.cuda.synchronize()
    w, one = w.cpu(), one.cpu()
    assert w[0].tolist() == [0.0] * 6 and ids[0].tolist() == [-1] * 6
    assert w[3].tolist() == [2.5] + [0.0] * 5
    for j in range(6):
        for got, want in ((w[4, j], 2.5 / 3 if j < 3 else 0.0), (w[10, j], 2.5 / 6), (w[12, j], 2.5 / 6),
                          (w[11, j], 2.5 / 6), (one[10, j], 1 / 72), (one[12, j], 1 / 36), (one[11, j], 1 / 72),
                          (one[4, j], 1 / 3 if j < 3 else 0.0)):
            assert math.isclose(float(got), want, rel_tol=24 * 2.0**-24, abs_tol=0.0), (j, float(got), want)
    assert w[6].tolist() == [2.5] + [0.0] * 5 and ids[6].tolist() == [5, 0, 1, 2, 3, 4]
    assert not bool(w[9].any())
    assert sorted(ids[13].tolist()) == x[13, :7].topk(6).indices.sort().values.tolist()


@pytest.mark.parametrize("score,bound", [("sigmoid", 2.34 * 2.0**-24), ("softmax", 2.0**-18)])
def test_scores_within_the_bound_that_the_order_relies_on(score, bound):
    """Weights that are neither divided nor scaled are the 32-bit scores themselves: a
    sigmoid is off by at most (4 s (1 - s) + s^2 + 1) 2^-24, 2.34 of them at s = 2/3."""
    note(f"route score errors {score}")
    for sd in (0.5, 2.0, 8.0, 30.0):
        x = logits_of(20000, 64, torch.float32, int(sd * 2), sd)
        ids, w = qg.route(x, 64, score=score, renormalize=False)
        s = torch.sigmoid(x.double()) if score == "sigmoid" else torch.softmax(x.double(), 1)
        err = (w.double() - s.gather(1, ids.long())).abs().max()
        assert float(err) <= bound, float(err) * 2.0**24
