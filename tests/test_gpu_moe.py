"""GPU parity of the routing, sorting and combining of experts' rows against
plain 64-bit computations, and runs of them together with the quantizers and
grouped products.

Tolerances.  Ids are whole numbers: equal.  A weight is an exponential in
32 bits at worst: its argument off by 2^-24 of the logits' range, plus a
handful of roundings.  A combined value is a sum of topk FMAs in 32 bits (each
off by at most 2^-24 of the sum of magnitudes), then half a step of the output."""
import math

import numpy as np
import pytest
import torch

import int4_weight_only_uint32_amd as qg
import oracle
import synth
from tests.gpu_util import dev, note

pytestmark = pytest.mark.gpu

HALF = {torch.float16: 2.0**-11, torch.bfloat16: 2.0**-8}
INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available()
    assert qg.qg_device_supported(0), "GPU visible but not gfx950"
    torch.cuda.set_device(0)


def ref_route(logits, k, bias=None, score="softmax", n_group=1, topk_group=1, group_score="max",
              renormalize=True, scaling=1.0):
    """One token after another, in 64 bits."""
    x = logits.double().cpu().numpy()
    T, E = x.shape
    b = None if bias is None else bias.double().cpu().numpy()
    ids, ws = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        l = np.where(np.isnan(x[t]), -INF, x[t])
        live = l > -INF
        with np.errstate(all="ignore"):
            if score == "softmax":
                top = l.max()
                p = np.where(live, np.where(l == top, 1.0, np.exp(l - top)), 0.0)
                s = p / p.sum() if live.any() else p
            else:
                s = 1.0 / (1.0 + np.exp(-l))
        # without a bias the logits rank the experts (the order of the scores, which saturate)
        c = l if b is None else s + b
        c = np.where(live & ~np.isnan(c), c, -INF)
        if n_group > 1:
            size = E // n_group
            v = []
            for g in range(n_group):
                o = np.sort((c if b is not None or group_score == "max" else np.where(live, s, -INF))
                            [g * size:(g + 1) * size])[::-1]
                v.append(o[0] if group_score == "max" or size < 2 or o[1] == -INF else o[0] + o[1])
            kept = sorted(range(n_group), key=lambda g: (-v[g], g))[:topk_group]
            for g in range(n_group):
                if g not in kept:
                    c[g * size:(g + 1) * size] = -INF
        for j, e in enumerate(sorted((e for e in range(E) if c[e] > -INF), key=lambda e: (-c[e], e))[:k]):
            ids[t, j], ws[t, j] = e, s[e]
    if renormalize:
        tot = ws.sum(1, keepdims=True)
        ws = np.divide(ws, tot, out=np.zeros_like(ws), where=tot > 0)
    return ids, ws * scaling


def check_route(logits, k, **kw):
    ids, w = qg.route(logits, k, **kw)
    torch.cuda.synchronize()
    ri, rw = ref_route(logits, k, **kw)
    bad = np.argwhere(ids.cpu().numpy() != ri)
    assert bad.size == 0, f"{len(bad)} ids differ, first at {bad[:3].tolist()}"
    fin = logits.double()[logits.isfinite()]
    span = float(fin.max() - fin.min()) if fin.numel() else 0.0
    tol = (span + 16) * 2.0**-24 * np.abs(rw) + 1e-37
    err = np.abs(w.cpu().double().numpy() - rw)
    assert (err <= tol).all(), float((err - tol).max())
    return ids, w


def logits_of(T, E, dtype, seed, sd=1.5):
    return (sd * torch.randn(T, E, generator=torch.Generator().manual_seed(seed))).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,g,kg", [
    (1, 1, 1, 1, 1), (1, 8, 2, 1, 1), (3, 7, 7, 1, 1), (70, 60, 4, 1, 1), (33, 64, 6, 8, 3), (17, 65, 8, 5, 2),
    (40, 128, 8, 1, 1), (65, 160, 6, 8, 3), (130, 256, 8, 8, 4), (9, 257, 10, 1, 1), (5, 384, 8, 1, 1),
    (11, 512, 10, 64, 7), (6, 1000, 64, 10, 4), (4, 1024, 64, 1, 1)])
def test_route(T, E, k, g, kg, score, dtype):
    note(f"route T={T} E={E} k={k} groups {kg}/{g} {score} {dtype}")
    x = logits_of(T, E, dtype, T * E + k)
    bias = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(E)).cuda()
    for b in (None, bias):
        for gs in ("max", "top2"):
            check_route(x, k, bias=b, score=score, n_group=g, topk_group=kg, group_score=gs, renormalize=b is None,
                        scaling=1.0 if b is None else 2.5)


def test_route_many_tokens():
    """Enough tokens that 32-bit scores alone would order some of them wrongly."""
    x = logits_of(16384, 256, torch.float32, 3)
    bias = 0.1 * torch.randn(256, generator=torch.Generator().manual_seed(4)).cuda()
    ids, w = qg.route(x, 8, bias=bias, score="sigmoid", n_group=8, topk_group=4, group_score="top2", scaling=2.5)
    s = torch.sigmoid(x.double())
    c = s + bias.double()
    v = c.view(-1, 8, 32).topk(2, 2).values.sum(2)
    out = torch.ones_like(v, dtype=torch.bool).scatter_(1, v.topk(4, 1).indices, False)
    top = c.masked_fill(out.repeat_interleave(32, 1), -INF).topk(8, 1).indices
    assert torch.equal(ids.long(), top)
    rw = s.gather(1, top)
    assert float((w.double() - 2.5 * rw / rw.sum(1, keepdim=True)).abs().max()) <= 40 * 2.0**-24 * 2.5


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_weights_down_to_the_least_values(score, renormalize):
    """Scores down to 2^-149 and below, with and without a largest one beside
    them: each weight to its own size.  (fast path: as check_route; the 64-bit one
    rounds once; both to half the least step, 2^-150, times the scaling.)"""
    x = torch.linspace(-110, -60, 64).repeat(8, 1)
    for t in range(8):
        x[t] = x[t, torch.randperm(64, generator=torch.Generator().manual_seed(t))] + t / 8
    x[1::2, 7] = 3.0
    ids, w = qg.route(x.cuda(), 64, score=score, renormalize=renormalize, scaling=2.5)
    torch.cuda.synchronize()
    ri, rw = ref_route(x, 64, score=score, renormalize=renormalize, scaling=2.5)
    assert (ids.cpu().numpy() == ri).all()
    tol = (113 + 16) * 2.0**-24 * np.abs(rw) + 2.5 * 2.0**-150
    assert (np.abs(w.cpu().double().numpy() - rw) <= tol).all()


def test_route_scores_closer_than_32_bits():
    """Choices that differ by less than a 32-bit step, in every position: the
    order is that of the real numbers."""
    E, T = 64, 200
    g = torch.Generator().manual_seed(8)
    base = torch.randn(T, 1, generator=g)
    x = (base + torch.randint(-3, 4, (T, E), generator=g) * 2.0**-22).cuda()
    bias = (torch.randint(0, 2, (E,), generator=g) * 2.0**-25).cuda()
    for score in ("softmax", "sigmoid"):
        for b in (None, bias):
            for gk in ((1, 1), (8, 3)):
                check_route(x, 8, bias=b, score=score, n_group=gk[0], topk_group=gk[1], group_score="top2")


def test_route_ties_go_to_the_lowest_index():
    x = torch.zeros(5, 96, device="cuda")
    x[1, 50:] = 1
    x[2] = torch.arange(96, device="cuda").float() // 7
    for score in ("softmax", "sigmoid"):
        for b in (None, torch.zeros(96, device="cuda"), torch.full((96,), -3.0, device="cuda")):
            check_route(x, 9, bias=b, score=score)
            check_route(x, 9, bias=b, score=score, n_group=12, topk_group=3, group_score="top2")
            check_route(x, 9, bias=b, score=score, n_group=12, topk_group=3)


def test_route_masks_and_extremes():
    E = 72
    x = logits_of(12, E, torch.float32, 1)
    x[0] = -INF                                  # nothing left
    x[1, 3:] = -INF                              # fewer experts than slots
    x[2, ::2] = float("nan")
    x[3, 10] = INF
    x[4, 10:13] = INF
    x[5] = 300 * torch.randn(E, generator=torch.Generator().manual_seed(2)).cuda()
    x[6] = torch.finfo(torch.float32).min        # a mask by the lowest value
    x[6, 5] = 0
    x[7, 9:] = -INF                              # groups with no expert
    x[8, 9:] = -INF
    x[8, 40] = -50
    x[9] = float("nan")
    x[10] = torch.finfo(torch.float32).max
    bias = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(3)).cuda()
    bias[7] = -INF
    bias[8] = float("nan")
    for score in ("softmax", "sigmoid"):
        for b in (None, bias):
            for kw in (dict(), dict(n_group=8, topk_group=3), dict(n_group=8, topk_group=3, group_score="top2")):
                for renorm in (True, False):
                    check_route(x, 6, bias=b, score=score, renormalize=renorm, **kw)


def ref_sort(ids, E):
    flat = ids.cpu().numpy().reshape(-1).astype(np.int64)
    keep = np.flatnonzero((flat >= 0) & (flat < E))
    order = keep[np.argsort(flat[keep], kind="stable")]
    slot = np.full(flat.size, -1, np.int32)
    slot[order] = np.arange(order.size)
    off = np.concatenate([[0], np.cumsum(np.bincount(flat[keep], minlength=E))])
    return off, order // ids.shape[1], slot.reshape(ids.shape)


def check_sort(ids, E):
    row = torch.full((ids.numel(),), -7, dtype=torch.int32, device="cuda")
    off, row, slot = qg.sort_rows(ids, E, row_token=row)
    torch.cuda.synchronize()
    ro, rr, rs = ref_sort(ids, E)
    assert np.array_equal(off.cpu().numpy(), ro)
    assert np.array_equal(slot.cpu().numpy(), rs)
    assert np.array_equal(row.cpu().numpy()[:len(rr)], rr)
    assert bool((row[len(rr):] == -7).all())


@pytest.mark.parametrize("T,k,E", [
    (1, 1, 1), (1, 8, 64), (16, 8, 64), (5, 3, 4), (64, 1, 8), (65, 1, 1024), (100, 7, 60), (129, 8, 256), (257, 8, 256),
    (511, 8, 384), (513, 8, 384), (512, 8, 512), (500, 8, 513), (1500, 1, 500), (4096, 1, 3), (1000, 6, 160), (2049, 8, 257), (4099, 8, 1024), (16383, 8, 256), (70001, 2, 8),
    (40000, 9, 128)])
def test_sort(T, k, E):
    note(f"sort T={T} k={k} E={E}")
    g = torch.Generator().manual_seed(T + k + E)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32).cuda()
    check_sort(ids, E)
    ids = torch.randint(-2, E + 3, (T, k), generator=g, dtype=torch.int32).cuda()     # some dropped
    check_sort(ids, E)
    check_sort(torch.full((T, k), E - 1, dtype=torch.int32, device="cuda"), E)        # one expert, each slot again
    check_sort(torch.full((T, k), -1, dtype=torch.int32, device="cuda"), E)           # nothing left
    far = torch.where(torch.rand(T, k, generator=g) < 0.3, 2**31 - 1, -2**31).to(torch.int32).cuda()
    check_sort(far, E)


def test_sort_no_tokens():
    off, row, slot = qg.sort_rows(torch.empty(0, 8, dtype=torch.int32, device="cuda"), 300)
    torch.cuda.synchronize()
    assert off.tolist() == [0] * 301 and row.numel() == 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (1, 8, 7168), (3, 2, 7), (5, 8, 100), (17, 6, 2048), (130, 3, 4104),
                                   (70000, 2, 24), (9, 64, 520), (33, 8, 258)])
def test_combine(T, k, N, dtype):
    note(f"combine T={T} k={k} N={N} {dtype}")
    g = torch.Generator().manual_seed(T + N)
    R = T * k + 3
    Y = torch.randn(R, N, generator=g).to(dtype)
    slot = torch.randint(-1, R + 2, (T, k), generator=g, dtype=torch.int32)
    slot[T // 2] = -1
    w = torch.rand(T, k, generator=g) - 0.3
    w[T // 2] = float("nan")                             # of dropped slots
    out = qg.combine_rows(Y.cuda(), slot.cuda(), w.cuda())
    torch.cuda.synchronize()
    ref, mag = torch.zeros(T, N, dtype=torch.float64), torch.zeros(T, N, dtype=torch.float64)
    for j in range(k):
        r = slot[:, j].long()
        live = (r >= 0) & (r < R)
        y = Y[r.clamp(0, R - 1)].double() * torch.where(live, w[:, j].double(), 0.0)[:, None]
        ref += y
        mag += y.abs()
    err = (out.cpu().double() - ref).abs()
    tol = HALF[dtype] * ref.abs() + 1.01 * k * 2.0**-24 * mag + 2.0**-25
    assert bool((err <= tol).all())
    assert not bool(out[T // 2].any())


def test_combine_unaligned_and_empty():
    Y = torch.randn(8 * 64 + 1, device="cuda").half()[1:].view(8, 64)      # a 2-byte address
    slot = torch.arange(8, dtype=torch.int32, device="cuda").view(4, 2)
    w = torch.ones(4, 2, device="cuda")
    out = qg.combine_rows(Y, slot, w)
    assert torch.equal(out, (Y[::2].float() + Y[1::2].float()).half())
    none = qg.combine_rows(Y[:0], torch.full((4, 2), -1, dtype=torch.int32, device="cuda"), w)
    assert none.shape == (4, 64) and not bool(none.any())
    assert qg.combine_rows(Y, slot[:0], w[:0]).shape == (0, 64)


def _weights(E, N, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    W = torch.randn(E, N, K, device="cuda", generator=g) * 0.05
    s = W.view(E, N // 128, 128, K // 128, 128).abs().amax((2, 4)) / 448
    q = (W.view(E, N // 128, 128, K // 128, 128) / s[:, :, None, :, None]).view(E, N, K)
    return q.to(torch.float8_e4m3fn), s.contiguous()


def _value(q, s):
    return q.double() * s.double().repeat_interleave(128, -2)[..., :q.shape[-2], :].repeat_interleave(128, -1)


def _moe(x, logits, bias, W1, S1, W2, S2, k):
    """A mixture-of-experts MLP as a program would run it."""
    E = W1.shape[0]
    ids, w = qg.route(logits, k, bias=bias, score="sigmoid", n_group=4, topk_group=2, group_score="top2", scaling=2.5)
    off, tok, slot = qg.sort_rows(ids, E)
    q, s = qg.quantize_fp8(x)
    gu = qg.fp8_gemm(q, s, W1, S1, expert_offsets=off, a_rows=tok)
    hq, hs = qg.quantize_fp8(gu, swiglu=True)
    y = qg.fp8_gemm(hq, hs, W2, S2, expert_offsets=off)
    return qg.combine_rows(y, slot, w), (ids, w, q, s)


@pytest.mark.parametrize("T", [1, 13, 300])
def test_mixture_of_experts_layer(T):
    """Every step against the formula from its inputs would hide a mistake
    between them; this holds the layer's output to the formula: sum over the
    chosen experts of w W2 (silu(Wg x) * Wu x), x and the weights the values of
    their codes.  What the steps round: the pair to bf16, the hidden row to
    e4m3 (half a step 2^-4 of a value, 2^-10 of a block's scale below), the
    experts' rows and the sum to bf16."""
    note(f"moe layer T={T}")
    E, D, F, k = 16, 256, 384, 4
    W1, S1 = _weights(E, 2 * F, D, 1)
    W2, S2 = _weights(E, D, F, 2)
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, D, device="cuda", generator=g).bfloat16()
    logits = torch.randn(T, E, device="cuda", generator=g)
    if T > 5:
        logits[5] = -INF                                   # a padded token
    bias = 0.1 * torch.randn(E, device="cuda", generator=g)
    out, (ids, w, q, s) = _moe(x, logits, bias, W1, S1, W2, S2, k)
    torch.cuda.synchronize()
    X = (q.double() * s.double().repeat_interleave(128, 1)).cpu()
    V1, V2 = _value(W1, S1).cpu(), _value(W2, S2).cpu()
    ids, w = ids.cpu(), w.cpu().double()
    b8 = 2.0**-8
    for t in range(T):
        ref, tol = torch.zeros(D, dtype=torch.float64), torch.zeros(D, dtype=torch.float64)
        for j in range(k):
            e = int(ids[t, j])
            if e < 0:
                continue
            pair = V1[e] @ X[t]
            # what the fp8 matrix instruction cuts (each product at most 2^-13 of the
            # largest of its eight, so 7 2^-13 of the magnitudes), and one bf16 rounding
            dp = b8 * pair.abs() + 1.01 * 7 * 2.0**-13 * (V1[e].abs() @ X[t].abs())
            gate, up, dg, du = pair[:F], pair[F:], dp[:F], dp[F:]
            h = gate * torch.sigmoid(gate) * up
            # |silu'| <= 1.1, |silu(x)| <= |x|
            dh = 1.1 * dg * (up.abs() + du) + gate.abs() * du + 2.0**-20 * h.abs()
            top = (h.abs() + dh).view(-1, 128).amax(1).repeat_interleave(128) / 448
            dh = dh + 2.0**-4 * (h.abs() + dh) + 2.0**-10 * top
            y = V2[e] @ h
            dy = (V2[e].abs() @ dh) * 1.001 + 1.01 * 7 * 2.0**-13 * (V2[e].abs() @ (h.abs() + dh)) + b8 * (y.abs() + V2[e].abs() @ dh)
            ref += w[t, j] * y
            tol += w[t, j] * dy
        err = (out[t].cpu().double() - ref).abs()
        assert bool((err <= tol + b8 * (ref.abs() + tol) + 1e-6).all()), t
    if T > 5:
        assert not bool(out[5].any())


def test_layer_in_a_graph():
    E, D, F, k, T = 16, 256, 384, 4, 40
    W1, S1 = _weights(E, 2 * F, D, 1)
    W2, S2 = _weights(E, D, F, 2)
    x = torch.randn(T, D, device="cuda").bfloat16()
    logits = torch.randn(T, E, device="cuda")
    bias = 0.1 * torch.randn(E, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _moe(x, logits, bias, W1, S1, W2, S2, k)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, _ = _moe(x, logits, bias, W1, S1, W2, S2, k)
    for rep in range(4):
        x.copy_(torch.randn(T, D, device="cuda").bfloat16())
        logits.copy_(torch.randn(T, E, device="cuda"))
        want, _ = _moe(x, logits, bias, W1, S1, W2, S2, k)
        junk = (torch.randn(256, 256, device="cuda") @ torch.randn(256, 256, device="cuda")).sum()
        g.replay()
        torch.cuda.synchronize()
        assert float(junk) == float(junk) and torch.equal(out, want), rep


def test_two_graphs_of_one_pool_replayed_together():
    """Two captured sorts replayed on two streams at once: each has its own
    workspace."""
    inputs, outs, graphs, refs = [], [], [], []
    for i in range(2):
        ids = torch.randint(0, 256, (9000 + i, 8), generator=torch.Generator().manual_seed(i), dtype=torch.int32).cuda()
        inputs.append(ids)
        qg.sort_rows(ids, 256)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(qg.sort_rows(ids, 256))
        graphs.append(g)
        refs.append([torch.from_numpy(np.ascontiguousarray(v)).int() for v in ref_sort(ids, 256)])
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, r in zip(outs, refs):
            assert all(torch.equal(a.cpu(), b) for a, b in zip(o, r))


def test_routed_rows_through_the_w4a8_product():
    """The same offsets and rows serve the int4 experts."""
    E, K, N, T, k = 4, 256, 256, 30, 2
    c = synth.w4a8_case(E, 16, K, N, 128, stream=7, case_id=1)
    packs = [qg.pack(dev(c.q[e]), dev(c.s[e]), None, 128, fold=True) for e in range(E)]
    W = torch.stack([p.w for p in packs]).contiguous()
    S = torch.stack([p.scale for p in packs]).contiguous()
    x = torch.randn(T, K, generator=torch.Generator().manual_seed(5)).half().cuda()
    ids, w = qg.route(logits_of(T, E, torch.float16, 6), k)
    off, tok, slot = qg.sort_rows(ids, E)
    q, s = qg.quantize_rows(x)
    rows = tok.long()
    y = qg.w4a8(q[rows].contiguous(), s[rows].contiguous(), W, S, off, E, T, N, 128)
    out = qg.combine_rows(y, slot, w)
    torch.cuda.synchronize()
    ref8, _ = oracle.w4a8(q[rows].cpu().numpy(), s[rows].cpu().numpy(), c.q, c.s, off.cpu().numpy(), 128)
    # as the W4A8 parity tests hold its rows, then the sum's own bound
    y64 = torch.from_numpy(np.asarray(ref8, dtype=np.float64))
    sl, w = slot.cpu().long(), w.cpu().double()
    ref = (y64[sl] * w[..., None]).sum(1)
    err = out.cpu().double() - ref
    assert float(err.norm() / ref.norm()) <= 1e-2
