"""Low-rank adapters on the GPU against 64 bits, and the run of a layer's attention half:
int4 projections with adapters around append and attention, eager and captured."""
import pytest
import torch

import int4_weight_only_uint32_amd as qg
from tests.gpu_util import note
from tests.kv4_util import angles, attend, rng

pytestmark = pytest.mark.gpu

HALF = {"fp16": torch.float16, "bf16": torch.bfloat16}


def reference(x, A, B, ids, y, scaling):
    """(out, tolerance) in 64 bits.  The tolerance adds up, for each value: its rounding (eps / 2
    of it); H's row entering as two 16-bit values (fp16 2^-24, bf16 2^-18 of each value, and
    2^-24 of the row's largest where the second one is subnormal); 32-bit sums: 2^-24 of the
    terms' sizes for each of K/32 + 40 additions in a row (and R/32 + 8 of the second product);
    the sum with y and the scaling, 2^-23 each."""
    out, tol = y.double().clone(), torch.zeros(y.shape, dtype=torch.float64)
    K, R = x.shape[1], A.shape[1]
    part = 2.0**-18 if x.dtype is torch.bfloat16 else 2.0**-24
    for t, a in enumerate(ids.tolist()):
        if not 0 <= a < A.shape[0]:
            continue
        s = float(scaling[a]) if scaling is not None else 1.0
        xt, Aa, Ba = x[t].double(), A[a].double(), B[a].double()
        h = Aa @ xt
        size = Aa.abs() @ xt.abs()
        dh = size * (K / 32 + 40) * 2.0**-24 + h.abs() * (part + 2.0**-23) + h.abs().max() * 2.0**-24
        d = Ba @ h * s
        out[t] += d
        tol[t] = abs(s) * (Ba.abs() @ dh + (Ba.abs() @ h.abs()) * (R / 32 + 8) * 2.0**-23) + 2.0**-23 * (d.abs() + out[t].abs())
    return out, tol + torch.finfo(x.dtype).eps / 2 * out.abs() * 1.01 + 1e-30


CASES = [
    # T, L, R, K, N, share without, scaling, type
    (1, 1, 8, 8, 8, 0.0, False, "fp16"),
    (1, 8, 16, 512, 256, 0.0, True, "bf16"),
    (5, 3, 16, 1000, 264, 0.3, True, "fp16"),
    (17, 2, 24, 520, 1288, 0.0, True, "bf16"),
    (64, 32, 16, 1024, 640, 0.1, True, "bf16"),
    (70, 5, 40, 136, 72, 0.0, False, "fp16"),
    (33, 1, 64, 2056, 512, 0.0, True, "bf16"),
    (40, 100, 8, 256, 128, 0.5, True, "fp16"),
    (20, 3, 128, 384, 320, 0.0, True, "bf16"),
    (9, 2, 512, 128, 128, 0.0, True, "fp16"),
    (300, 3, 16, 640, 1000, 0.1, True, "fp16"),
    (257, 2, 64, 520, 264, 0.0, True, "bf16"),
    (200, 2, 200, 256, 136, 0.0, True, "fp16"),
    (1000, 7, 32, 320, 200, 0.2, True, "bf16"),
    (12, 4, 16, 256, 128, 1.0, True, "bf16"),
]


def _inputs(T, L, R, K, N, none, scaling, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    dt = HALF[dtype]
    x = torch.randn((T, K), generator=gen).to(dt)
    A = (torch.randn((L, R, K), generator=gen) / K**0.5).to(dt)
    B = (0.1 * torch.randn((L, N, R), generator=gen)).to(dt)
    y = torch.randn((T, N), generator=gen).to(dt)
    ids = torch.randint(0, L, (T,), generator=gen)
    ids[torch.rand(T, generator=gen) < none] = -1
    s = torch.rand(L, generator=gen) + 0.5 if scaling else None
    return x, A, B, ids.to(torch.int32), y, s


def _plan(ids, L):
    return qg.sort_rows(ids.cuda()[:, None].contiguous(), L, row_token=torch.full((len(ids),), 1 << 20, dtype=torch.int32,
                                                                                device="cuda"))


def _cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


@pytest.mark.parametrize("T,L,R,K,N,none,scaling,dtype", CASES)
def test_lora(T, L, R, K, N, none, scaling, dtype):
    note(f"lora T={T} L={L} R={R} K={K} N={N} none={none} {dtype}")
    x, A, B, ids, y, s = _inputs(T, L, R, K, N, none, scaling, dtype, T + L + R)
    xd, Ad, Bd, yd, sd = _cuda(x, A, B, y, s)
    got = qg.lora(xd, Ad, Bd, _plan(ids, L), yd, scaling=sd)
    assert got is yd
    torch.cuda.synchronize()
    ref, tol = reference(x, A, B, ids, y, s)
    err = (got.cpu().double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    assert torch.equal(got.cpu()[ids < 0], y[ids < 0])
    # the same bits again
    yd.copy_(y)
    again = qg.lora(xd, Ad, Bd, _plan(ids, L), yd.clone(), scaling=sd)
    yd.copy_(y)
    assert torch.equal(qg.lora(xd, Ad, Bd, _plan(ids, L), yd, scaling=sd), again)


@pytest.mark.parametrize("size", [1e-7, 1e-3, 1e4])
def test_lora_sizes_of_the_narrow_product(size):
    """A product past fp16's range, and one below it, brought back by the scaling."""
    x, A, B, ids, y, s = _inputs(20, 2, 16, 256, 64, 0.0, True, "fp16", 3)
    x = (x.float() * min(size, 50.0)).half()
    A = (A.float() * max(size / 50.0, 1.0)).half()
    s = s / size
    ref, tol = reference(x, A, B, ids, y, s)
    xd, Ad, Bd, yd, sd = _cuda(x, A, B, y, s)
    got = qg.lora(xd, Ad, Bd, _plan(ids, 2), yd, scaling=sd)
    err = (got.cpu().double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


def test_lora_odd_plans():
    """Rows outside the tokens, a token named twice, offsets past the rows: each token is taken in
    the row that its slot names, others keep their y."""
    x, A, B, ids, y, s = _inputs(10, 3, 16, 128, 64, 0.0, True, "bf16", 4)
    off = torch.tensor([0, 4, 4, 30], dtype=torch.int32)
    rows = torch.tensor([0, 1, 1, -1, 7, 7, 99, 2, 3, 1 << 30], dtype=torch.int32)
    slots = torch.tensor([[0], [2], [7], [1], [-1], [5], [-1], [5], [3], [9]], dtype=torch.int32)
    want = torch.full((10,), -1)
    want[0], want[1], want[7], want[2] = 0, 0, 2, 2
    xd, Ad, Bd, yd, sd = _cuda(x, A, B, y, s)
    got = qg.lora(xd, Ad, Bd, (off.cuda(), rows.cuda(), slots.cuda()), yd, scaling=sd).cpu()
    ref, tol = reference(x, A, B, want, y, s)
    assert bool(((got.double() - ref).abs() <= tol).all())
    assert torch.equal(got[want < 0], y[want < 0])


def test_lora_no_numbers_stay_with_their_token():
    x, A, B, ids, y, s = _inputs(40, 2, 16, 256, 64, 0.0, True, "fp16", 5)
    x[3, 7] = float("nan")
    x[5, 9] = float("inf")
    xd, Ad, Bd, yd, sd = _cuda(x, A, B, y, s)
    got = qg.lora(xd, Ad, Bd, _plan(ids, 2), yd, scaling=sd).cpu()
    bad = ~torch.isfinite(got)
    assert bool(bad[3].all()) and bool(bad[5].any()) and not bool(bad[[i for i in range(40) if i not in (3, 5)]].any())


class Layer:
    """A layer's attention half: qkv and output projections of int4 weights with adapters,
    rotation, the 4-bit cache and attention over it."""

    def __init__(self, width=512, H=2, R=2, D=128, L=3, rank=16, B=4, page=32, pages=24):
        gen = torch.Generator().manual_seed(21)
        self.H, self.R, self.D = H, R, D

        def weight(K, N):
            q = torch.randint(0, 16, (K, N), generator=gen, dtype=torch.uint8)
            s = (0.01 + 0.01 * torch.rand((K // 128, N), generator=gen)).half()
            z = (-7.5 * s.float() + 0.01 * torch.randn((K // 128, N), generator=gen)).half()
            return qg.pack(q.cuda(), s.cuda(), z.cuda(), 128)

        def adapter(K, N):
            return ((torch.randn((L, rank, K), generator=gen) / K**0.5).half().cuda(),
                    (0.1 * torch.randn((L, N, rank), generator=gen)).half().cuda())

        self.n_qkv = (R + 2) * H * D
        self.wqkv, self.wo = weight(width, self.n_qkv), weight(R * H * D, width)
        self.aqkv, self.ao = adapter(width, self.n_qkv), adapter(R * H * D, width)
        self.L, self.cs = L, angles(page * 8, D).cuda()
        self.cache = qg.kv4_cache(pages, H, D, page, 64)
        order = torch.randperm(pages, generator=gen).to(torch.int32)
        self.table = order[:B * (pages // B)].view(B, -1).contiguous().cuda()

    def run(self, x, ids, lens, off=None, max_new=None, window=0, sinks=0):
        H, R, D = self.H, self.R, self.D
        plan = qg.sort_rows(ids, self.L)
        qkv = qg.lora(x, *self.aqkv, plan, qg.w4a16(x, self.wqkv))
        q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([R * H * D, H * D, H * D], 1))
        q = qg.kv4_append(self.cache, k, v, lens, self.table, seq_offsets=off, cos_sin=self.cs, q=q)
        o = qg.kv4_attend(q, self.cache, lens, self.table, seq_offsets=off, max_new=max_new, window=window, sinks=sinks)
        o = o.flatten(1)
        return qg.lora(o, *self.ao, plan, qg.w4a16(o, self.wo)), qkv, q, o


def test_layer_prefill_then_decode():
    """Each step of the layer from the inputs that the step before gave: attention's output
    against 64 bits on the cache's own contents, the adapters' against theirs."""
    layer = Layer()
    rnd, gen = rng(22)
    lens = torch.tensor([40, 1, 77, 100], dtype=torch.int32)
    news = [40, 1, 77, 100]
    off = torch.tensor([0, 40, 41, 118, 218], dtype=torch.int32)
    for step in range(3):
        T = int(off[-1])
        x = torch.randn((T, 512), generator=gen).half()
        ids = torch.randint(-1, 3, (T, 1), generator=gen, dtype=torch.int32)
        y, qkv, q, o = layer.run(x.cuda(), ids.cuda(), lens.cuda(), off.cuda() if step == 0 else None,
                                 max(news) if step == 0 else None, window=60, sinks=4)
        ref, tol = attend(q.cpu(), layer.cache, lens, off, layer.table.cpu(), 128 ** -0.5, 60, 4)
        err = (o.cpu().double().view_as(ref) - ref).abs()
        assert bool((err <= tol).all()), (step, float((err / tol).max()))
        plain = qg.w4a16(o, layer.wo).cpu()
        ref, tol = reference(o.cpu(), *(t.cpu() for t in layer.ao), ids[:, 0], plain, None)
        assert bool(((y.cpu().double() - ref).abs() <= tol).all())
        lens, news, off = lens + 1, [1] * 4, torch.arange(5, dtype=torch.int32)


def test_layer_in_a_graph():
    """Decode steps captured once and replayed with new inputs and lengths in place, with eager
    work between; each replay bit for bit the eager run on a copy of the cache.  Two graphs
    captured side by side, replayed in turn, do not disturb each other."""
    layer = Layer()
    gen = torch.Generator().manual_seed(23)
    lens0 = torch.tensor([40, 7, 77, 100], dtype=torch.int32)
    x = torch.randn((4, 512), generator=gen).half().cuda()
    ids = torch.tensor([[0], [2], [-1], [1]], dtype=torch.int32).cuda()
    lens = lens0.cuda()
    fill = torch.randn((226, 2, 128), generator=gen).half().cuda()
    off = torch.tensor([0, 40, 47, 124, 224], dtype=torch.int32).cuda()
    qg.kv4_append(layer.cache, fill[:224], fill[:224], lens, layer.table, seq_offsets=off, cos_sin=layer.cs)
    start = [t.clone() for t in (layer.cache.k, layer.cache.v, layer.cache.k_sz, layer.cache.v_sz)]

    def reset():
        for t, s in zip((layer.cache.k, layer.cache.v, layer.cache.k_sz, layer.cache.v_sz), start):
            t.copy_(s)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.run(x, ids, lens)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(layer.run(x, ids, lens)[0])
        graphs.append(g)
    reset()
    inputs = [torch.randn((4, 512), generator=gen).half().cuda() for _ in range(4)]
    want = []
    for i, xi in enumerate(inputs):
        x.copy_(xi)
        lens.copy_(lens0 + 1 + i)
        want.append(layer.run(x, ids, lens)[0].clone())
    end = [t.clone() for t in (layer.cache.k, layer.cache.v, layer.cache.k_sz, layer.cache.v_sz)]
    reset()
    for i, xi in enumerate(inputs):
        x.copy_(xi)
        lens.copy_(lens0 + 1 + i)
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i % 2], want[i]), i
        (torch.randn((64, 64), device="cuda") @ torch.randn((64, 64), device="cuda")).sum().item()
    for t, e in zip((layer.cache.k, layer.cache.v, layer.cache.k_sz, layer.cache.v_sz), end):
        assert torch.equal(t, e)
