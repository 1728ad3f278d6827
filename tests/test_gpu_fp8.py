"""GPU parity of the fp8 row quantizer and the block-scaled fp8 GEMM against
plain 64-bit computations.

Tolerances.  Codes and scales are the definition's own (bit-exact).

The e4m3 matrix instruction adds eight products of consecutive k at a time,
each cut (toward zero) to a multiple of 2^(e - 13), e the largest exponent sum
of the eight pairs (a subnormal code counts with exponent -6): up to seven
products lose up to 2^-13 of that power of two each, which the largest of the
products of the magnitudes, subnormal ones raised to 2^-6, bounds.  The sums of
the sixteen eights of a block keep 24 bits, cut as well (2^-23 of the
magnitudes each), then a scale product, one FMA a block (2^-24 each) and
one rounding of the output, half a step."""
import numpy as np
import pytest
import torch

import int4_weight_only_uint32_amd as qg
from tests.gpu_util import note

pytestmark = pytest.mark.gpu

HALF = {torch.float16: 2.0**-11, torch.bfloat16: 2.0**-8}
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available()
    assert qg.qg_device_supported(0), "GPU visible but not gfx950"
    torch.cuda.set_device(0)


def kb(n):
    return -(-n // 128)


def ref_quant(x64):
    """Codes (as values) and scales of [M,K] by the definition, on the CPU:
    each quotient rounded once to 32 bits."""
    M, K = x64.shape
    p = torch.zeros(M, kb(K) * 128, dtype=torch.float64)
    p[:, :K] = x64
    p = p.view(M, kb(K), 128)
    s = (p.abs().amax(2) / 448.0).float()
    q = (p / s.double()[..., None]).float()
    q = torch.where(s[..., None] == 0, torch.zeros_like(q), q).clamp(-448, 448)
    return q.to(F8).double().view(M, -1)[:, :K], s


def rows(M, K, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    mag = 10.0 ** (torch.rand(M, 1, generator=g) * 6 - 4)
    x = (torch.randn(M, K, generator=g) * mag).to(dtype)
    if M >= 7:
        x[0] = 0
        x[1] = 0
        x[1, K // 2] = -3.0
        x[2] = torch.finfo(dtype).tiny / 4 if dtype == torch.float16 else 1e-39
        x[3] = 448.0                                     # scale 1: codes are the values
        x[3, : K // 2] = (torch.arange(K // 2) % 449).to(dtype)   # with exact ties
        x[4] = -1.5
        x[5, : min(K, 128)] = 0                          # a block of zeros in a live row
        x[6] = torch.finfo(dtype).max
    return x


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("M,K", [(1, 16), (1, 128), (3, 144), (7, 112), (16, 5120), (9, 17408), (257, 2064),
                                 (1030, 1024), (33, 40000)])
def test_quantize_bit_exact(M, K, dtype):
    note(f"quantize_fp8 M={M} K={K} {dtype}")
    x = rows(M, K, dtype, M + K)
    q, s = qg.quantize_fp8(x.cuda())
    torch.cuda.synchronize()
    rq, rs = ref_quant(x.double())
    assert torch.equal(s.cpu(), rs)
    assert torch.equal(q.cpu().double(), rq)


def test_quantize_non_finite_blocks():
    x = torch.randn(4, 300 // 4 * 4 + 4, generator=torch.Generator().manual_seed(1)).bfloat16()[:, :288].contiguous()
    x[0, 5] = float("nan")
    x[1, 130] = float("inf")
    x[2, 287] = -float("inf")
    q, s = qg.quantize_fp8(x.cuda())
    torch.cuda.synchronize()
    bad = torch.zeros(4, 3, dtype=torch.bool)
    bad[0, 0] = bad[1, 1] = bad[2, 2] = True
    assert torch.equal(s.cpu().isnan(), bad)
    assert torch.equal(q.cpu().float().isnan(), bad.repeat_interleave(128, 1)[:, :288])
    x[bad.repeat_interleave(128, 1)[:, :288]] = 0
    rq, rs = ref_quant(x.double())
    ok = ~bad.repeat_interleave(128, 1)[:, :288]
    assert torch.equal(q.cpu().float().nan_to_num(0)[ok].double(), rq[ok])


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("M,K", [(1, 16), (5, 144), (64, 2048), (300, 1040)])
def test_quantize_swiglu(M, K, dtype):
    note(f"quantize_fp8 swiglu M={M} K={K} {dtype}")
    g = torch.Generator().manual_seed(M * K)
    x = (3 * torch.randn(M, 2 * K, generator=g)).to(dtype)
    x[0, :16] = torch.tensor([-200.0, -100, -90, -30, -1, 0, 1e-4, 1, 30, 90, 100, 200, -88, 88, -0.0, 5]).to(dtype)
    q, s = qg.quantize_fp8(x.cuda(), swiglu=True)
    torch.cuda.synchronize()
    gate, up = x.double().chunk(2, 1)
    rq, rs = ref_quant(gate * torch.sigmoid(gate) * up)
    assert torch.equal(s.cpu(), rs)
    assert torch.equal(q.cpu().double(), rq)


def test_quantize_swiglu_many_values():
    """Enough values that silu in 32 bits alone would move some codes and
    most scales; blocks of equal magnitudes and of zeros among them."""
    M, K = 2000, 2064
    g = torch.Generator().manual_seed(3)
    x = (2 * torch.randn(M, 2 * K, generator=g)).bfloat16()
    x[7, :128] = 1.5
    x[7, K:K + 128] = torch.where(torch.arange(128) % 2 == 0, 2.0, -2.0).bfloat16()
    x[8, 128:256] = 0
    x[9, K:K + 128] = 0
    q, s = qg.quantize_fp8(x.cuda(), swiglu=True)
    torch.cuda.synchronize()
    gate, up = x.double().chunk(2, 1)
    rq, rs = ref_quant(gate * torch.sigmoid(gate) * up)
    assert torch.equal(s.cpu(), rs)
    assert torch.equal(q.cpu().double(), rq)


def test_quantize_swiglu_non_finite_and_far_gates():
    x = torch.randn(6, 512, generator=torch.Generator().manual_seed(4)).half()
    x[0, 3] = float("nan")
    x[1, 256 + 200] = float("inf")
    x[2, :128] = -1000.0                        # silu 0
    x[3, :128] = -60.0
    x[4, :128] = 60000.0                        # up to the largest products
    x[4, 256:384] = 60000.0
    q, s = qg.quantize_fp8(x.cuda(), swiglu=True)
    torch.cuda.synchronize()
    q, s = q.cpu().double(), s.cpu()
    assert bool(q[0, :128].isnan().all()) and bool(q[1, 128:].isnan().all()) and int(s.isnan().sum()) == 2
    assert not bool(q[2, :128].any()) and float(s[2, 0]) == 0
    gate, up = x.double().chunk(2, 1)
    rq, rs = ref_quant((gate * torch.sigmoid(gate) * up).nan_to_num(0, 0, 0))
    for r, c in ((0, 1), (1, 0), (2, 1), (3, 0), (3, 1), (4, 0), (4, 1), (5, 0), (5, 1)):
        assert float(s[r, c]) == float(rs[r, c]), (r, c)
        assert torch.equal(q[r, 128 * c:128 * c + 128], rq[r, 128 * c:128 * c + 128]), (r, c)


@pytest.mark.parametrize("far", [-60.0, -86.5, -87.5, -88.5, -95.0, -120.0, 1e-37, -1e-37, 9e-40])
def test_quantize_swiglu_gates_that_only_the_product_raises(far):
    """silu(gate) near or under the least 32-bit value, times a bf16 up value as
    large as the type's: an ordinary product.  In every position of a block, as
    its only value, among ordinary ones, and with a small up value (a product that
    32 bits hold with few bits or not at all)."""
    far = float(torch.tensor(far).bfloat16())
    K, n = 128, 24
    gate, up = torch.zeros(6 * n, K), torch.zeros(6 * n, K)
    g = torch.Generator().manual_seed(int(abs(far) * 8) + 1)
    silu = abs(far / (1.0 + np.exp(-far)))
    for i in range(n):
        at = (5 * i) % K
        gate[6 * i:6 * i + 6, at] = far
        gate[6 * i + 1], up[6 * i + 1] = torch.randn(2, K, generator=g)
        gate[6 * i + 1, at] = far
        gate[6 * i + 4] = far
        gate[6 * i + 5] = far
        most = 1e38 * (i + 1) / n * 3
        up[6 * i, at] = most
        up[6 * i + 1, at] = min(most, (i + 1) / 8.0 / silu)    # about as large as the others
        up[6 * i + 2, at] = 1e-3 * (i + 1)
        up[6 * i + 3, at] = min(most, 2.0 ** (-150 + i) / silu)
        up[6 * i + 4] = torch.randn(K, generator=g) * min(1e37, 1e3 / silu)
        up[6 * i + 5] = torch.randn(K, generator=g) * min(1e37, 1e-41 / silu)
    x = torch.cat([gate, up], 1).bfloat16()
    q, s = qg.quantize_fp8(x.cuda(), swiglu=True)
    torch.cuda.synchronize()
    gate, up = x.double().chunk(2, 1)
    rq, rs = ref_quant(gate / (1.0 + torch.exp(-gate)) * up)
    assert torch.equal(s.cpu(), rs)
    assert torch.equal(q.cpu().double(), rq)


def codes(shape, seed, scale=1.0):
    """Random codes (on the GPU) and their values."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, device="cuda", generator=g) * 30 * scale).clamp(-448, 448).to(F8)


def scales(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand(shape, device="cuda", generator=g) * 0.02 + 0.001


def dequant(a, sa, w, sw):
    """Values of the operands, and the magnitudes that bound what the matrix
    instruction cuts (codes below 2^-6 raised to it)."""
    K, N = a.shape[1], w.shape[0]
    fa = sa.double().repeat_interleave(128, 1)[:, :K]
    fw = sw.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    av, wv = a.double(), w.double()
    up = lambda v: torch.where(v != 0, v.abs().clamp_min(2.0**-6), 0.0)
    return (av * fa).cpu(), (wv * fw).cpu(), (up(av) * fa).float(), (up(wv) * fw).float()


def check(got, A, W, A6, W6, dtype):
    M, K = A.shape
    ref, mag = A @ W.t(), A.abs() @ W.abs().t()
    err = (got.cpu().double() - ref).abs()
    eights = torch.zeros(M, W.shape[0], device="cuda")
    for k in range(0, K, 8):
        eights += torch.stack([A6[:, i, None] * W6[None, :, i] for i in range(k, k + 8)]).amax(0)
    wide = 7 * 2.0**-13 * 1.001 * eights.cpu().double() + (16 + 2 + kb(K)) * 2.0**-23 * mag
    tol = HALF[dtype] * ref.abs() + wide * (1 + HALF[dtype])
    if dtype == torch.float16:
        tol = tol + 2.0**-25            # half a step of the subnormals
    worst = float((err - tol).max())
    assert worst <= 0, f"{worst:.3e} beyond the bound, at {int((err - tol).argmax())}"


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 16), (1, 128, 128), (1, 513, 1024), (2, 130, 112), (5, 7, 144), (15, 256, 256), (16, 1000, 640),
    (17, 129, 2064), (31, 96, 384), (33, 255, 1152), (64, 64, 4096), (65, 128, 128), (100, 1027, 528), (127, 640, 272),
    (130, 132, 1280), (200, 2050, 640), (257, 260, 512), (300, 516, 2048), (513, 1030, 400)])
def test_dense(M, N, K, dtype):
    note(f"fp8_gemm M={M} N={N} K={K} {dtype}")
    a, w = codes((M, K), 1), codes((N, K), 2)
    sa, sw = scales((M, kb(K)), 3), scales((kb(N), kb(K)), 4)
    C = torch.full((M, N), float("nan"), dtype=dtype, device="cuda")
    qg.fp8_gemm(a, sa, w, sw, C=C)
    torch.cuda.synchronize()
    check(C, *dequant(a, sa, w, sw), dtype)


# shapes for every kernel that the rule on rows and workgroups can choose, on
# both sides of its thresholds (rows 16, 32, 64, 128; workgroups 128, 192, 256, 2048;
# K 4096), with one k block, odd numbers of them and partial ones
WIDE = [
    (3, 65540, 272), (16, 65600, 4112), (9, 4100, 4112), (16, 4096, 1040), (20, 65600, 272), (32, 70000, 144),
    (40, 4100, 272), (64, 5120, 4240), (100, 4100, 4240), (128, 2050, 1168), (50, 16500, 400), (64, 20000, 128),
    (128, 8200, 656), (100, 17408, 1296), (128, 20000, 80), (200, 3000, 2000), (300, 3000, 112), (290, 5000, 656),
    (256, 8192, 784), (300, 17000, 400), (300, 17000, 4112), (512, 9000, 128), (500, 8200, 912), (700, 2050, 1152), (2000, 4096, 272),
    (260, 17500, 272), (512, 17408, 5120), (1025, 8196, 656), (1300, 6000, 400), (900, 4700, 144),
    (40, 33500, 144), (100, 33500, 272), (100, 50257, 2064),
    # columns left over from whole rounds, few to many
    (1000, 17500, 272), (1024, 17408, 144), (1000, 19500, 272), (1024, 21900, 144), (16500, 1000, 144),
    (1024, 26000, 144)]


@pytest.mark.parametrize("M,N,K", WIDE)
def test_dense_wide(M, N, K):
    note(f"fp8_gemm M={M} N={N} K={K}")
    a, w = codes((M, K), 1), codes((N, K), 2)
    sa, sw = scales((M, kb(K)), 3), scales((kb(N), kb(K)), 4)
    C = torch.full((M, N), float("nan"), dtype=torch.float16, device="cuda")
    qg.fp8_gemm(a, sa, w, sw, C=C)
    torch.cuda.synchronize()
    # every column block's edge and a stretch of each, to keep the 64-bit product small
    cols = torch.cat([torch.arange(0, 260), torch.arange(N // 2, N // 2 + 130), torch.arange(N - 261, N)])
    part = (cols // 128).cuda()
    cols = cols.cuda()
    assert bool(C.isfinite().all())
    A = a.double() * sa.double().repeat_interleave(128, 1)[:, :K]
    fw = sw[part].double().repeat_interleave(128, 1)[:, :K]
    wv, av = w[cols].double(), a.double()
    up = lambda v: torch.where(v != 0, v.abs().clamp_min(2.0**-6), 0.0)
    fa = sa.double().repeat_interleave(128, 1)[:, :K]
    check(C[:, cols], A.cpu(), (wv * fw).cpu(), (up(av) * fa).float(), (up(wv) * fw).float(), torch.float16)


@pytest.mark.parametrize("M,N,K", [(3, 130, 272), (70, 260, 640), (300, 384, 1152)])
def test_exact_on_small_integers(M, N, K):
    """Codes -4..4 and power-of-two scales: every sum is exact, so is C."""
    g = torch.Generator(device="cuda").manual_seed(5)
    a = torch.randint(-4, 5, (M, K), device="cuda", generator=g).float().to(F8)
    w = torch.randint(-4, 5, (N, K), device="cuda", generator=g).float().to(F8)
    sa = 2.0 ** torch.randint(-2, 1, (M, kb(K)), device="cuda", generator=g).float()
    sw = 2.0 ** torch.randint(-2, 1, (kb(N), kb(K)), device="cuda", generator=g).float()
    C = qg.fp8_gemm(a, sa, w, sw, dtype=torch.float16)
    torch.cuda.synchronize()
    A, W = dequant(a, sa, w, sw)[:2]
    assert torch.equal(C.cpu(), (A @ W.t()).half())


def offsets_of(counts, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(counts)]).astype(np.int32), device="cuda")


GROUPED = [
    # (counts of each expert, N, K, rows of A, first row, rows behind the last expert)
    ([1], 128, 128, 1, 0, 0),
    ([0, 1, 0, 2, 0], 130, 144, 4, 0, 0),
    ([3, 0, 17, 64, 65, 1, 0, 40], 260, 640, 60, 0, 5),
    ([0] * 70 + [5] + [0] * 70 + [1, 2] + [0] * 60, 96, 256, 8, 2, 3),
    ([1] * 200, 64, 256, 20, 0, 0),
    ([300, 0, 257, 1], 132, 400, 128, 0, 1),
    ([0, 0, 0], 64, 128, 4, 0, 6),
    ([129, 128, 127, 200, 90, 333], 516, 512, 700, 0, 0),
    # the same, large enough for the large tile and the streaming kernels of many workgroups
    ([129, 0, 700, 200, 90, 333], 8200, 272, 700, 3, 2),
    ([1, 2, 3, 0, 16, 17, 5, 9], 16400, 272, 40, 0, 1),
    ([30, 20, 31, 0, 70, 17, 5, 9], 16400, 144, 40, 0, 1),
    # few rows an expert on the large tile; experts of more row blocks than one band, large tile and small
    ([64, 1, 0, 65, 128, 257, 100, 140], 7300, 2064, 300, 1, 2),
    ([1700, 5, 300], 8200, 144, 900, 0, 3),
    ([0] * 12 + [1700] + [0] * 17, 600, 144, 400, 0, 0),
]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("case", range(len(GROUPED)))
@pytest.mark.parametrize("gather", [False, True])
def test_grouped(case, gather, dtype):
    counts, N, K, Ma, first, tail = GROUPED[case]
    E, M = len(counts), sum(counts) + first + tail
    note(f"fp8_gemm grouped case {case} E={E} M={M} N={N} K={K} gather={gather} {dtype}")
    Ma = Ma if gather else M
    a, w = codes((Ma, K), 1), codes((E, N, K), 2)
    sa, sw = scales((Ma, kb(K)), 3), scales((E, kb(N), kb(K)), 4)
    off = offsets_of(counts, first)
    idx = None
    if gather:
        idx = torch.randint(0, Ma, (M,), generator=torch.Generator().manual_seed(6), dtype=torch.int32)
        if M > 3:
            idx[first + sum(counts) // 2] = Ma          # outside: a row of zeros
            idx[first] = -1
        idx = idx.cuda()
    C = torch.full((M, N), 7.0, dtype=dtype, device="cuda")
    qg.fp8_gemm(a, sa, w, sw, expert_offsets=off, a_rows=idx, C=C)
    torch.cuda.synchronize()
    o = off.tolist()
    assert bool((C[:first] == 7).all()) and bool((C[o[-1]:] == 7).all())
    for e in range(E):
        if o[e] == o[e + 1]:
            continue
        r = torch.arange(o[e], o[e + 1], device="cuda") if idx is None else idx[o[e]:o[e + 1]].long()
        out = (r < 0) | (r >= Ma)
        r = r.clamp(0, Ma - 1)
        A, W, A6, W6 = dequant(a[r], sa[r], w[e], sw[e])
        A[out.cpu()] = 0
        check(C[o[e]:o[e + 1]], A, W, A6, W6, dtype)
        assert bool((C[o[e]:o[e + 1]][out] == 0).all())


def test_gather_without_experts():
    a, w = codes((5, 256), 1), codes((96, 256), 2)
    sa, sw = scales((5, 2), 3), scales((1, 2), 4)
    idx = torch.tensor([4, 4, 0, 2, 9, 1, 1], dtype=torch.int32, device="cuda")
    C = qg.fp8_gemm(a, sa, w, sw, a_rows=idx, dtype=torch.float16)
    torch.cuda.synchronize()
    rows_of = torch.tensor([4, 4, 0, 2, 0, 1, 1], device="cuda")
    A, W, A6, W6 = dequant(a[rows_of], sa[rows_of], w, sw)
    A[4] = 0
    check(C, A, W, A6, W6, torch.float16)


def test_offsets_that_are_no_offsets_stay_in_bounds():
    """Offsets beyond the rows are clipped, decreasing ones give empty experts."""
    a, w = codes((40, 128), 1), codes((4, 64, 128), 2)
    sa, sw = scales((40, 1), 3), scales((4, 1, 1), 4)
    off = torch.tensor([-5, 10, 4, 1000, 20], dtype=torch.int32, device="cuda")
    C = torch.full((40, 64), 7.0, dtype=torch.float16, device="cuda")
    qg.fp8_gemm(a, sa, w, sw, expert_offsets=off, C=C)
    torch.cuda.synchronize()
    check(C[:4], *dequant(a[:4], sa[:4], w[0], sw[0]), torch.float16)
    assert bool(C.isfinite().all())


def test_nan_stays_in_its_row():
    for M in (4, 40, 300):
        a, w = codes((M, 400), 1), codes((260, 400), 2)
        sa, sw = scales((M, 4), 3), scales((3, 4), 4)
        sa[1, 3] = float("nan")
        b = a.view(torch.uint8)
        b[2, 399] = 0x7F                                # the row before and behind a K tail stay clean
        C = qg.fp8_gemm(a, sa, w, sw)
        torch.cuda.synchronize()
        bad = torch.zeros(M, dtype=torch.bool, device="cuda")
        bad[1:3] = True
        assert bool(C[bad].isnan().all()) and not bool(C[~bad].isnan().any())


def test_empty_batch():
    a, w = codes((0, 128), 1), codes((2, 64, 128), 2)
    C = qg.fp8_gemm(a, scales((0, 1), 3), w, scales((2, 1, 1), 4),
                    expert_offsets=torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert C.shape == (0, 64)
    q, s = qg.quantize_fp8(torch.zeros(0, 256, dtype=torch.float16, device="cuda"))
    assert q.shape == (0, 256) and s.shape == (0, 2)


def test_weights_past_32_bit_offsets():
    """The last of five 1 GiB experts: its codes start 4 GiB in."""
    E, N, K = 5, 65536, 16384
    w = torch.zeros((E, N, K), dtype=torch.uint8, device="cuda").view(F8)
    part = codes((128, K), 2)
    w[4, N - 128:] = part
    sw = torch.full((E, N // 128, K // 128), 0.5, device="cuda")
    for M in (3, 70):
        a, sa = codes((M, K), 1), scales((M, K // 128), 3)
        off = torch.tensor([0, 0, 1, 1, 1, M], dtype=torch.int32, device="cuda")
        C = qg.fp8_gemm(a, sa, w, sw, expert_offsets=off)
        torch.cuda.synchronize()
        check(C[1:, N - 128:], *dequant(a[1:], sa[1:], part, sw[4, :1]), torch.bfloat16)
        assert not bool(C[:, :N - 128].any()) and not bool(C[0].any())


def test_outputs_and_rows_past_32_bit_offsets():
    """C of 2.1e9 elements; a gather from 4.28e9 bytes of codes."""
    M, N = 131073, 16400
    a, w = codes((M, 16), 1), codes((N, 16), 2)
    sa, sw = scales((M, 1), 3), scales((kb(N), 1), 4)
    C = qg.fp8_gemm(a, sa, w, sw, dtype=torch.float16)
    torch.cuda.synchronize()
    for r in (0, 65535, 131000):
        check(C[r:r + 73], *dequant(a[r:r + 73], sa[r:r + 73], w, sw), torch.float16)
    del C
    # 4.4e9 bytes of codes with a partial last k block: what lies behind it reads as
    # zeros for the first rows too
    M, K = 1060000, 4112
    a = torch.zeros((M, K), dtype=torch.uint8, device="cuda")
    a.view(-1)[2**32 - 2**23:] = 0x7F                # (NaN codes where a far offset could land)
    part = codes((300, K), 11)
    a[:300] = part.view(torch.uint8)
    a[-300:] = part.view(torch.uint8)
    sa, w, sw = torch.full((M, kb(K)), 0.25, device="cuda"), codes((16, K), 12), scales((1, kb(K)), 13)
    C = qg.fp8_gemm(a.view(F8), sa, w, sw)
    torch.cuda.synchronize()
    for r in (slice(0, 300), slice(M - 300, M)):
        check(C[r], *dequant(part, sa[:300], w, sw), torch.bfloat16)
    del a, sa, C
    Ma, K = 2**20, 4080
    a = torch.zeros((Ma, K), dtype=torch.uint8, device="cuda").view(F8)
    a[-9:] = codes((9, K), 7)
    sa = torch.full((Ma, kb(K)), 0.25, device="cuda")
    w, sw = codes((64, K), 8), scales((1, kb(K)), 9)
    idx = torch.arange(Ma - 1, Ma - 12, -1, dtype=torch.int32, device="cuda")
    for reps in (1, 9):
        C = qg.fp8_gemm(a, sa, w, sw, a_rows=idx.repeat(reps))
        torch.cuda.synchronize()
        r = idx.long().repeat(reps)
        check(C, *dequant(a[r], sa[r], w, sw), torch.bfloat16)


@pytest.mark.parametrize("M", [1, 16, 200, 700])
def test_repeats_graphs_and_streams_agree(M):
    K, N = 1040, 1028
    a, w = codes((M, K), 1), codes((N, K), 2)
    sa, sw = scales((M, kb(K)), 3), scales((kb(N), kb(K)), 4)
    x = torch.randn(M, K, device="cuda").half()
    q, s = qg.quantize_fp8(x)
    C = qg.fp8_gemm(a, sa, w, sw)
    torch.cuda.synchronize()
    first = [t.clone() for t in (q, s, C)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        D = qg.fp8_gemm(a, sa, w, sw)
    torch.cuda.synchronize()
    assert torch.equal(C, D)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qg.quantize_fp8(x, A_q=q, a_scale=s)
        qg.fp8_gemm(a, sa, w, sw, C=C)
    for _ in range(3):
        for t in (q.view(torch.uint8), s, C):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for t, f in zip((q, s, C), first):
            assert torch.equal(t.view(torch.uint8), f.view(torch.uint8))


def test_unaligned_output_rows():
    """C at an odd 2-byte address and N % 4 != 0: no wide stores, nothing
    beyond the rows is touched."""
    for M, N in ((3, 128), (70, 128), (300, 258)):
        a, w = codes((M, 256), 1), codes((N, 256), 2)
        sa, sw = scales((M, 2), 3), scales((kb(N), 2), 4)
        buf = torch.full((M * N + 9,), 7.0, dtype=torch.float16, device="cuda")
        C = buf[1:1 + M * N].view(M, N)
        qg.fp8_gemm(a, sa, w, sw, C=C)
        torch.cuda.synchronize()
        check(C, *dequant(a, sa, w, sw), torch.float16)
        assert float(buf[0]) == 7 and bool((buf[1 + M * N:] == 7).all())


def test_binding_refusals():
    a, w = codes((4, 256), 1), codes((64, 256), 2)
    sa, sw = scales((4, 2), 3), scales((1, 2), 4)
    with pytest.raises(ValueError):
        qg.fp8_gemm(a, sa[:, :1], w, sw)                      # strided and too small
    with pytest.raises(ValueError):
        qg.fp8_gemm(a[:, ::2], sa, w, sw)
    with pytest.raises(ValueError):
        qg.fp8_gemm(a, sa, w, sw.repeat(2, 1))
    with pytest.raises(ValueError):
        qg.fp8_gemm(a, sa, w, sw, C=torch.empty(4, 63, device="cuda", dtype=torch.float16))
    with pytest.raises(TypeError):
        qg.fp8_gemm(a.view(torch.uint8), sa, w, sw)
    with pytest.raises(TypeError):
        qg.fp8_gemm(a, sa, w, sw, a_rows=torch.zeros(4, dtype=torch.int64, device="cuda"))
    with pytest.raises(qg.QGemmError):
        qg.quantize_fp8(torch.zeros(2, 24, device="cuda").half())
