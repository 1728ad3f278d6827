"""CPU checks of the fp8 and expert-routing entry points: bad arguments are
refused on the host before a device is touched, valid ones reach the device
check, empty batches succeed, and the binding checks types, shapes and
devices.  No kernel runs here."""
import ctypes

import pytest
import torch

import int4_weight_only_uint32_amd as qg

P = ctypes.c_void_p
FAKE = P(0x10000)     # never dereferenced
OK, INV, UNS, WSP, DEV = (qg.QG_OK, qg.QG_ERR_INVALID_ARG, qg.QG_ERR_UNSUPPORTED, qg.QG_ERR_WORKSPACE,
                          qg.QG_ERR_DEVICE)

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake pointers: only where no kernel can start")


def _quant(A=FAKE, dtype=qg.QG_DTYPE_BF16, M=4, K=256, flags=0, q=FAKE, s=FAKE):
    return qg.lib().quantize_rows_fp8(A, dtype, M, K, flags, q, s, None)


@no_gpu
@pytest.mark.parametrize("kw,rc", [
    (dict(), DEV), (dict(flags=qg.QG_QUANT_SWIGLU), DEV), (dict(K=16), DEV), (dict(K=144), DEV),
    (dict(M=0, A=None, q=None, s=None), OK),
    (dict(M=-1), INV), (dict(K=0), INV), (dict(K=8), UNS), (dict(K=129), UNS),
    (dict(dtype=qg.QG_DTYPE_F32), INV), (dict(dtype=9), INV), (dict(flags=2), INV),
    (dict(A=None), INV), (dict(q=None), INV), (dict(s=None), INV),
    (dict(A=P(0x10008)), INV), (dict(q=P(0x10008)), INV), (dict(s=P(0x10002)), INV),
    (dict(M=2**31 - 1, K=16 * 2**20), UNS), (dict(M=2**29, K=128), UNS),
])
def test_quantize_rows_fp8_refusals(kw, rc):
    assert _quant(**kw) == rc
    assert rc == OK or qg.lib().qg_last_error()


def _gemm(A=FAKE, sa=FAKE, rows=None, Ma=8, W=FAKE, sw=FAKE, off=None, E=1, M=8, N=256, K=256,
          dtype=qg.QG_DTYPE_F16, C=FAKE, flags=0):
    return qg.lib().qgemm_fp8(A, sa, rows, Ma, W, sw, off, E, M, N, K, dtype, C, None, 0, flags, None)


@no_gpu
@pytest.mark.parametrize("kw,rc", [
    (dict(), DEV), (dict(off=FAKE, E=3), DEV), (dict(rows=FAKE, Ma=3), DEV), (dict(N=1, K=16), DEV),
    (dict(M=0, Ma=0, A=None, C=None), OK),
    (dict(M=-1), INV), (dict(N=0), INV), (dict(K=0), INV), (dict(K=24), UNS), (dict(K=2**22), UNS),
    (dict(N=2**30, K=2**20), UNS), (dict(M=2**31 - 1, Ma=2**31 - 1), UNS),
    (dict(E=2), INV), (dict(E=0), INV), (dict(off=FAKE, E=70000), INV), (dict(flags=1), INV),
    (dict(Ma=7), INV), (dict(rows=FAKE, Ma=-1), INV), (dict(rows=FAKE, Ma=0), INV),
    (dict(A=None), INV), (dict(sa=None), INV), (dict(W=None), INV), (dict(sw=None), INV), (dict(C=None), INV),
    (dict(A=P(0x10008)), INV), (dict(W=P(0x10008)), INV), (dict(C=P(0x10001)), INV), (dict(sa=P(0x10002)), INV),
    (dict(rows=P(0x10002)), INV), (dict(off=P(0x10002)), INV),
    (dict(dtype=qg.QG_DTYPE_F32), INV),
    (dict(rows=FAKE, Ma=2**20, K=4096), UNS),           # codes past 32-bit offsets
    (dict(rows=FAKE, Ma=2**20, K=4080), DEV),           # just below
    (dict(M=2**31 - 2048, Ma=2**31 - 2048, N=1024, K=16), UNS),   # more workgroups than a grid holds
])
def test_qgemm_fp8_refusals(kw, rc):
    assert _gemm(**kw) == rc
    assert rc == OK or qg.lib().qg_last_error()


def _route(x=FAKE, dtype=qg.QG_DTYPE_F32, bias=None, T=4, E=64, k=8, g=1, kg=1, flags=0, ids=FAKE, w=FAKE):
    return qg.lib().moe_route(x, dtype, bias, T, E, k, g, kg, 1.0, flags, ids, w, None)


@no_gpu
@pytest.mark.parametrize("kw,rc", [
    (dict(), DEV), (dict(g=8, kg=4, flags=7, bias=FAKE), DEV), (dict(E=1, k=1), DEV), (dict(E=1024, k=64), DEV),
    (dict(T=0, x=None, ids=None, w=None), OK),
    (dict(T=-1), INV), (dict(E=0), INV), (dict(k=0), INV), (dict(E=1025), UNS), (dict(E=256, k=65), UNS),
    (dict(E=1024, g=128, kg=128), UNS), (dict(g=7, kg=1), INV), (dict(g=0), INV), (dict(g=8, kg=9), INV),
    (dict(g=8, kg=0), INV), (dict(g=16, kg=1, k=5), INV), (dict(E=4, k=5), INV), (dict(flags=8), INV),
    (dict(T=2**27), UNS), (dict(dtype=3), INV), (dict(x=None), INV), (dict(ids=None), INV), (dict(w=None), INV),
    (dict(x=P(0x10002)), INV), (dict(x=P(0x10001), dtype=qg.QG_DTYPE_F16), INV), (dict(bias=P(0x10002)), INV),
])
def test_moe_route_refusals(kw, rc):
    assert _route(**kw) == rc
    assert rc == OK or qg.lib().qg_last_error()


def _sort(ids=FAKE, T=4, k=8, E=64, off=FAKE, row=FAKE, slot=FAKE, ws=None, n=0):
    return qg.lib().moe_sort_rows(ids, T, k, E, off, row, slot, ws, n, None)


@no_gpu
@pytest.mark.parametrize("kw,rc", [
    (dict(), DEV), (dict(E=1024), DEV), (dict(T=0, ids=None, row=None, slot=None), DEV),
    (dict(T=-1), INV), (dict(k=0), INV), (dict(E=0), INV), (dict(E=1025), UNS), (dict(T=2**28, k=4), UNS),
    (dict(off=None), INV), (dict(ids=None), INV), (dict(row=None), INV), (dict(slot=None), INV),
    (dict(ids=P(0x10002)), INV),
])
def test_moe_sort_refusals(kw, rc):
    assert _sort(**kw) == rc
    assert rc == OK or qg.lib().qg_last_error()


def test_moe_sort_workspace():
    assert qg.qg_workspace_bytes(qg.QG_OP_MOE_SORT, 1, 8, 0, 0, 64) == 0
    n = qg.qg_workspace_bytes(qg.QG_OP_MOE_SORT, 16384, 8, 0, 0, 256)
    if n and not torch.cuda.is_available():
        big = dict(T=16384, k=8, E=256)
        assert _sort(**big) == WSP
        assert _sort(**big, ws=FAKE, n=n - 1) == WSP
        assert _sort(**big, ws=P(0x10040), n=n) == INV
        assert _sort(**big, ws=FAKE, n=n) == DEV
    with pytest.raises(qg.QGemmError):
        qg.qg_workspace_bytes(qg.QG_OP_MOE_SORT, 1, 8, 0, 0, 2000)
    assert qg.qg_workspace_bytes(qg.QG_OP_FP8, 16, 100, 128, 128, 4) == 0


def _combine(Y=FAKE, dtype=qg.QG_DTYPE_F16, slot=FAKE, w=FAKE, T=4, k=8, M=32, N=100, out=FAKE):
    return qg.lib().moe_combine_rows(Y, dtype, slot, w, T, k, M, N, out, None)


@no_gpu
@pytest.mark.parametrize("kw,rc", [
    (dict(), DEV), (dict(M=0, Y=None), DEV), (dict(T=0, slot=None, w=None, out=None), OK),
    (dict(T=-1), INV), (dict(k=0), INV), (dict(k=65), UNS), (dict(M=-1), INV), (dict(N=0), INV),
    (dict(Y=None), INV), (dict(slot=None), INV), (dict(w=None), INV), (dict(out=None), INV),
    (dict(Y=P(0x10001)), INV), (dict(out=P(0x10001)), INV), (dict(slot=P(0x10002)), INV),
    (dict(dtype=qg.QG_DTYPE_F32), INV),
])
def test_moe_combine_refusals(kw, rc):
    assert _combine(**kw) == rc
    assert rc == OK or qg.lib().qg_last_error()


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError, match="device tensor"):
        qg.route(x, 2)
    with pytest.raises(TypeError):
        qg.route(x.double(), 2)
    with pytest.raises(ValueError, match="score"):
        qg.route(x, 2, score="linear")
    with pytest.raises(ValueError, match="group_score"):
        qg.route(x, 2, group_score="sum")
    with pytest.raises(TypeError):
        qg.quantize_fp8(x)
    with pytest.raises(ValueError, match="device tensor"):
        qg.quantize_fp8(x.half())
    with pytest.raises(ValueError, match="even width"):
        qg.quantize_fp8(torch.zeros(2, 33).half(), swiglu=True)
    with pytest.raises(ValueError, match="device tensor"):
        qg.sort_rows(torch.zeros(2, 2, dtype=torch.int32), 4)
    with pytest.raises(TypeError):
        qg.combine_rows(x, torch.zeros(2, 2, dtype=torch.int32), x)
    with pytest.raises(TypeError):
        qg.fp8_gemm(x, x, x, x, dtype=torch.float32)


def test_binding_refuses_counts_past_32_bits():
    """A count of 2^32 + 2 is not the 2 that an int would make of it."""
    n = 2**32 + 2

    def t(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="meta")

    f8, i32 = torch.float8_e4m3fn, torch.int32
    calls = [lambda: qg.quantize_fp8(t(n, 16, dtype=torch.float16)),
             lambda: qg.fp8_gemm(t(n, 16, dtype=f8), t(n, 1), t(16, 16, dtype=f8), t(1, 1)),
             lambda: qg.fp8_gemm(t(4, 16, dtype=f8), t(4, 1), t(16, 16, dtype=f8), t(1, 1), a_rows=t(n, dtype=i32)),
             lambda: qg.route(t(n, 8), 2),
             lambda: qg.combine_rows(t(n, 8, dtype=torch.float16), t(4, 2, dtype=i32), t(4, 2)),
             lambda: qg.moe_sort_rows(t(n, 2, dtype=i32), n, 2, 8, t(9, dtype=i32), t(2 * n, dtype=i32),
                                      t(n, 2, dtype=i32))]
    for call in calls:
        with pytest.raises(ValueError, match="counts"):
            call()
