"""CPU checks of the 4-bit cache's and the adapters' entry points: bad arguments are refused
on the host before a device is touched, valid ones reach the device check, empty
batches succeed, and the binding checks types, shapes, strides and devices.  No kernel
runs here."""
import ctypes

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import int4_weight_only_uint32_amd as qg

P = ctypes.c_void_p
FAKE = P(0x10000)     # never dereferenced
OK, INV, UNS, WSP, DEV = (qg.QG_OK, qg.QG_ERR_INVALID_ARG, qg.QG_ERR_UNSUPPORTED, qg.QG_ERR_WORKSPACE,
                          qg.QG_ERR_DEVICE)
BF, F16, F32 = qg.QG_DTYPE_BF16, qg.QG_DTYPE_F16, qg.QG_DTYPE_F32

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake pointers: only where no kernel can start")

CACHE = [
    (dict(pages=0), INV), (dict(H=0), INV), (dict(width=0), INV), (dict(B=-1), INV), (dict(T=-1, B=-1), INV),
    (dict(D=96), UNS), (dict(D=0), UNS), (dict(g=16), UNS), (dict(g=256), UNS), (dict(D=64, g=128), UNS),
    (dict(page=16), UNS), (dict(page=48), UNS), (dict(page=2048), UNS), (dict(page=0), UNS), (dict(H=5000), UNS),
    (dict(width=2**25, page=64), UNS), (dict(T=4, B=3, off=None), INV),
    (dict(kc=None), INV), (dict(vc=None), INV), (dict(ks=None), INV), (dict(vs=None), INV), (dict(lens=None), INV),
    (dict(table=None), INV), (dict(kc=P(0x10008)), INV), (dict(vs=P(0x10008)), INV), (dict(lens=P(0x10002)), INV),
    (dict(off=P(0x10002)), INV), (dict(dtype=9), INV),
]


def _append(k=FAKE, v=FAKE, q=None, dtype=BF, T=4, ldk=256, ldv=256, ldq=1024, qh=8, off=FAKE, lens=FAKE, table=FAKE,
            B=2, width=4, pos=None, cs=FAKE, rot=128, maxp=100, flags=0, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, pages=9,
            H=2, page=64, D=128, g=64, qo=None):
    return qg.lib().kv4_append(k, v, q, dtype, T, ldk, ldv, ldq, qh, off, lens, table, B, width, pos, cs, rot, maxp,
                               flags, kc, vc, ks, vs, pages, H, page, D, g, qo, None)


@no_gpu
@pytest.mark.parametrize("kw,rc", CACHE + [
    (dict(), DEV), (dict(q=FAKE, qo=FAKE), DEV), (dict(off=None, T=2), DEV), (dict(cs=None, rot=0), DEV),
    (dict(D=64, g=32, rot=32), DEV), (dict(page=1024, flags=1, pos=FAKE), DEV), (dict(D=256, g=128, ldk=512, ldv=512), DEV),
    (dict(T=0, k=None, v=None), OK), (dict(T=0, B=0, off=None, k=None, lens=None), OK),
    (dict(k=None), INV), (dict(v=None), INV), (dict(k=P(0x10008)), INV), (dict(ldk=250), INV), (dict(ldk=248), INV),
    (dict(ldv=0), INV), (dict(ldv=-256), INV), (dict(q=FAKE), INV), (dict(q=FAKE, qo=P(0x10008)), INV),
    (dict(q=FAKE, qo=FAKE, ldq=1016), INV), (dict(q=FAKE, qo=FAKE, qh=0), INV), (dict(q=FAKE, qo=FAKE, qh=2**19), INV),
    (dict(q=FAKE, qo=FAKE, qh=2**18, ldq=2**25), INV),
    (dict(rot=144), UNS), (dict(rot=-16), UNS), (dict(rot=24), UNS), (dict(cs=None), INV), (dict(maxp=0), INV),
    (dict(cs=P(0x10004)), INV), (dict(pos=P(0x10002)), INV), (dict(flags=2), INV), (dict(dtype=F32), INV),
    (dict(T=2**28), UNS),
])
def test_append_refusals(kw, rc):
    assert _append(**kw) == rc
    assert rc == OK or qg.lib().qg_last_error()


def _read(kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, pages=9, H=2, page=64, D=128, g=64, off=FAKE, lens=FAKE, table=FAKE, B=2,
          width=4, T=4, dtype=BF, ko=FAKE, vo=FAKE):
    return qg.lib().kv4_read(kc, vc, ks, vs, pages, H, page, D, g, off, lens, table, B, width, T, dtype, ko, vo, None)


@no_gpu
@pytest.mark.parametrize("kw,rc", CACHE + [
    (dict(), DEV), (dict(dtype=F32), DEV), (dict(off=None, T=2), DEV), (dict(T=0, ko=None, vo=None), OK),
    (dict(ko=None), INV), (dict(vo=None), INV), (dict(ko=P(0x10008)), INV),
])
def test_read_refusals(kw, rc):
    assert _read(**kw) == rc
    assert rc == OK or qg.lib().qg_last_error()


def _attend(q=FAKE, dtype=BF, T=4, ldq=1024, qh=8, new=2, off=FAKE, lens=FAKE, table=FAKE, B=2, width=4, kc=FAKE,
            vc=FAKE, ks=FAKE, vs=FAKE, pages=9, H=2, page=64, D=128, g=64, scale=0.1, window=0, sinks=0, out=FAKE,
            ws=FAKE, nb=1 << 40, flags=0):
    return qg.lib().kv4_attend(q, dtype, T, ldq, qh, new, off, lens, table, B, width, kc, vc, ks, vs, pages, H, page, D,
                               g, scale, window, sinks, out, ws, nb, flags, None)


@no_gpu
@pytest.mark.parametrize("kw,rc", CACHE + [
    (dict(), DEV), (dict(off=None, T=2, new=1), DEV), (dict(window=1, sinks=2**31 - 1), DEV),
    (dict(T=0, q=None, out=None), OK), (dict(B=0, T=0, off=None, lens=None), OK),
    (dict(q=None), INV), (dict(out=None), INV), (dict(out=P(0x10008)), INV), (dict(q=P(0x10008)), INV),
    (dict(ldq=1020), INV), (dict(ldq=1016), INV), (dict(qh=7), INV), (dict(qh=0), INV), (dict(new=0), INV),
    (dict(window=-1), INV), (dict(sinks=-1), INV), (dict(scale=0.0), INV), (dict(scale=-1.0), INV),
    (dict(scale=float("inf")), INV), (dict(scale=float("nan")), INV), (dict(flags=1), INV), (dict(dtype=F32), INV),
    # (four pages are seen without parts: no workspace is asked for)
    (dict(ws=None), DEV), (dict(nb=16), DEV), (dict(ws=None, nb=0), DEV),
    (dict(ws=None, width=64), WSP), (dict(nb=16, width=64), WSP), (dict(ws=P(0x10010), width=64), INV),
    (dict(T=2**24, qh=64, ldq=64 * 128), UNS),
    # a launch's threads: 2^17 blocks of rows of 64 heads, 512 threads each where few tokens are seen
    (dict(T=2**21, H=64, qh=64, ldq=64 * 128, new=1), UNS), (dict(T=2**20, H=64, qh=64, ldq=64 * 128, new=1), DEV),
])
def test_attend_refusals(kw, rc):
    assert _attend(**kw) == rc
    assert rc == OK or qg.lib().qg_last_error()


def test_attend_workspace_sizes():
    f = qg.lib().kv4_attend_workspace_bytes
    bad = ctypes.c_size_t(-1).value
    assert f(0, 1, 4, 8, 2, 128, 4, 64, 0, 0) == 0
    n = f(1, 1, 1, 8, 8, 128, 2048, 64, 0, 0)
    assert n > 8 * 130 * 4 and n % (8 * 4) == 0                   # parts of 8 rows of 128 values, maximum and sum; their number
    assert f(1, 1, 1, 8, 8, 128, 2048, 64, 128, 0) < n            # a window needs fewer
    assert f(4096, 4096, 1, 64, 8, 128, 2048, 64, 0, 0) == 0      # enough rows: no parts
    assert f(2**24, 1, 1, 8, 8, 128, 2048, 64, 0, 0) == 0         # nor where max_new says there are few
    for args in ((-1, 1, 1, 8, 8, 128, 4, 64, 0, 0), (1, 0, 1, 8, 8, 128, 4, 64, 0, 0), (1, 1, 1, 8, 3, 128, 4, 64, 0, 0),
                 (1, 1, 1, 8, 8, 128, 0, 64, 0, 0), (1, 1, 1, 8, 8, 128, 2**25, 64, 0, 0), (1, 1, 1, 8, 8, 128, 4, 64, -1, 0)):
        assert f(*args) == bad and qg.lib().qg_last_error()


def _lora(x=FAKE, a=FAKE, b=FAKE, sc=None, off=FAKE, rows=FAKE, slots=FAKE, L=3, T=4, K=256, N=128, R=16, dtype=BF,
          y=FAKE, ws=FAKE, nb=1 << 40):
    return qg.lib().lora_add(x, a, b, sc, off, rows, slots, L, T, K, N, R, dtype, y, ws, nb, None)


@no_gpu
@pytest.mark.parametrize("kw,rc", [
    (dict(), DEV), (dict(sc=FAKE, R=512), DEV), (dict(K=8, N=8, R=8, L=1, T=1), DEV),
    (dict(T=0, x=None, y=None, ws=None), OK),
    (dict(T=-1), INV), (dict(L=0), INV), (dict(K=0), INV), (dict(N=0), INV), (dict(R=0), INV),
    (dict(K=12), UNS), (dict(N=12), UNS), (dict(R=12), UNS), (dict(R=520), UNS), (dict(L=70000), UNS),
    (dict(K=2**25), UNS), (dict(N=2**25), UNS), (dict(T=2**24), UNS), (dict(dtype=F32), INV),
    (dict(x=None), INV), (dict(a=None), INV), (dict(b=None), INV), (dict(y=None), INV), (dict(off=None), INV),
    (dict(rows=None), INV), (dict(slots=None), INV), (dict(x=P(0x10008)), INV), (dict(b=P(0x10008)), INV),
    (dict(y=P(0x10008)), INV), (dict(sc=P(0x10002)), INV), (dict(rows=P(0x10002)), INV),
    (dict(ws=None), WSP), (dict(nb=16), WSP), (dict(ws=P(0x10010)), INV),
])
def test_lora_refusals(kw, rc):
    assert _lora(**kw) == rc
    assert rc == OK or qg.lib().qg_last_error()


def test_lora_workspace_sizes():
    f = qg.qg_workspace_bytes
    assert f(qg.QG_OP_LORA, 0, 128, 256, 16, 3) == 0
    assert f(qg.QG_OP_LORA, 4, 128, 256, 16, 3) >= 4 * 16 * 4      # sums of 16 columns for four rows
    for args in ((-1, 128, 256, 16, 3), (4, 12, 256, 16, 3), (4, 128, 256, 12, 3), (4, 128, 256, 16, 0)):
        with pytest.raises(qg.QGemmError):
            f(qg.QG_OP_LORA, *args)


@pytest.mark.skipif(torch.cuda.is_available(), reason="tensors without storage: only where no kernel can start")
@pytest.mark.filterwarnings("ignore:Accessing the data pointer of FakeTensor")
def test_binding_refuses_shapes_types_strides_and_devices():
    with FakeTensorMode():
        def t(*shape, dtype=torch.bfloat16, dev="cuda:0"):
            return torch.empty(shape, dtype=dtype, device=dev)

        i32, f16, f32 = torch.int32, torch.float16, torch.float32

        def cache(dev="cuda:0", **kw):
            d = dict(k=t(9, 2, 64, 16, dtype=i32, dev=dev), v=t(9, 2, 64, 16, dtype=i32, dev=dev),
                     k_sz=t(9, 2, 2, 64, 2, dtype=f16, dev=dev), v_sz=t(9, 2, 2, 64, 2, dtype=f16, dev=dev))
            d.update(kw)
            return qg.KV4Cache(**d)

        lens, table, off = t(2, dtype=i32), t(2, 4, dtype=i32), t(3, dtype=i32)

        def append(c=None, k=None, v=None, lens=lens, table=table, off=off, **kw):
            return qg.kv4_append(c or cache(), t(5, 2, 128) if k is None else k, t(5, 2, 128) if v is None else v, lens, table,
                                 seq_offsets=off, **kw)

        def attend(q=None, c=None, lens=lens, table=table, off=off, **kw):
            return qg.kv4_attend(t(5, 8, 128) if q is None else q, c or cache(), lens, table, seq_offsets=off, **kw)

        for call, err, match in (
                (lambda: append(k=t(5, 2, 128, dtype=f32)), TypeError, "k must be fp16 or bf16"),
                (lambda: append(v=t(5, 2, 128, dtype=f16)), TypeError, "v must be"),
                (lambda: append(k=t(5, 2, 64)), ValueError, "k must be"),
                (lambda: append(k=t(5, 3, 128)), ValueError, "k must be"),
                (lambda: append(v=t(4, 2, 128)), ValueError, "v must be"),
                (lambda: append(k=t(2, 5, 128).transpose(0, 1)), ValueError, "stand together"),
                (lambda: append(v=t(5, 2, 256)[..., ::2]), ValueError, "stand together"),
                (lambda: append(v=t(5, 2, 128, dev="cuda:1")), ValueError, "v is on cuda:1"),
                (lambda: append(c=cache("cuda:1")), ValueError, "cache.k is on cuda:1"),
                (lambda: append(c=cache(v=t(9, 2, 64, 8, dtype=i32))), ValueError, "cache.v"),
                (lambda: append(c=cache(k_sz=t(9, 2, 2, 64, 2))), TypeError, "cache.k_sz"),
                (lambda: append(c=cache(k_sz=t(9, 2, 0, 64, 2, dtype=f16))), ValueError, "groups"),
                (lambda: append(c=cache(k_sz=t(9, 2, 3, 64, 2, dtype=f16))), ValueError, "groups"),
                (lambda: append(c=cache(k=t(9, 2, 64, 32, dtype=i32)[..., ::2])), ValueError, "contiguous"),
                (lambda: append(lens=t(3, dtype=i32)), ValueError, "kv_lens"),
                (lambda: append(lens=t(2, dtype=torch.int64)), TypeError, "kv_lens"),
                (lambda: append(off=t(2, dtype=i32)), ValueError, "seq_offsets"),
                (lambda: append(table=t(8, dtype=i32)), ValueError, "page_table"),
                (lambda: append(table=t(2, 4, dtype=i32, dev="cuda:1")), ValueError, "page_table is on"),
                (lambda: append(q_out=t(5, 8, 128)), ValueError, "without q"),
                (lambda: append(q=t(5, 8, 64)), ValueError, "q must be"),
                (lambda: append(q=t(5, 8, 128), q_out=t(5, 8, 64)), ValueError, "q_out"),
                (lambda: append(positions=t(4, dtype=i32)), ValueError, "positions"),
                (lambda: append(cos_sin=t(100, 128)), TypeError, "cos_sin"),
                (lambda: append(cos_sin=t(100, 0, dtype=f32)), ValueError, "angles"),
                (lambda: attend(t(5, 8, 128, dtype=f32)), TypeError, "q must be"),
                (lambda: attend(t(5, 8, 64)), ValueError, "q must be"),
                (lambda: attend(t(5, 1024)), ValueError, "q must be"),
                (lambda: attend(t(5, 7, 128)), qg.QGemmError, "query heads"),
                (lambda: attend(window=-1), ValueError, "window"),
                (lambda: attend(window=2**31), ValueError, "window"),
                (lambda: attend(out=t(5, 8, 128, dtype=f16)), TypeError, "out"),
                (lambda: attend(out=t(4, 8, 128)), ValueError, "out"),
                (lambda: attend(out=t(5, 8, 128, dev="cuda:1")), ValueError, "out is on"),
                (lambda: qg.kv4_read(cache(), lens, table, seq_offsets=off), ValueError, "rows"),
                (lambda: qg.kv4_read(cache(), lens, table, seq_offsets=off, rows=-1), ValueError, "rows"),
                (lambda: qg.kv4_read(cache(), lens, table, dtype=i32), TypeError, "dtype"),
                (lambda: qg.kv4_read(cache(), lens, table, seq_offsets=off, k_out=t(5, 2, 128), v_out=t(4, 2, 128)),
                 ValueError, "v_out"),
        ):
            with pytest.raises(err, match=match):
                call()

        def lora(x=None, A=None, B=None, plan=None, y=None, **kw):
            pl = plan or (t(4, dtype=i32), t(5, dtype=i32), t(5, 1, dtype=i32))
            return qg.lora(t(5, 256) if x is None else x, t(3, 16, 256) if A is None else A,
                           t(3, 64, 16) if B is None else B, pl, t(5, 64) if y is None else y, **kw)

        for call, err, match in (
                (lambda: lora(x=t(5, 256, dtype=f32)), TypeError, "x must be"),
                (lambda: lora(A=t(3, 16, 256, dtype=f16)), TypeError, "A must be"),
                (lambda: lora(A=t(3, 16, 128)), ValueError, "A must be"),
                (lambda: lora(B=t(3, 64, 8)), ValueError, "B must be"),
                (lambda: lora(B=t(2, 64, 16)), ValueError, "B must be"),
                (lambda: lora(y=t(5, 128)), ValueError, "y must be"),
                (lambda: lora(y=t(5, 64, dev="cuda:1")), ValueError, "y is on"),
                (lambda: lora(x=t(5, 512)[:, ::2]), ValueError, "contiguous"),
                (lambda: lora(scaling=t(2, dtype=f32)), ValueError, "scaling"),
                (lambda: lora(plan=(t(5, dtype=i32), t(5, dtype=i32), t(5, 1, dtype=i32))), ValueError, "offsets"),
                (lambda: lora(plan=(t(4, dtype=i32), t(10, dtype=i32), t(5, 2, dtype=i32))), ValueError, "rows"),
                (lambda: lora(plan=(t(4, dtype=i32), t(5, dtype=i32), t(5, 2, dtype=i32))), ValueError, "slots"),
                (lambda: lora(A=t(3, 256)), ValueError, "x is"),
        ):
            with pytest.raises(err, match=match):
                call()


def test_binding_refuses_host_tensors():
    c = qg.kv4_cache(2, 1, 64, 32, 32, device="cpu")
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensor"):
        qg.kv4_append(c, torch.zeros(1, 1, 64).half(), torch.zeros(1, 1, 64).half(), i, i[None])
    with pytest.raises(ValueError, match="device tensor"):
        qg.kv4_attend(torch.zeros(1, 1, 64).half(), c, i, i[None])
    with pytest.raises(ValueError, match="device tensor"):
        qg.kv4_read(c, i, i[None])
    with pytest.raises(ValueError, match="device tensor"):
        qg.lora(torch.zeros(1, 8).half(), torch.zeros(1, 8, 8).half(), torch.zeros(1, 8, 8).half(), (i, i, i[None]),
                torch.zeros(1, 8).half())
