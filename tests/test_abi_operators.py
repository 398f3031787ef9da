"""CPU checks of the host validation of the conv-prefill, commit, scan and verification
entry points: each bad call returns its status before any CUDA call."""

import ctypes

import pytest

from linear_attention_recurrent_selective_b200 import build, ssu

P16 = ctypes.c_void_p(256)          # never dereferenced
ODD = ctypes.c_void_p(260)


@pytest.fixture(scope="module")
def L():
    build.build()
    return ssu.lib()


def call(fn, good, **kw):
    a = dict(good)
    assert set(kw) <= set(a)
    a.update(kw)
    return fn(*a.values())


CONV = dict(xbc=P16, dt=2, ld=5376, w=P16, bias=None, pool=P16, cs=5376 * 3, cc=3, ck=1, width=4,
            silu=1, P=32, x=P16, B=P16, C=P16, idx=P16, ctx=P16, par=None, upd=1, batch=16,
            active=16, T=512, xd=5120, bc=128, err=None, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(xbc=None), 1), (dict(w=None), 1), (dict(pool=None), 1), (dict(x=None), 1),
    (dict(B=None), 1), (dict(C=None), 1), (dict(dt=3), 3), (dict(dt=-1), 3),
    (dict(ld=5375), 2), (dict(width=0), 2), (dict(width=17), 2), (dict(active=17), 2),
    (dict(active=-1), 2), (dict(T=-1), 2), (dict(xd=0), 2), (dict(bc=-1), 2), (dict(P=-1), 2),
    (dict(idx=None, P=15), 2), (dict(cs=5376 * 3 - 1), 2), (dict(cc=2), 2), (dict(ck=0), 2),
    (dict(cc=1, ck=5375), 2), (dict(cc=-3), 2), (dict(par=P16), 2),
    (dict(par=P16, upd=0, T=129), 2),
    (dict(cc=1 << 62, cs=(1 << 62) + 5), 2), (dict(xd=2 ** 31 - 1, bc=2 ** 30, ld=2 ** 40), 2),
])
def test_conv_prefill(L, kw, status):
    assert call(L.ssu_conv_prefill, CONV, **kw) == status


def test_conv_prefill_with_nothing_to_do(L):
    nulls = dict(xbc=None, w=None, pool=None, x=None, B=None, C=None)
    assert call(L.ssu_conv_prefill, CONV, active=0, **nulls) == 0
    assert call(L.ssu_conv_prefill, CONV, T=0, **nulls) == 0


COMMIT = dict(xbc=P16, dt=2, ld=5376, pool=P16, cs=5376 * 3, cc=3, ck=1, width=4, P=128, acc=P16,
              idx=P16, batch=64, active=64, T=5, ch=5376, ids=None, most=0, err=None, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(xbc=None), 1), (dict(pool=None), 1), (dict(acc=None), 1), (dict(dt=9), 3),
    (dict(ld=100), 2), (dict(ch=0), 2), (dict(ids=P16, most=-1), 2), (dict(active=65), 2),
    (dict(idx=None, P=63), 2), (dict(cc=1), 2), (dict(width=1, pool=None, xbc=None), 0),
    (dict(T=0, xbc=None), 0), (dict(active=0, acc=None), 0),
])
def test_conv_replay(L, kw, status):
    assert call(L.ssu_conv_replay, COMMIT, **kw) == status


SCAN = dict(x=P16, xdt=2, ldx=5120, dt=P16, ddt=2, lddt=5120, A=P16, B=P16, C=P16, bdt=2, ldb=16,
            ldc=16, bias=None, D=None, z=P16, ldz=5120, pool=P16, sdt=0, stride=5120 * 16, P=32,
            out=P16, idx=P16)
PRE = dict(SCAN, ctx=None, upd=1, batch=16, active=16, T=512, ch=5120, G=1, N=16, sp=1, err=None,
           stream=None)
DEC = dict(SCAN, batch=16, active=16, ch=5120, G=1, N=16, sp=1, err=None, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(dt=None), 1), (dict(A=None), 1), (dict(B=None), 1),
    (dict(C=None), 1), (dict(pool=None), 1), (dict(xdt=3), 3), (dict(ddt=-1), 3),
    (dict(bdt=5), 3), (dict(sdt=4), 3), (dict(ldx=5119), 2), (dict(lddt=0), 2),
    (dict(ldz=100), 2), (dict(ldb=15), 2), (dict(ldc=15), 2), (dict(stride=100), 2),
    (dict(active=17), 2), (dict(G=3), 2), (dict(G=0), 2), (dict(ch=0), 2),
    (dict(idx=None, P=3), 2), (dict(N=24, stride=5120 * 24, ldb=24, ldc=24), 4),
    (dict(pool=ctypes.c_void_p(264)), 6), (dict(A=ODD), 6), (dict(stride=5120 * 16 + 1), 6),
])
def test_scan(L, kw, status):
    assert call(L.scan_prefill, PRE, **kw) == status
    assert call(L.scan_decode, DEC, **kw) == status


def test_scan_outputs_and_empty_calls(L):
    assert call(L.scan_prefill, PRE, out=None, upd=0) == 1
    assert call(L.scan_decode, DEC, out=None) == 1
    assert call(L.scan_prefill, PRE, T=-1) == 2
    nulls = dict(x=None, dt=None, A=None, B=None, C=None, pool=None, out=None)
    assert call(L.scan_prefill, PRE, T=0, **nulls) == 0
    assert call(L.scan_prefill, PRE, active=0, **nulls) == 0
    assert call(L.scan_decode, DEC, active=0, **nulls) == 0


def test_sizes_near_the_counters_range(L):
    big = 2 ** 30 + 1
    assert call(L.ssu_conv_prefill, CONV, T=big) == 2
    assert call(L.ssu_conv_prefill, CONV, batch=big, active=1) == 2
    wide = dict(ld=2 ** 31, cs=2 ** 34)
    assert call(L.ssu_conv_prefill, CONV, xd=2 ** 30 - 1, bc=1, **wide) == 2
    assert call(L.ssu_conv_replay, COMMIT, ch=big, **wide) == 2
    assert call(L.ssu_conv_replay, COMMIT, T=big) == 2
    assert call(L.scan_prefill, PRE, T=big) == 2
    rows = dict(ch=big, ldx=2 ** 31, lddt=2 ** 31, ldz=2 ** 31, stride=2 ** 36)
    for fn, good in ((L.scan_prefill, PRE), (L.scan_decode, DEC)):
        assert call(fn, good, **rows) == 2
        assert call(fn, good, batch=big, active=1) == 2
    assert call(L.spec_verify, VERIFY, T=big) == 2


VERIFY = dict(tok=P16, p=P16, q=P16, dt=0, ldp=32768, ldq=32768, u=P16, us=P16, ctx=None,
              par=None, idx=None, acc=P16, nxt=P16, ids=None, most=0, batch=64, active=64, T=5,
              V=32768, err=None, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(tok=None), 1), (dict(p=None), 1), (dict(u=None), 1), (dict(us=None), 1),
    (dict(acc=None), 1), (dict(nxt=None), 1), (dict(dt=3), 3), (dict(ldp=32767), 2),
    (dict(ldq=32767), 2), (dict(V=0), 2), (dict(V=2 ** 30 + 1, ldp=2 ** 31, ldq=2 ** 31), 2),
    (dict(active=65), 2), (dict(T=-1), 2), (dict(par=P16), 2), (dict(par=P16, q=None, T=129), 2),
    (dict(ids=P16, most=5), 2), (dict(par=P16, q=None, ids=P16, most=0), 2),
    (dict(T=0, tok=None, p=None), 0), (dict(active=0, acc=None, nxt=None), 0),
])
def test_verify(L, kw, status):
    assert call(L.spec_verify, VERIFY, **kw) == status
