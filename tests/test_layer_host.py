"""Host-side refusals of the layer operators: every mistake the host can see is refused before a launch."""
import ctypes

import pytest

FAKE = 0x10000   # a 16-byte aligned non-null address; never dereferenced on the host
OUT = FAKE + 0x1000000
NAN, INF = float("nan"), float("inf")


class Opts(ctypes.Structure):
    _fields_ = [("act", ctypes.c_int32), ("gated", ctypes.c_int32), ("bias", ctypes.c_void_p),
                ("residual", ctypes.c_void_p), ("residual_stride", ctypes.c_int64)]


class Out(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("stride", ctypes.c_int64), ("cols", ctypes.c_int32)]


class Norm(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("eps", ctypes.c_float), ("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p)]


@pytest.fixture(scope="module")
def lib():
    from decode_attention_self_gb300 import build

    return ctypes.CDLL(build.build())


def vp(x):
    return ctypes.c_void_p(x)


def linear(lib, x=FAKE, xs=1024, W=FAKE, opts=None, T=4, K=1024, N=1024, outs=None, n_outs=None, od=0, stall=None):
    outs = [(OUT, 1024, 1024)] if outs is None else outs
    arr = (Out * max(1, len(outs)))(*[Out(*o) for o in outs])
    o = None if opts is None else ctypes.byref(Opts(**opts))
    args = (vp(x), ctypes.c_int64(xs), vp(W), o, T, K, N, arr, len(outs) if n_outs is None else n_outs, od, None)
    if stall is None:
        return lib.dr_linear(*args, None)
    return lib.dr_linear_stall_test(*args, stall, None)


@pytest.mark.parametrize("bad", [
    dict(T=0), dict(T=-1), dict(K=0), dict(K=1020), dict(K=4), dict(N=0), dict(x=None), dict(W=None), dict(x=FAKE + 8),
    dict(W=FAKE + 2), dict(xs=1016), dict(xs=1028), dict(od=2), dict(n_outs=0), dict(n_outs=5),
    dict(outs=[(None, 1024, 1024)]), dict(outs=[(OUT, 1023, 1024)]), dict(outs=[(OUT + 1, 1024, 1024)]),
    dict(outs=[(OUT + 2, 1024, 1024)], od=1), dict(outs=[(OUT, 1024, 1000)]), dict(outs=[(OUT, 1100, 1100)]),
    dict(outs=[(OUT, 1000, 1000), (OUT + 0x100000, 24, 24)]), dict(outs=[(OUT, 64, 0), (OUT + 0x100000, 1024, 1024)]),
    dict(outs=[(OUT, 512, 512), (OUT + 0x100000, 1024, 1024)]),
    dict(opts=dict(act=5)), dict(opts=dict(act=-1)), dict(opts=dict(gated=2)), dict(opts=dict(bias=FAKE + 2)),
    dict(opts=dict(residual=FAKE, residual_stride=1000)), dict(opts=dict(residual=FAKE + 1, residual_stride=1024)),
    dict(opts=dict(residual=OUT, residual_stride=2048)),             # the output itself with another stride
    dict(opts=dict(residual=FAKE, residual_stride=1024), outs=[(OUT, 512, 512), (OUT + 0x100000, 512, 512)]),
    dict(outs=[(OUT, 512, 512), (OUT, 512, 512)]),                  # two outputs in one place
    dict(outs=[(FAKE, 1024, 1024)]), dict(W=OUT), dict(opts=dict(bias=OUT)),   # an output that is an input
    dict(T=2 ** 31 - 4095), dict(K=2 ** 30 + 8, xs=2 ** 30 + 8), dict(xs=2 ** 37 + 8), dict(outs=[(OUT, 2 ** 37 + 8, 1024)]),
    dict(stall=-1), dict(N=1 << 30, outs=[(OUT, 1 << 30, 1 << 30)]),
])
def test_linear_refusals(lib, bad):
    assert linear(lib, **bad) == 1


def norm(lib, x=FAKE, xs=1024, xd=0, post=None, gate=None, gs=0, scale=1.0, res=None, rs=1024, h=None, hs=1024, hd=0,
         pre=(1, 1e-5, FAKE, FAKE), y=FAKE + 0x100000, ys=1024, yd=0, T=4, Dm=1024):
    i64 = ctypes.c_int64
    mk = lambda n: None if n is None else ctypes.byref(Norm(*n))
    return lib.dr_residual_norm(vp(x), i64(xs), xd, mk(post), vp(gate), i64(gs), ctypes.c_float(scale), vp(res), i64(rs),
                                vp(h), i64(hs), hd, mk(pre), vp(y), i64(ys), yd, T, Dm, None)


@pytest.mark.parametrize("bad,status", [
    (dict(T=0), 1), (dict(Dm=0), 1), (dict(Dm=1020), 1), (dict(Dm=4), 1), (dict(x=None), 1), (dict(y=None), 1),
    (dict(x=FAKE + 8), 1), (dict(y=FAKE + 2), 1), (dict(xs=1000), 1), (dict(xs=1028), 1), (dict(ys=512), 1),
    (dict(xd=3), 1), (dict(hd=2), 1), (dict(yd=-1), 1), (dict(scale=NAN), 1), (dict(scale=INF), 1),
    (dict(pre=(3, 1e-5, None, None)), 1), (dict(pre=(-1, 1e-5, None, None)), 1), (dict(pre=(1, -1e-5, None, None)), 1),
    (dict(pre=(1, NAN, None, None)), 1), (dict(post=(2, INF, None, None)), 1), (dict(post=(2, 0.0, FAKE + 2, None)), 1),
    (dict(pre=(1, 1e-5, None, FAKE + 8)), 1), (dict(gate=FAKE + 2), 1), (dict(gate=FAKE, gs=512), 1),
    (dict(gate=FAKE, gs=1025), 1), (dict(res=FAKE + 8), 1), (dict(res=FAKE, rs=1028), 1), (dict(h=FAKE + 4), 1),
    (dict(res=FAKE + 0x10000, h=FAKE + 0x10000, hs=2048), 1),         # in place with another stride
    (dict(h=FAKE, hs=2048), 1), (dict(h=FAKE, hd=1), 1),              # x itself with another stride or type
    (dict(y=FAKE, ys=2048), 1), (dict(y=FAKE, yd=1), 1), (dict(h=FAKE + 0x100000), 1),
    (dict(h=FAKE, hd=1, T=1), 1), (dict(y=FAKE, yd=1, T=1), 1),       # also for a single token
    (dict(res=FAKE + 0x200000, y=FAKE + 0x200000, hd=1), 1), (dict(gate=FAKE + 0x100000), 1), (dict(T=2 ** 31 - 4095), 1),
    (dict(xs=1026, xd=1), 1), (dict(Dm=16392, xs=16392, ys=16392), 2),
])
def test_residual_norm_refusals(lib, bad, status):
    assert norm(lib, **bad) == status
