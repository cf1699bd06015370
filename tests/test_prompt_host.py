"""Host-side refusals of the prompt-side operators: every mistake the host can see is refused before a launch."""
import ctypes

import pytest

FAKE = 0x10000   # a 16-byte aligned non-null address; never dereferenced on the host


class Cache(ctypes.Structure):
    _fields_ = [("layout", ctypes.c_int32), ("max_len", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("num_blocks", ctypes.c_int32), ("max_blocks_per_seq", ctypes.c_int32), ("kv_dtype", ctypes.c_int32),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


class Opts(ctypes.Structure):
    _fields_ = [("causal", ctypes.c_int32), ("softcap", ctypes.c_float), ("slopes", ctypes.c_void_p),
                ("prefix_len", ctypes.c_void_p), ("first_key", ctypes.c_void_p)]


GOOD = dict(layout=0, max_len=2048, k=FAKE, v=FAKE)
BAD_CACHES = [(dict(GOOD, k=None), 1), (dict(GOOD, v=FAKE + 8), 1), (dict(GOOD, layout=3), 1),
              (dict(GOOD, max_len=0), 1), (dict(GOOD, kv_dtype=4), 1),
              (dict(GOOD, kv_dtype=1, k_scale=0.0, v_scale=1.0), 1),
              (dict(GOOD, kv_dtype=1, k_scale=1.0, v_scale=float("inf")), 1),
              (dict(layout=1, block_size=16, num_blocks=4, max_blocks_per_seq=2, k=FAKE, v=FAKE), 1),
              (dict(layout=1, block_size=32, num_blocks=4, max_blocks_per_seq=2, k=FAKE, v=FAKE, block_table=FAKE), 2),
              (dict(GOOD, max_len=2 ** 31 - 4095), 1),     # key numbers past a row's end have to fit 32 bits
              (dict(layout=1, block_size=16, num_blocks=4, max_blocks_per_seq=1 << 27, k=FAKE, v=FAKE, block_table=FAKE), 1),
              (dict(layout=1, block_size=16, num_blocks=0, max_blocks_per_seq=2, k=FAKE, v=FAKE, block_table=FAKE), 1)]


@pytest.fixture(scope="module")
def lib():
    from decode_attention_self_gb300 import build

    return ctypes.CDLL(build.build())


def vp(x):
    return ctypes.c_void_p(x)


def rope(lib, cache=None, q=FAKE, qs=1024, k=FAKE, ks=1024, v=FAKE, vs=1024, qo=FAKE, qos=1024, rs=FAKE, sp=FAKE,
         po=None, table=FAKE, rope_len=64, rot=64, inter=0, T=4, B=2, Hq=16, Hkv=16, D=64):
    c = Cache(**(cache or GOOD))
    i64 = ctypes.c_int64
    return lib.dr_rope_append(ctypes.byref(c), vp(q), i64(qs), vp(k), i64(ks), vp(v), i64(vs), vp(qo), i64(qos), vp(rs),
                              vp(sp), vp(po), vp(table), rope_len, rot, inter, T, B, Hq, Hkv, D, None, None)


@pytest.mark.parametrize("bad,status", [
    (dict(T=0), 1), (dict(B=0), 1), (dict(B=65536), 1), (dict(Hq=0), 1), (dict(Hkv=5), 1), (dict(D=128), 2),
    (dict(k=None), 1), (dict(v=None), 1), (dict(rs=None), 1), (dict(sp=None), 1), (dict(k=FAKE + 2), 1),
    (dict(q=None), 1), (dict(qo=None), 1), (dict(qo=FAKE + 8), 1), (dict(ks=1020), 1), (dict(vs=512), 1),
    (dict(qs=1028), 1), (dict(qos=64), 1), (dict(inter=2), 1), (dict(rot=8), 2), (dict(rot=40), 2), (dict(rot=80), 2),
    (dict(rope_len=0), 1), (dict(table=FAKE + 4), 1), (dict(T=1 << 30, Hq=16), 1), (dict(Hq=258, Hkv=2, qs=1 << 15, qos=1 << 15), 2),
])
def test_rope_append_refusals(lib, bad, status):
    assert rope(lib, **bad) == status


@pytest.mark.parametrize("cache,status", BAD_CACHES)
def test_rope_append_refuses_bad_caches(lib, cache, status):
    assert rope(lib, cache=cache) == status


def test_rope_table_refusals(lib):
    d = ctypes.c_double
    call = lambda t=FAKE, n=8, rot=64, base=1e4: lib.dr_rope_table(vp(t), n, rot, d(base), None)
    assert call(t=None) == 1 and call(t=FAKE + 4) == 1 and call(n=0) == 1 and call(base=0.0) == 1
    assert call(base=float("inf")) == 1 and call(base=float("nan")) == 1
    assert call(rot=8) == 2 and call(rot=24) == 2 and call(rot=128) == 2


def prompt(lib, cache=None, q=FAKE, qs=1024, rs=FAKE, kl=FAKE, opts=None, T=4, B=2, Hq=16, Hkv=16, D=64, scale=0.0,
           out=FAKE, od=0, ws=None, ws_bytes=0):
    c = Cache(**(cache or GOOD))
    o = None if opts is None else ctypes.byref(Opts(**opts))
    return lib.dr_prompt_attn(vp(q), ctypes.c_int64(qs), ctypes.byref(c), vp(rs), vp(kl), o, T, B, Hq, Hkv, D, 0,
                              ctypes.c_float(scale), vp(out), od, vp(ws), ctypes.c_size_t(ws_bytes), None, None)


@pytest.mark.parametrize("bad,status", [
    (dict(T=0), 1), (dict(B=0), 1), (dict(Hkv=3), 1), (dict(D=32), 2), (dict(q=None), 1), (dict(rs=None), 1),
    (dict(kl=None), 1), (dict(out=None), 1), (dict(q=FAKE + 4), 1), (dict(out=FAKE + 2), 1), (dict(qs=1000), 1),
    (dict(qs=1029), 1), (dict(od=7), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(ws=FAKE + 8, ws_bytes=64), 1), (dict(opts=dict(causal=2)), 1), (dict(opts=dict(causal=1, softcap=-1.0)), 1),
    (dict(opts=dict(causal=1, softcap=float("nan"))), 1), (dict(opts=dict(causal=1, softcap=1e-9)), 1),
    (dict(out=FAKE + 16), 1), (dict(ws=FAKE + 16, ws_bytes=64), 1), (dict(cache=dict(GOOD, k=FAKE + 16)), 1),
    (dict(cache=dict(GOOD, v=FAKE + 16)), 1), (dict(opts=dict(causal=0, prefix_len=FAKE)), 1), (dict(Hq=258, Hkv=2, qs=1 << 15), 2),
])
def test_prompt_attn_refusals(lib, bad, status):
    assert prompt(lib, **bad) == status


@pytest.mark.parametrize("cache,status", BAD_CACHES)
def test_prompt_attn_refuses_bad_caches(lib, cache, status):
    assert prompt(lib, cache=cache) == status


def shared(lib, prefix=None, own=None, seq=FAKE, opts=None, q=FAKE, qs=1024, pl=FAKE, B=2, Hq=16, Hkv=16, D=64, scale=0.0,
           out=FAKE, od=0, ws=FAKE, ws_bytes=1 << 30):
    pc = Cache(**(prefix or GOOD))
    oc = None if own == "none" else ctypes.byref(Cache(**(own or GOOD)))
    o = None if opts is None else ctypes.byref(Opts(**opts))
    return lib.dr_shared_prefix_attn(vp(q), ctypes.c_int64(qs), ctypes.byref(pc), vp(pl), oc, vp(seq), o, B, Hq, Hkv, D, 0,
                                     0, ctypes.c_float(scale), vp(out), od, vp(ws), ctypes.c_size_t(ws_bytes), None, None)


@pytest.mark.parametrize("bad,status", [
    (dict(B=0), 1), (dict(Hkv=3), 1), (dict(D=128), 2), (dict(q=None), 1), (dict(pl=None), 1), (dict(out=None), 1),
    (dict(seq=None), 1), (dict(own="none"), 1), (dict(ws=None), 1), (dict(ws=FAKE + 8), 1),
    (dict(ws_bytes=2 * 16 * 66 * 4 - 1), 1), (dict(opts=dict(first_key=FAKE)), 1), (dict(opts=dict(causal=1, prefix_len=FAKE)), 1),
    (dict(od=3), 1), (dict(qs=8), 1), (dict(scale=float("nan")), 1), (dict(out=FAKE + 4), 1), (dict(out=FAKE + 16), 1),
    (dict(ws=FAKE + 16), 1), (dict(prefix=dict(GOOD, k=FAKE + 16)), 1), (dict(own=dict(GOOD, v=FAKE + 16)), 1),
])
def test_shared_prefix_refusals(lib, bad, status):
    assert shared(lib, **bad) == status


@pytest.mark.parametrize("cache,status", BAD_CACHES)
def test_shared_prefix_refuses_bad_caches(lib, cache, status):
    assert shared(lib, prefix=cache) == status
    assert shared(lib, own=cache) == status


def test_workspace_sizes(lib):
    lib.dr_prompt_attn_workspace.restype = lib.dr_shared_prefix_attn_workspace.restype = ctypes.c_size_t
    prompt_ws, shared_ws = lib.dr_prompt_attn_workspace, lib.dr_shared_prefix_attn_workspace
    assert prompt_ws(1, 1, 16, 16, 4096, 152) == 0            # single tokens take none
    assert prompt_ws(128, 128, 16, 16, 4096, 152) == 0
    assert prompt_ws(1 << 20, 4, 16, 16, 1 << 18, 152) == 0   # enough tiles to fill the GPU
    assert prompt_ws(64, 1, 16, 16, 255, 152) == 0            # too few keys to share out
    assert prompt_ws(64, 1, 16, 16, 65536, 152) == 19 * 64 * 16 * 66 * 4
    assert shared_ws(128, 16, 16, 1, 152) == 128 * 16 * 66 * 4
    assert shared_ws(128, 16, 16, 65536, 152) == 19 * 128 * 16 * 66 * 4
    for bad in ((0, 1, 16, 16, 9, 152), (4, 1, 16, 5, 9, 152), (4, 1, 16, 16, 0, 152), (4, 1, 16, 16, 9, 0)):
        assert prompt_ws(*bad) == 0
    assert shared_ws(0, 16, 16, 9, 152) == 0 and shared_ws(4, 16, 5, 9, 152) == 0
