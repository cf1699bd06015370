"""GPU checks of dr_rope_table and dr_rope_append against 64-bit rotations; untouched slots keep their bits."""
import math

import numpy as np
import pytest
import torch

from decode_attention_self_gb300 import workloads as W
from prompt_reference import Cache, D, assert_close, starts, to64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api(cuda_device):
    from decode_attention_self_gb300 import api as _api

    return _api


def table64(n, rot, base=10000.0):
    ang = torch.arange(n, dtype=torch.float64)[:, None] * base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    return torch.cat([ang.cos(), ang.sin()], 1)


@pytest.mark.parametrize("rot,n,base", [(16, 1, 10000.0), (32, 77, 10000.0), (48, 1000, 500000.0), (64, 300001, 1e6)])
def test_rope_table(api, cuda_device, rot, n, base):
    t = torch.zeros(n, rot, dtype=torch.float32, device=cuda_device)
    api.dr_rope_table(t, base)
    ref = table64(n, rot, base)
    # one rounding to fp32, and 64-bit angles of up to 3e5 radians (off by 2^-53 * 3e5 * 2)
    assert ((t.cpu().double() - ref).abs() <= 2.0 ** -24 * ref.abs() + 1e-10).all()


def rotate(x, tab, inter):
    """x [n, H, D] float64, tab [n, rot] -> (rotated, error bound of fp32 products and sum)."""
    rot = tab.shape[1]
    c, s = tab[:, None, :rot // 2].double(), tab[:, None, rot // 2:].double()
    i1 = torch.arange(0, rot, 2) if inter else torch.arange(rot // 2)
    i2 = i1 + (1 if inter else rot // 2)
    y, e = x.clone(), torch.zeros_like(x)
    x1, x2 = x[..., i1], x[..., i2]
    y[..., i1], y[..., i2] = x1 * c - x2 * s, x2 * c + x1 * s
    e[..., i1] = e[..., i2] = 3 * 2.0 ** -24 * (x1.abs() + x2.abs())
    return y, e


CASES = [  # lens, starts, Hq, Hkv, paged, fp8, rot, interleaved, offset, packed
    ([1], [0], 1, 1, False, False, 64, False, 0, False),
    ([1], [37], 16, 16, True, False, 64, False, 0, True),
    ([1] * 128, list(range(0, 256, 2)), 16, 16, True, True, 64, True, 7, True),
    ([5, 0, 1, 33, 0, 16], [0, 3, 15, 16, 0, 31], 8, 2, True, False, 32, False, 100, True),
    ([0, 0, 3], [1, 2, 3], 6, 2, False, True, 48, True, 0, False),
    ([257, 64], [0, 5], 4, 4, False, False, 16, False, 0, True),
    ([100], [29], 32, 1, True, True, 0, False, 0, False),
    ([1500, 700, 1], [0, 11, 2], 16, 4, True, True, 64, False, 5000, True),
    ([40] * 70, [0] * 70, 3, 3, True, False, 64, True, 0, False),
]


@pytest.mark.parametrize("lens,start,Hq,Hkv,paged,fp8,rot,inter,offset,packed", CASES)
def test_rope_append(api, cuda_device, lens, start, Hq, Hkv, paged, fp8, rot, inter, offset, packed):
    dev = cuda_device
    B, used = len(lens), sum(lens)
    T = used + 3                                     # three tokens behind the last row
    caps = [n + s for n, s in zip(lens, start)]
    cache = Cache(caps, Hkv, paged, fp8, seed=sum(caps) + Hq)
    qkv = W.randn_bf16((T, Hq + 2 * Hkv, D), "cpu", 55, T)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    g = qkv.to(dev)
    gq, gk, gv = g[:, :Hq], g[:, Hq:Hq + Hkv], g[:, Hq + Hkv:]
    if not packed:
        gq, gk, gv = gq.contiguous(), gk.contiguous(), gv.contiguous()
    kv = cache.gpu(api, dev)
    q_out = torch.full((T, Hq, D), 9.0, dtype=torch.bfloat16, device=dev)
    n_tab = max(caps) + offset
    tab = table64(n_tab, rot).float() if rot else None
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    off = torch.full((B,), offset, dtype=torch.int32, device=dev) if offset else None
    api.dr_rope_append(kv, gk, gv, starts(lens).to(dev), torch.tensor(start, dtype=torch.int32, device=dev), q=gq,
                       q_out=q_out, table=None if tab is None else tab.to(dev), interleaved=inter, pos_offset=off,
                       err_flag=err)
    assert int(err.item()) == 0
    want_k, want_v = cache.k.clone(), cache.v.clone()
    got_k, got_v = kv.k.cpu(), kv.v.cpu()
    at = 0
    for b, (n, s) in enumerate(zip(lens, start)):
        if n == 0:
            continue
        i0, i2 = (i[s:] for i in cache.slots(b, s + n))
        xq, xk = q[at:at + n].double(), k[at:at + n].double()
        eq, ek = torch.zeros_like(xq), torch.zeros_like(xk)
        if rot:
            rows = tab[s + offset:s + offset + n]
            (xq, eq), (xk, ek) = rotate(xq, rows, inter), rotate(xk, rows, inter)
        assert_close(q_out[at:at + n], xq, eq + 2.0 ** -8 * xq.abs() + 2.0 ** -130, "q")
        gotk = got_k[i0, :, i2]
        if fp8:
            # the code of x / scale: half a step of e4m3 (2^-4 of the value, 2^-10 below the normal range), saturating
            x = xk / cache.k_scale
            lim = x.clamp(-448, 448)
            assert_close(to64(gotk, 1.0), lim, ek / cache.k_scale + 2.0 ** -4 * lim.abs() + 2.0 ** -10, "k codes")
            want = W.to_e4m3_codes(v[at:at + n], cache.v_scale)
            assert torch.equal(got_v[i0, :, i2], want)
        else:
            assert_close(gotk, xk, ek + 2.0 ** -8 * xk.abs() + 2.0 ** -130, "k")
            assert torch.equal(got_v[i0, :, i2].view(torch.int16), v[at:at + n].contiguous().view(torch.int16))
        want_k[i0, :, i2] = gotk
        want_v[i0, :, i2] = got_v[i0, :, i2]
        at += n
    # every other slot and every token behind the last row keeps its bits
    bits = (lambda t: t if fp8 else t.view(torch.int16))
    assert torch.equal(bits(got_k), bits(want_k)) and torch.equal(bits(got_v), bits(want_v))
    assert (q_out[used:] == 9.0).all()
    # without q: the same cache
    kv2 = cache.gpu(api, dev)
    api.dr_rope_append(kv2, gk, gv, starts(lens).to(dev), torch.tensor(start, dtype=torch.int32, device=dev),
                       table=None if tab is None else tab.to(dev), interleaved=inter, pos_offset=off)
    assert torch.equal(bits(kv2.k.cpu()), bits(got_k)) and torch.equal(bits(kv2.v.cpu()), bits(got_v))


def test_unrotated_append_equals_kv_append(api, cuda_device):
    dev = cuda_device
    for fp8 in (False, True):
        cache = Cache([40, 17, 300], 16, True, fp8, seed=3)
        k, v = W.randn_bf16((3, 16, D), dev, 1), W.randn_bf16((3, 16, D), dev, 2)
        pos = torch.tensor([39, 0, 255], dtype=torch.int32, device=dev)
        a, b = cache.gpu(api, dev), cache.gpu(api, dev)
        api.dr_kv_append(a, k, v, pos)
        api.dr_rope_append(b, k, v, starts([1, 1, 1]).to(dev), pos)
        view = torch.uint8 if fp8 else torch.int16
        assert torch.equal(a.k.view(view), b.k.view(view)) and torch.equal(a.v.view(view), b.v.view(view))


@pytest.mark.parametrize("k_scale,v_scale", [(1 / 64, 0.0173), (0.75, 2.0 ** -20), (2.0 ** -126, 3e-39), (2.0 ** 90, 7.3),
                                             (2.0 ** 127, 2.0 ** -124)])
def test_codes_of_any_scale_equal_kv_append(api, cuda_device, k_scale, v_scale):
    """The same codes as dr_kv_append's divisions, for scales that are powers of two and others, ties and tiny values."""
    dev = cuda_device
    cache = Cache([40, 17, 300], 16, True, True, seed=3, k_scale=k_scale, v_scale=v_scale)
    gain = torch.tensor([1.0, 2.0 ** -9, 200.0]).view(3, 1, 1)
    k, v = ((W.randn_bf16((3, 16, D), "cpu", i).float() * gain * s).to(torch.bfloat16).to(dev)
            for i, s in ((1, k_scale), (2, v_scale)))
    pos = torch.tensor([39, 0, 255], dtype=torch.int32, device=dev)
    a, b = cache.gpu(api, dev), cache.gpu(api, dev)
    api.dr_kv_append(a, k, v, pos)
    api.dr_rope_append(b, k, v, starts([1, 1, 1]).to(dev), pos)
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
    assert len(a.k.unique()) > 100


def test_rotation_in_place(api, cuda_device):
    dev = cuda_device
    q = W.randn_bf16((50, 16, D), dev, 1)
    k, v = W.randn_bf16((50, 4, D), dev, 2), W.randn_bf16((50, 4, D), dev, 3)
    tab = table64(60, 64).float().to(dev)
    cache = Cache([60], 4, False, False, seed=4)
    args = (starts([50]).to(dev), torch.tensor([10], dtype=torch.int32, device=dev))
    apart = torch.empty_like(q)
    api.dr_rope_append(cache.gpu(api, dev), k, v, *args, q=q, q_out=apart, table=tab)
    api.dr_rope_append(cache.gpu(api, dev), k, v, *args, q=q, q_out=q, table=tab)
    assert torch.equal(q, apart)


def test_positions_outside_are_flagged_and_left_out(api, cuda_device):
    dev = cuda_device
    cache = Cache([32, 32, 32, 32], 2, True, False, seed=5)
    table = cache.table.clone()
    table[1, 1] = -1
    table[2, 1] = 10 ** 6
    kv = api.KVCache(cache.k.to(dev), cache.v.to(dev), table.to(dev))
    k, v = W.randn_bf16((8, 2, D), dev, 1), W.randn_bf16((8, 2, D), dev, 2)
    q, q_out = W.randn_bf16((8, 4, D), dev, 3), torch.full((8, 4, D), 5.0, dtype=torch.bfloat16, device=dev)
    tab = table64(34, 64).float().to(dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    # row 0: slots 31, 32 (32 is past the capacity); row 1: 15, 16 (unmapped); row 2: 16, 17 (outside); row 3: -1, 0
    api.dr_rope_append(kv, k, v, starts([2, 2, 2, 2]).to(dev), torch.tensor([31, 15, 16, -1], dtype=torch.int32, device=dev),
                       q=q, q_out=q_out, table=tab, err_flag=err)
    assert int(err.item()) == api.DR_ERRF_POS
    got = kv.k.cpu()
    same = got.view(torch.int16) == cache.k.view(torch.int16)
    changed = (~same.all(-1).all(1)).nonzero().tolist()
    want = sorted([[int(table[0, 1]), 15], [int(table[1, 0]), 15], [int(table[3, 0]), 0]])
    assert sorted(changed) == want
    assert (q_out[6] == 5.0).all() and not (q_out[[0, 1, 2, 3, 4, 5, 7]] == 5.0).all(-1).any()


def test_rows_that_do_not_rise_are_cut(api, cuda_device):
    dev = cuda_device
    cache = Cache([64, 64], 2, False, False, seed=6)
    k, v = W.randn_bf16((10, 2, D), dev, 1), W.randn_bf16((10, 2, D), dev, 2)
    sp = torch.zeros(2, dtype=torch.int32, device=dev)
    for rs in ([0, 5, 99], [-3, 5, 10], [0, 10, 4000000]):
        err = torch.zeros(1, dtype=torch.int32, device=dev)
        kv = cache.gpu(api, dev)
        api.dr_rope_append(kv, k, v, torch.tensor(rs, dtype=torch.int32, device=dev), sp, err_flag=err)
        assert int(err.item()) == api.DR_ERRF_ROW_START, rs


def test_binding_refusals(api, cuda_device):
    dev = cuda_device
    cache = Cache([32], 2, False, False, seed=7)
    kv = cache.gpu(api, dev)
    k, v = W.randn_bf16((2, 2, D), dev, 1), W.randn_bf16((2, 2, D), dev, 2)
    rs, sp = starts([2]).to(dev), torch.zeros(1, dtype=torch.int32, device=dev)
    with pytest.raises(ValueError):
        api.dr_rope_append(kv, k.cpu(), v, rs, sp)
    with pytest.raises(ValueError):
        api.dr_rope_append(kv, k.float(), v, rs, sp)
    with pytest.raises(ValueError):
        api.dr_rope_append(kv, k, v[:1], rs, sp)
    with pytest.raises(ValueError):
        api.dr_rope_append(kv, k, v, rs[:1], sp)
    with pytest.raises(ValueError):
        api.dr_rope_append(kv, k.transpose(0, 1), v.transpose(0, 1), rs, sp)
    with pytest.raises(ValueError):
        api.dr_rope_append(kv, k[:, :1], v[:, :1], rs, sp)       # the cache has two heads
    with pytest.raises(ValueError):
        api.dr_rope_append(kv, k, v, rs.long(), sp)
    with pytest.raises(api.DrError):
        api.dr_rope_append(kv, k, v, rs, sp, q=k)                # q without q_out
