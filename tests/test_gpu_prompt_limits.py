"""GPU checks of the prompt-side operators at their limits: offsets past 32 bits in static and paged caches, the most
rows, many rows of mixed lengths, long rows, and launches that follow one another without a pause."""
import numpy as np
import pytest
import torch

from decode_attention_self_gb300 import workloads as W
from prompt_reference import D, PAGE, assert_close, attend, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api(cuda_device):
    from decode_attention_self_gb300 import api as _api

    return _api


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def big_cache(api, dev, paged, fp8):
    """A cache whose last row's keys lie past 2^32 elements; (KVCache, keys per row, row, slot -> (i0, i2))."""
    Hkv = 16
    dt = torch.uint8 if fp8 else torch.bfloat16
    if paged:
        blocks, cap = 300_000, 4096
        k, v = (torch.empty((blocks, Hkv, PAGE, D), dtype=dt, device=dev) for _ in range(2))
        table = torch.full((3, cap // PAGE), -1, dtype=torch.int32)
        table[2] = torch.arange(blocks - cap // PAGE, blocks, dtype=torch.int32).flip(0)
        c = api.KVCache(k, v, table.to(dev), 1 / 64 if fp8 else 1.0, 1 / 32 if fp8 else 1.0)
        return c, cap, lambda j: (table[2].long()[j // PAGE].to(dev), (j % PAGE).to(dev))
    cap = 1_500_000
    k, v = (torch.empty((3, Hkv, cap, D), dtype=dt, device=dev) for _ in range(2))
    c = api.KVCache(k, v, None, 1 / 64 if fp8 else 1.0, 1 / 32 if fp8 else 1.0)
    return c, cap, lambda j: (torch.full_like(j, 2).to(dev), j.to(dev))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("paged", [False, True])
def test_offsets_past_32_bits(api, cuda_device, paged, fp8):
    dev = cuda_device
    c, cap, at = big_cache(api, dev, paged, fp8)
    assert c.k.numel() > 2 ** 32
    Hq, Hkv, n = 32, 16, 300
    k, v = W.randn_bf16((n, Hkv, D), dev, 1), W.randn_bf16((n, Hkv, D), dev, 2)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    # rows 0 and 1 get nothing; row 2's last 300 slots are written
    api.dr_rope_append(c, k, v, i32([0, 0, 0, n], dev), i32([0, 0, cap - n], dev), err_flag=err)
    j = torch.arange(cap - n, cap)
    i0, i2 = at(j)
    if fp8:
        K, V = (x.view(torch.uint8)[i0, :, i2].view(torch.float8_e4m3fn).double() * s
                for x, s in ((c.k, c.k_scale), (c.v, c.v_scale)))
        want = W.to_e4m3_codes(k, c.k_scale)
        assert torch.equal(c.k[i0, :, i2], want)
    else:
        K, V = c.k[i0, :, i2].double(), c.v[i0, :, i2].double()
        assert torch.equal(K, k.double()) and torch.equal(V, v.double())
    K, V = K.transpose(0, 1).cpu(), V.transpose(0, 1).cpu()
    for m in (1, 150):                                    # the token kernel, the tile kernel
        q = W.randn_bf16((m, Hq, D), dev, 3, m)
        out = torch.empty((m, Hq, D), device=dev)
        api.dr_prompt_attn(q, c, i32([0, 0, 0, m], dev), i32([0, 0, cap], dev), out,
                           first_key=i32([cap - n + 7] * m, dev), err_flag=err)
        pos = torch.arange(n - m, n)
        ref, tol = attend(q.cpu(), K, V, torch.full((m,), 7), pos + 1, pos, fp8=fp8)
        assert_close(out, ref, tol, f"{m} tokens")
    assert int(err.item()) == 0


def test_most_rows(api, cuda_device):
    dev = cuda_device
    B = 65535
    k, v = (W.randn_bf16((B, 1, 16, D), dev, 5, i) for i in range(2))
    c = api.KVCache(k, v)
    q = W.randn_bf16((B, 1, D), dev, 6)
    lens = torch.randint(1, 17, (B,), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    out, err = torch.empty((B, 1, D), device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    rs = torch.arange(B + 1, dtype=torch.int32, device=dev)
    api.dr_prompt_attn(q, c, rs, lens.to(dev), out, err_flag=err)
    s = torch.einsum("bd,bjd->bj", q[:, 0].double(), k[:, 0].double()) / 8
    s = s.masked_fill(torch.arange(16, device=dev)[None] >= lens.to(dev)[:, None], -float("inf"))
    p = torch.softmax(s, 1)
    ref = torch.einsum("bj,bjd->bd", p, v[:, 0].double())
    tol = (2.0 ** -8 + 1e-4) * torch.einsum("bj,bjd->bd", p, v[:, 0].double().abs())   # see prompt_reference
    assert ((out[:, 0].double() - ref).abs() <= tol).all() and int(err.item()) == 0
    new_k = W.randn_bf16((B, 1, D), dev, 7)
    api.dr_rope_append(c, new_k, new_k, rs, lens.to(dev) - 1, err_flag=err)
    at = (torch.arange(B, device=dev), (lens.long() - 1).to(dev))
    assert torch.equal(c.k[at[0], 0, at[1]], new_k[:, 0]) and int(err.item()) == 0
    ws = torch.empty(api.dr_shared_prefix_attn_workspace(B, 1, 1, 16), dtype=torch.uint8, device=dev)
    pre = api.KVCache(k[:1].contiguous(), v[:1].contiguous())
    api.dr_shared_prefix_attn(q, pre, i32([16], dev), out, ws, err_flag=err)
    s = torch.einsum("bd,jd->bj", q[:, 0].double(), pre.k[0, 0].double()) / 8
    p = torch.softmax(s, 1)
    ref, tol = p @ pre.v[0, 0].double(), (2.0 ** -8 + 1e-4) * (p @ pre.v[0, 0].double().abs())
    assert ((out[:, 0].double() - ref).abs() <= tol).all() and int(err.item()) == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_thousands_of_rows_of_mixed_lengths(api, cuda_device, fp8):
    """Rows of no, one and several tokens: the search over rows, and both kernels in one call."""
    dev = cuda_device
    rng = np.random.default_rng(4)
    B = 3000
    new = rng.choice([0, 1, 1, 1, 2, 9], size=B)
    kv = np.where(new > 0, new + rng.integers(0, 20, size=B), 0)
    T = int(new.sum())
    k, v = (W.randn_bf16((B, 2, 32, D), dev, 9, i) for i in range(2))
    if fp8:
        c = api.KVCache(W.to_e4m3_codes(k, 1 / 64), W.to_e4m3_codes(v, 1 / 32), None, 1 / 64, 1 / 32)
        k, v = c.k.view(torch.float8_e4m3fn).double() / 64, c.v.view(torch.float8_e4m3fn).double() / 32
    else:
        c = api.KVCache(k, v)
        k, v = k.double(), v.double()
    q = W.randn_bf16((T, 4, D), dev, 10)
    out, err = torch.empty((T, 4, D), device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    api.dr_prompt_attn(q, c, starts(new).to(dev), torch.tensor(kv, dtype=torch.int32, device=dev), out, err_flag=err)
    assert int(err.item()) == 0
    row = torch.from_numpy(np.repeat(np.arange(B), new)).to(dev)
    pos = torch.from_numpy(np.concatenate([np.arange(L - n, L) for n, L in zip(new, kv)])).to(dev)
    kk, vv = k[row].repeat_interleave(2, 1), v[row].repeat_interleave(2, 1)          # [T, 4, 32, D]
    s = torch.einsum("thd,thjd->thj", q.double(), kk) / 8
    s = s.masked_fill(torch.arange(32, device=dev)[None, None] > pos[:, None, None], -float("inf"))
    p = torch.softmax(s, -1)
    ref = torch.einsum("thj,thjd->thd", p, vv)
    tol = ((2.0 ** -11 if fp8 else 2.0 ** -8) + 1e-4) * torch.einsum("thj,thjd->thd", p, vv.abs())
    assert ((out.double() - ref).abs() <= tol).all()


def test_long_row_split_and_not(api, cuda_device):
    """A token and a chunk at the end of 131072 keys, with and without a workspace: within rounding of each other and of
    64 bits."""
    dev = cuda_device
    L, Hq, Hkv = 131072, 4, 1
    k, v = (W.randn_bf16((1, Hkv, L, D), dev, 11, i) for i in range(2))
    c = api.KVCache(k, v)
    for m in (1, 33):
        q = W.randn_bf16((m, Hq, D), dev, 12, m)
        nb = api.dr_prompt_attn_workspace(m, 1, Hq, Hkv, L)
        assert (nb > 0) == (m > 1)
        for ws in (None, torch.empty(max(nb, 32), dtype=torch.uint8, device=dev)):
            out = torch.empty((m, Hq, D), device=dev)
            api.dr_prompt_attn(q, c, i32([0, m], dev), i32([L], dev), out, workspace=ws)
            kk, vv = k[0, 0].double(), v[0, 0].double()
            s = torch.einsum("thd,jd->thj", q.double(), kk) / 8
            pos = torch.arange(L - m, L, device=dev)
            s = s.masked_fill(torch.arange(L, device=dev)[None, None] > pos[:, None, None], -float("inf"))
            p = torch.softmax(s, -1)
            # fp32 sums of 131072 weights in a fixed order: 1024 tiles or passes, each rounded to 2^-24, twice
            tol = (2.0 ** -8 + 1e-4 + 2048 * 2.0 ** -24) * (p @ vv.abs())
            assert ((out.double() - p @ vv).abs() <= tol).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_steps_without_a_pause_read_what_was_just_written(api, cuda_device, fp8):
    """400 steps in a graph: every step appends a key and value of its own over the same slots and attends prefix and own
    keys; each step's output is that of the same step run alone."""
    dev = cuda_device
    B, Hq, Hkv, P, own, steps = 24, 8, 4, 700, 40, 400
    pre = api.KVCache(*(W.randn_bf16((1, Hkv, P, D), dev, 20, i) for i in range(2)))
    kc, vc = (W.randn_bf16((B, Hkv, own, D), dev, 21, i) for i in range(2))
    if fp8:
        pre = api.KVCache(*(W.to_e4m3_codes(x, 1 / 64) for x in (pre.k, pre.v)), None, 1 / 64, 1 / 64)
        kc, vc = W.to_e4m3_codes(kc, 1 / 64), W.to_e4m3_codes(vc, 1 / 64)
    c = api.KVCache(kc, vc, None, *((1 / 64, 1 / 64) if fp8 else (1.0, 1.0)))
    q, k, v = (W.randn_bf16((steps, B, h, D), dev, 22, h + i) for i, h in enumerate((Hq, Hkv, Hkv)))
    rs, pos, seq, plen = starts([1] * B).to(dev), i32([own - 1] * B, dev), i32([own] * B, dev), i32([P], dev)
    ws = torch.empty(api.dr_shared_prefix_attn_workspace(B, Hq, Hkv, P), dtype=torch.uint8, device=dev)
    outs, alone = torch.empty((steps, B, Hq, D), device=dev), torch.empty((steps, B, Hq, D), device=dev)

    def step(i, out):
        api.dr_rope_append(c, k[i], v[i], rs, pos)
        api.dr_shared_prefix_attn(q[i], pre, plen, out[i], ws, cache=c, seq_len=seq)

    step(0, outs)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for i in range(steps):
            step(i, outs)
    g.replay()
    torch.cuda.synchronize()
    for i in range(steps):
        step(i, alone)
        torch.cuda.synchronize()
    assert torch.equal(outs, alone)
