"""GPU checks of dr_shared_prefix_attn against 64-bit attention over the prefix and each row's own keys, and of the
prompt-side operators run together as a serving loop runs them."""
import pytest
import torch

from decode_attention_self_gb300 import workloads as W
from prompt_reference import Cache, D, assert_close, attend, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api(cuda_device):
    from decode_attention_self_gb300 import api as _api

    return _api


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def reference(prefix, P, cache, own, q, softcap, slopes, fp8, out_dtype, scale=D ** -0.5):
    pk, pv = prefix.rows(0, P)
    refs, tols = [], []
    for b, n in enumerate(own):
        k, v = (pk, pv)
        if cache is not None:
            ok, ov = cache.rows(b, n)
            k, v = torch.cat([pk, ok], 1), torch.cat([pv, ov], 1)
        L = P + n
        r, t = attend(q[b:b + 1], k, v, torch.zeros(1, dtype=torch.long), torch.tensor([L]), torch.tensor([L - 1]), scale,
                      softcap, slopes, fp8, out_dtype)
        refs.append(r)
        tols.append(t)
    return torch.cat(refs), torch.cat(tols)


def check(api, dev, P, own, Hq, Hkv, paged=True, fp8=False, softcap=0.0, bias=False, out_dtype=torch.float32, seed=1,
          hints=True, no_own=False, small_ws=False, pad=0):
    B = len(own)
    prefix = Cache([max(P, 1) + 5], Hkv, paged, fp8, seed, valid=[P])
    cache = None if no_own else Cache([max(n, 1) for n in own], Hkv, paged, fp8, seed + 1, valid=own)
    q = W.randn_bf16((B, Hq + pad, D), "cpu", seed, 7)
    slopes = torch.tensor([2.0 ** (-(i % 7) - 2) for i in range(Hq)]) if bias else None
    out = torch.empty((B, Hq, D), dtype=out_dtype, device=dev)
    ws = torch.full((api.dr_shared_prefix_attn_workspace(B, Hq, Hkv, 1 if small_ws else P + 5),), 255, dtype=torch.uint8,
                    device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    api.dr_shared_prefix_attn(q.to(dev)[:, :Hq], prefix.gpu(api, dev), i32([P], dev), out, ws,
                              cache=None if no_own else cache.gpu(api, dev), seq_len=None if no_own else i32(own, dev),
                              softcap=softcap, slopes=None if slopes is None else slopes.to(dev),
                              max_prefix_hint=P if hints else 0, max_seq_len_hint=max(own) if hints else 0, err_flag=err)
    assert int(err.item()) == 0
    ref, tol = reference(prefix, P, cache, [0] * B if no_own else own, q[:, :Hq], softcap, slopes, fp8, out_dtype)
    assert_close(out, ref, tol, "shared prefix")
    return out


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("P,own,Hq,Hkv", [(1, [1], 1, 1), (16, [3, 0], 4, 4), (100, [1, 17, 64, 0, 5], 8, 2),
                                          (129, [200] * 7, 7, 1), (1000, [31] * 40, 16, 4), (5000, [7, 900, 0], 4, 4),
                                          (300, [2] * 130, 3, 3), (2048, [33] * 20, 32, 2)])
def test_shared_prefix(api, cuda_device, fp8, paged, P, own, Hq, Hkv):
    check(api, cuda_device, P, own, Hq, Hkv, paged, fp8, seed=P)


@pytest.mark.parametrize("fp8", [False, True])
def test_cap_bias_output_type_and_hints(api, cuda_device, fp8):
    check(api, cuda_device, 700, [5, 90, 0], 8, 2, True, fp8, softcap=3.0)
    check(api, cuda_device, 700, [5, 90, 0], 8, 2, True, fp8, bias=True)
    check(api, cuda_device, 700, [5, 90, 0], 8, 2, False, fp8, softcap=3.0, bias=True, out_dtype=torch.bfloat16, pad=3)
    check(api, cuda_device, 4000, [5, 90, 0], 8, 2, True, fp8, hints=False)
    check(api, cuda_device, 4000, [5, 90, 0], 8, 2, True, fp8, small_ws=True)


def test_no_own_keys_and_no_prefix(api, cuda_device):
    check(api, cuda_device, 333, [0] * 9, 4, 2, no_own=True)
    check(api, cuda_device, 0, [5, 40, 1], 4, 2)
    out = check(api, cuda_device, 0, [5, 0, 1], 4, 2, False, True)
    assert (out[1] == 0).all()


def test_split_of_a_long_prefix_and_many_rows(api, cuda_device):
    check(api, cuda_device, 33000, [10, 300], 2, 1, True, True)
    check(api, cuda_device, 20011, [10, 300], 2, 2, False, False)
    check(api, cuda_device, 257, [1] * 300, 4, 4, True, False)


def test_lengths_and_blocks_outside_are_flagged(api, cuda_device):
    dev = cuda_device
    prefix, cache = Cache([64], 2, True, False, 1), Cache([32, 32], 2, True, False, 2)
    q = W.randn_bf16((2, 4, D), dev, 3)
    ws = torch.empty(api.dr_shared_prefix_attn_workspace(2, 4, 2, 64), dtype=torch.uint8, device=dev)

    def flag(P, own, table=None):
        pre = Cache([64], 2, True, False, 1)
        if table is not None:
            pre.table[0, table[0]] = table[1]
        err = torch.zeros(1, dtype=torch.int32, device=dev)
        out = torch.empty((2, 4, D), device=dev)
        api.dr_shared_prefix_attn(q, pre.gpu(api, dev), i32([P], dev), out, ws, cache=cache.gpu(api, dev),
                                  seq_len=i32(own, dev), err_flag=err)
        assert torch.isfinite(out).all()
        return int(err.item())

    assert flag(64, [32, 0]) == 0
    assert flag(65, [32, 0]) == api.DR_ERRF_SEQ_LEN and flag(-1, [32, 0]) == api.DR_ERRF_SEQ_LEN
    assert flag(64, [33, 0]) == api.DR_ERRF_SEQ_LEN and flag(64, [2, -5]) == api.DR_ERRF_SEQ_LEN
    assert flag(64, [2, 2], (1, -1)) == api.DR_ERRF_BLOCK_ID
    assert flag(64, [2, 2], (3, 999)) == api.DR_ERRF_BLOCK_ID


def test_binding_refusals(api, cuda_device):
    dev = cuda_device
    prefix, cache = Cache([64], 2, True, False, 1).gpu(api, dev), Cache([32, 32], 2, True, False, 2).gpu(api, dev)
    q = W.randn_bf16((2, 4, D), dev, 3)
    out, sl = torch.empty_like(q), i32([1, 1], dev)
    ws = torch.empty(api.dr_shared_prefix_attn_workspace(2, 4, 2, 64), dtype=torch.uint8, device=dev)
    ok = dict(q=q, prefix=prefix, prefix_len=i32([9], dev), out=out, workspace=ws, cache=cache, seq_len=sl)
    api.dr_shared_prefix_attn(**ok)
    for bad in (dict(q=q.float()), dict(seq_len=None), dict(cache=None), dict(out=out[:1]), dict(workspace=ws.float()),
                dict(prefix_len=i32([9, 9], dev)), dict(slopes=torch.ones(2, device=dev)), dict(out=out.half())):
        with pytest.raises(ValueError):
            api.dr_shared_prefix_attn(**{**ok, **bad})
    with pytest.raises(api.DrError):
        api.dr_shared_prefix_attn(**{**ok, "workspace": ws[:16]})


@pytest.mark.parametrize("fp8", [False, True])
def test_serving_a_batch_of_one_voice(api, cuda_device, fp8):
    """A shared two-way prefix is written and attended; each row appends its own prompt behind it and attends prefix and
    prompt; then single tokens are appended and attend the prefix and their own keys.  Every output is compared with
    64-bit attention over the keys that the cache holds; single steps are captured in a graph and replayed."""
    dev = cuda_device
    P, B, Hq, Hkv, steps = 70, 5, 8, 2, 3
    prefix = Cache([P], Hkv, True, fp8, 50, valid=[0])
    prompts = [9, 33, 1, 20, 16]
    cache = Cache([n + steps for n in prompts], Hkv, True, fp8, 51, valid=[0] * B)
    pre, own = prefix.gpu(api, dev), cache.gpu(api, dev)
    table = torch.empty((256, 64), dtype=torch.float32, device=dev)
    api.dr_rope_table(table)
    err = torch.zeros(1, dtype=torch.int32, device=dev)

    def project(T, key):
        x = W.randn_bf16((T, Hq + 2 * Hkv, D), dev, 60, key)
        return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]

    def pull():
        prefix.k, prefix.v, cache.k, cache.v = pre.k.cpu(), pre.v.cpu(), own.k.cpu(), own.v.cpu()

    # the prefix: all of its tokens see all of it
    q, k, v = project(P, 1)
    qr, out = torch.empty((P, Hq, D), dtype=torch.bfloat16, device=dev), torch.empty((P, Hq, D), device=dev)
    api.dr_rope_append(pre, k, v, i32([0, P], dev), i32([0], dev), q=q, q_out=qr, table=table, err_flag=err)
    api.dr_prompt_attn(qr, pre, i32([0, P], dev), i32([P], dev), out, prefix_len=i32([P], dev), err_flag=err)
    pull()
    K, V = prefix.rows(0, P)
    ref, tol = attend(qr.cpu(), K, V, torch.zeros(P, dtype=torch.long), torch.full((P,), P), torch.arange(P), fp8=fp8)
    assert_close(out, ref, tol, "prefix")

    # the rows' prompts, rotated behind the prefix
    T, rs = sum(prompts), starts(prompts).to(dev)
    q, k, v = project(T, 2)
    qr, out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=dev), torch.empty((T, Hq, D), device=dev)
    api.dr_rope_append(own, k, v, rs, i32([0] * B, dev), q=q, q_out=qr, table=table, pos_offset=i32([P] * B, dev),
                       err_flag=err)
    api.dr_prompt_attn(qr, own, rs, i32(prompts, dev), out, err_flag=err)
    pull()
    at = 0
    for b, n in enumerate(prompts):
        K, V = cache.rows(b, n)
        ref, tol = attend(qr[at:at + n].cpu(), K, V, torch.zeros(n, dtype=torch.long), torch.arange(1, n + 1),
                          torch.arange(n), fp8=fp8)
        assert_close(out[at:at + n], ref, tol, f"prompt {b}")
        at += n

    # single tokens: append, then the prefix and the row's own keys; the second and third step are replays
    q, k, v = (x.contiguous() for x in project(B, 3))
    qr, out = torch.empty((B, Hq, D), dtype=torch.bfloat16, device=dev), torch.empty((B, Hq, D), device=dev)
    pos, seq, off, ones = i32(prompts, dev), i32(prompts, dev), i32([P] * B, dev), starts([1] * B).to(dev)
    ws = torch.empty(api.dr_shared_prefix_attn_workspace(B, Hq, Hkv, P), dtype=torch.uint8, device=dev)
    plen = i32([P], dev)

    def step():
        seq.add_(1)
        api.dr_rope_append(own, k, v, ones, pos, q=q, q_out=qr, table=table, pos_offset=off, err_flag=err)
        api.dr_shared_prefix_attn(qr, pre, plen, out, ws, cache=own, seq_len=seq, max_prefix_hint=P, err_flag=err)
        pos.add_(1)

    def compare(lens, what):
        pull()
        ref, tol = reference(prefix, P, cache, lens, qr.cpu(), 0.0, None, fp8, torch.float32)
        assert_close(out, ref, tol, what)

    step()
    compare([n + 1 for n in prompts], "step 1")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step()
    for i in (2, 3):
        for x, y in zip((q, k, v), project(B, 3 + i)):
            x.copy_(y)
        g.replay()
        compare([n + i for n in prompts], f"step {i}")
    assert int(err.item()) == 0
