"""GPU checks of dr_prompt_attn against 64-bit attention: ragged rows, grouped heads, masks, caps, bias, both caches."""
import numpy as np
import pytest
import torch

from decode_attention_self_gb300 import workloads as W
from prompt_reference import Cache, D, assert_close, attend, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api(cuda_device):
    from decode_attention_self_gb300 import api as _api

    return _api


def check(api, dev, new, kv_len, Hq, Hkv, paged=True, fp8=False, causal=True, softcap=0.0, bias=False, prefix=None,
          first=None, out_dtype=torch.float32, workspace=True, stride_pad=0, seed=1, caps=None, hint=0, scale=0.0,
          q_gain=1.0, spare=2, cache=None):
    B, used = len(new), sum(new)
    T = used + spare
    cache = cache or Cache(caps or kv_len, Hkv, paged, fp8, seed, valid=kv_len)
    q = (W.randn_bf16((T, Hq + stride_pad, D), "cpu", seed, 7).float() * q_gain).to(torch.bfloat16)
    gq = q.to(dev)[:, :Hq]
    out = torch.full((T, Hq, D), 3.0, dtype=out_dtype, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    slopes = torch.tensor([2.0 ** (-(i % 7) - 1) for i in range(Hq)]) if bias else None
    first_t = None
    if first is not None:
        first_t = torch.tensor(list(first) + [0] * (T - len(first)), dtype=torch.int32)
    gpu = lambda t: None if t is None else t.to(dev)
    ws = None
    if workspace:
        nb = api.dr_prompt_attn_workspace(T, B, Hq, Hkv, hint or max(max(kv_len), 1))
        ws = torch.full((nb,), 255, dtype=torch.uint8, device=dev) if nb else None
    prefix_t = None if prefix is None else torch.tensor(prefix, dtype=torch.int32)
    api.dr_prompt_attn(gq, cache.gpu(api, dev), starts(new).to(dev), torch.tensor(kv_len, dtype=torch.int32, device=dev),
                       out, causal=causal, softcap=softcap, slopes=gpu(slopes), prefix_len=gpu(prefix_t),
                       first_key=gpu(first_t), max_len_hint=hint, scale=scale, workspace=ws, err_flag=err)
    assert int(err.item()) == 0
    at = 0
    for b, (n, L) in enumerate(zip(new, kv_len)):
        if n == 0:
            continue
        pos = torch.arange(L - n, L)
        lo = torch.zeros(n, dtype=torch.long) if first is None else torch.tensor(first[at:at + n]).clamp_min(0)
        hi = pos + 1 if causal else torch.full((n,), L)
        if prefix is not None:
            hi = torch.maximum(hi, torch.tensor(prefix[b])).clamp_max(L)
        K, V = cache.rows(b, L)
        ref, tol = attend(q[at:at + n, :Hq], K, V, lo, hi, pos, scale or D ** -0.5, softcap, slopes, fp8, out_dtype)
        assert_close(out[at:at + n], ref, tol, f"row {b}")
        at += n
    assert (out[used:] == 3.0).all()          # tokens behind the last row
    return out


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (16, 16), (8, 2), (14, 2), (12, 1), (33, 3)])
def test_single_tokens(api, cuda_device, fp8, paged, Hq, Hkv):
    check(api, cuda_device, [1] * 6, [1, 15, 16, 17, 200, 1111], Hq, Hkv, paged, fp8, seed=Hq)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new,kv", [([1], [1]), ([2], [2]), ([64], [64]), ([127, 129], [127, 300]),
                                    ([128, 1, 0, 300], [128, 1000, 0, 301]), ([257], [1025]), ([16, 17], [4000, 17])])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (8, 2), (7, 1)])
def test_causal_prompts(api, cuda_device, fp8, new, kv, Hq, Hkv):
    check(api, cuda_device, new, kv, Hq, Hkv, True, fp8, seed=sum(kv))


@pytest.mark.parametrize("paged", [False, True])
def test_all_keys_visible(api, cuda_device, paged):
    check(api, cuda_device, [5, 130, 1], [64, 130, 77], 4, 4, paged, causal=False)


@pytest.mark.parametrize("fp8", [False, True])
def test_score_cap_and_bias(api, cuda_device, fp8):
    for n in ([1, 1], [140, 3]):
        check(api, cuda_device, n, [300, 500], 8, 2, True, fp8, softcap=2.0, q_gain=4.0)
        check(api, cuda_device, n, [300, 500], 8, 2, True, fp8, bias=True)
        check(api, cuda_device, n, [300, 500], 8, 2, False, fp8, softcap=20.0, bias=True, q_gain=8.0)


@pytest.mark.parametrize("fp8", [False, True])
def test_prefix_mask(api, cuda_device, fp8):
    check(api, cuda_device, [100, 1, 20, 300], [100, 40, 400, 700], 4, 2, True, fp8, prefix=[60, 40, 0, 5000],
          bias=True)


@pytest.mark.parametrize("fp8", [False, True])
def test_document_mask_with_empty_rows_of_the_mask(api, cuda_device, fp8):
    new, kv = [150, 1, 1, 260], [200, 90, 33, 260]
    rng = np.random.default_rng(3)
    first = []
    for n, L in zip(new, kv):
        for i in range(n):
            p = L - n + i
            first.append(int(rng.choice([0, max(0, p - 3), p, p + 1, 10 ** 9, -7, (p // 48) * 48])))
    out = check(api, cuda_device, new, kv, 4, 2, True, fp8, first=first)
    empty = [i for i, (f, p) in enumerate(zip(first, np.concatenate([np.arange(L - n, L) for n, L in zip(new, kv)])))
             if f > p]
    assert empty and (out[empty] == 0).all()


def test_bf16_output_strided_queries_and_scale(api, cuda_device):
    check(api, cuda_device, [70, 1], [99, 512], 6, 3, out_dtype=torch.bfloat16, stride_pad=5, scale=0.3)
    check(api, cuda_device, [1, 1], [99, 512], 6, 3, out_dtype=torch.bfloat16, stride_pad=5, scale=0.05)


@pytest.mark.parametrize("gain", [1e-30, 1e3, 1e20])
@pytest.mark.parametrize("new", [[1, 1], [140, 9]])
def test_query_magnitudes_in_an_e4m3_cache(api, cuda_device, gain, new):
    # scores of any size through a scale that undoes the gain
    check(api, cuda_device, new, [150, 260], 4, 2, True, True, q_gain=gain, scale=0.125 / gain)


@pytest.mark.parametrize("workspace", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_few_queries_over_many_keys(api, cuda_device, workspace, fp8):
    check(api, cuda_device, [40, 1], [9001, 5000], 4, 1, True, fp8, workspace=workspace)
    check(api, cuda_device, [1], [20000], 2, 1, False, fp8, workspace=workspace)


def test_longer_capacity_and_hints(api, cuda_device):
    for hint in (0, 1, 333, 10 ** 9):
        check(api, cuda_device, [33, 1], [333, 50], 4, 4, True, caps=[2000, 1000], hint=hint)


def test_many_rows_mixed_lengths(api, cuda_device):
    rng = np.random.default_rng(9)
    new = [int(x) for x in rng.choice([0, 1, 1, 2, 5, 31, 130], size=70)]
    kv = [n + int(rng.integers(0, 200)) if n else 0 for n in new]
    check(api, cuda_device, new, kv, 4, 2, True)
    check(api, cuda_device, new, kv, 4, 2, False, True, bias=True)


def test_results_do_not_depend_on_the_batch(api, cuda_device):
    dev = cuda_device
    cache = Cache([700], 2, True, False, 5, valid=[700])
    q = W.randn_bf16((200, 4, D), dev, 3)
    kl = torch.tensor([700], dtype=torch.int32, device=dev)
    outs = []
    for _ in range(3):
        out = torch.empty((200, 4, D), dtype=torch.float32, device=dev)
        api.dr_prompt_attn(q, cache.gpu(api, dev), starts([200]).to(dev), kl, out)
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("new", [[1, 1], [150, 40]])
@pytest.mark.parametrize("fill", [float("nan"), float("inf")])
def test_hidden_values_that_are_not_finite(api, cuda_device, new, fill):
    """Values past kv_len, before every query's first key, and values that only later queries see."""
    dev = cuda_device
    kv = [200, 90]
    cache = Cache([256, 256], 2, True, False, 8, valid=kv, fill=fill)
    first = [40] * sum(new)
    for b in range(2):
        i0, i2 = cache.slots(b, 40)
        cache.k[i0, :, i2] = fill
        cache.v[i0, :, i2] = fill
    check(api, dev, new, kv, 4, 2, True, first=first, cache=cache)
    if new[0] > 1:
        # a value that the last queries alone see
        i0, i2 = cache.slots(0, 200)
        cache.v[i0[190:], :, i2[190:], 5] = fill
        q = W.randn_bf16((sum(new), 4, D), "cpu", 1, 7)
        out = torch.empty((sum(new), 4, D), dtype=torch.float32, device=dev)
        api.dr_prompt_attn(q.to(dev), cache.gpu(api, dev), starts(new).to(dev),
                           torch.tensor(kv, dtype=torch.int32, device=dev), out,
                           first_key=torch.tensor(first, dtype=torch.int32, device=dev))
        K, V = cache.rows(0, 200)
        pos = torch.arange(50, 200)
        Vc = torch.where(torch.isfinite(V), V, 0.0)
        ref, tol = attend(q[:150], K, Vc, torch.full((150,), 40), pos + 1, pos)
        sees = pos >= 190
        assert_close(out[:150][~sees], ref[~sees], tol[~sees], "queries before")
        keep = [d for d in range(D) if d != 5]
        assert_close(out[:150][sees][..., keep], ref[sees][..., keep], tol[sees][..., keep], "other dimensions")
        assert not torch.isfinite(out[:150][sees][..., 5]).any()


def test_device_side_errors_are_flagged(api, cuda_device):
    dev = cuda_device

    def run(new, kv, rs=None, table=None, T=None):
        cache = Cache([64, 64], 2, True, False, 4)
        if table is not None:
            for b, j, x in table:
                cache.table[b, j] = x
        T = T or sum(new)
        q = W.randn_bf16((T, 2, D), dev, 3)
        out = torch.full((T, 2, D), 3.0, dtype=torch.float32, device=dev)
        err = torch.zeros(1, dtype=torch.int32, device=dev)
        api.dr_prompt_attn(q, cache.gpu(api, dev), (starts(new) if rs is None else torch.tensor(rs, dtype=torch.int32)).to(dev),
                           torch.tensor(kv, dtype=torch.int32, device=dev), out, err_flag=err)
        return int(err.item()), out, q, cache

    for new in ([1, 1], [20, 20]):
        assert run(new, [65, 30])[0] == api.DR_ERRF_SEQ_LEN
        assert run(new, [-1, 30])[0] == api.DR_ERRF_SEQ_LEN
        flag, out, _, _ = run(new, [0, 30])
        assert flag == api.DR_ERRF_SEQ_LEN and (out[:new[0]] == 0).all()
        # an unmapped block: its keys are skipped
        flag, out, q, cache = run(new, [64, 30], table=[(0, 1, -1), (0, 2, 10 ** 6)])
        assert flag == api.DR_ERRF_BLOCK_ID
        cache.table[0, 1:3] = 0
        K, V = cache.rows(0, 64)
        keep = torch.tensor([j for j in range(64) if j < 16 or j >= 48])
        n = new[0]
        pos = torch.arange(64 - n, 64)
        ref, tol = attend(q[:n].cpu(), K[:, keep], V[:, keep], torch.zeros(n, dtype=torch.long),
                          (keep[None] <= pos[:, None]).sum(1), pos)
        assert_close(out[:n], ref, tol, "skipped blocks")
    assert run([20, 20], [30, 30], rs=[0, 20, 500])[0] == api.DR_ERRF_ROW_START
    assert run([20, 20], [30, 30], rs=[-4, 20, 40])[0] == api.DR_ERRF_ROW_START


def test_captured_and_replayed(api, cuda_device):
    dev = cuda_device
    cache = Cache([600, 300], 2, True, False, 6, valid=[600, 300])
    kv = cache.gpu(api, dev)
    for new in ([1, 1], [200, 40]):
        q = W.randn_bf16((sum(new), 4, D), dev, 1)
        rs, kl = starts(new).to(dev), torch.tensor([600, 300], dtype=torch.int32, device=dev)
        nb = api.dr_prompt_attn_workspace(sum(new), 2, 4, 2, 600)
        ws = torch.empty(nb, dtype=torch.uint8, device=dev) if nb else None
        out, ref = torch.zeros(sum(new), 4, D, device=dev), torch.zeros(sum(new), 4, D, device=dev)
        api.dr_prompt_attn(q, kv, rs, kl, ref, max_len_hint=600, workspace=ws)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            api.dr_prompt_attn(q, kv, rs, kl, out, max_len_hint=600, workspace=ws)
        for i in range(3):
            q.copy_(W.randn_bf16((sum(new), 4, D), dev, 10 + i))
            g.replay()
            api.dr_prompt_attn(q, kv, rs, kl, ref, max_len_hint=600, workspace=ws)
            assert torch.equal(out, ref)


def test_two_streams_at_once(api, cuda_device):
    dev = cuda_device
    jobs = []
    for i, new in enumerate(([300, 5], [1, 1])):
        cache = Cache([800, 600], 2, True, bool(i), 20 + i, valid=[800, 600])
        q = W.randn_bf16((sum(new), 4, D), dev, 30 + i)
        nb = api.dr_prompt_attn_workspace(sum(new), 2, 4, 2, 800)
        jobs.append((q, cache.gpu(api, dev), starts(new).to(dev), torch.tensor([800, 600], dtype=torch.int32, device=dev),
                     torch.empty(nb, dtype=torch.uint8, device=dev) if nb else None))
    want = [api.dr_prompt_attn(q, c, rs, kl, torch.empty(q.shape, device=dev), workspace=ws, max_len_hint=800)
            for q, c, rs, kl, ws in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [[torch.empty(j[0].shape, device=dev) for _ in range(20)] for j in jobs]
    torch.cuda.synchronize()
    for i in range(20):
        for (q, c, rs, kl, ws), st, o in zip(jobs, streams, got):
            api.dr_prompt_attn(q, c, rs, kl, o[i], workspace=ws, max_len_hint=800, stream=st)
    torch.cuda.synchronize()
    for w, outs in zip(want, got):
        assert all(torch.equal(w, o) for o in outs)


def test_binding_refusals(api, cuda_device):
    dev = cuda_device
    cache = Cache([64], 2, True, False, 4)
    kv = cache.gpu(api, dev)
    q = W.randn_bf16((2, 4, D), dev, 3)
    rs, kl, out = starts([2]).to(dev), torch.tensor([9], dtype=torch.int32, device=dev), torch.empty_like(q)
    for bad in (dict(q=q.cpu()), dict(q=q.float()), dict(out=out.half()), dict(out=out[:1]), dict(row_start=rs[:1]),
                dict(kv_len=kl.float()), dict(slopes=torch.ones(3, device=dev)),
                dict(first_key=torch.zeros(1, dtype=torch.int32, device=dev)),
                dict(workspace=torch.zeros(16, device=dev))):
        args = dict(q=q, cache=kv, row_start=rs, kv_len=kl, out=out)
        args.update(bad)
        with pytest.raises(ValueError):
            api.dr_prompt_attn(**args)
    with pytest.raises(api.DrError):
        api.dr_prompt_attn(q[:, :3], kv, rs, kl, out[:, :3].contiguous())   # 3 query heads on 2
