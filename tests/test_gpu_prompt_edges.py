"""GPU checks of the prompt-side attention calls at corners that their documentation allows: large and odd groups of
heads, codes that are not numbers in masked places, blocks that are missing inside a row, small workspaces, biases on keys
behind and before the query, caches of different formats in one call, other streams, graphs that share a workspace.
Tolerances are those of prompt_reference."""
import pytest
import torch

from decode_attention_self_gb300 import workloads as W
from prompt_reference import PAGE, Cache, D, assert_close, attend, starts
from test_gpu_prompt_attn import check
from test_gpu_shared_prefix import check as check_shared
from test_gpu_shared_prefix import reference as shared_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api(cuda_device):
    from decode_attention_self_gb300 import api as _api

    return _api


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hq,Hkv", [(128, 1), (51, 3), (62, 2), (130, 13)])
def test_groups_of_heads(api, cuda_device, fp8, Hq, Hkv):
    check(api, cuda_device, [1, 1, 1], [3, 130, 400], Hq, Hkv, True, fp8, bias=True)
    check(api, cuda_device, [5, 0, 40], [129, 0, 300], Hq, Hkv, False, fp8, bias=True)
    check_shared(api, cuda_device, 300, [0, 7, 90], Hq, Hkv, True, fp8)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("causal", [False, True])
def test_bias_on_whole_tiles_before_and_behind_the_query(api, cuda_device, fp8, causal):
    check(api, cuda_device, [300], [1000], 4, 2, True, fp8, causal=causal, bias=True)
    if causal:
        check(api, cuda_device, [300, 2], [700, 900], 4, 2, False, fp8, prefix=[650, 900], bias=True)


@pytest.mark.parametrize("fp8", [False, True])
def test_cap_of_large_scores(api, cuda_device, fp8):
    check(api, cuda_device, [1, 140], [200, 300], 4, 2, True, fp8, softcap=5.0, q_gain=1e4)


@pytest.mark.parametrize("paged", [False, True])
def test_hidden_codes_that_are_not_numbers(api, cuda_device, paged):
    """e4m3 NaN codes behind a row's end, before every first key, and in a value that the last queries alone see."""
    dev, new, kv = cuda_device, [150, 1], [200, 90]
    cache = Cache([256, 256], 2, paged, True, 8, valid=kv)
    first = [40] * sum(new)
    for b in range(2):
        i0, i2 = cache.slots(b, 40)
        cache.k[i0, :, i2] = 0x7F
        cache.v[i0, :, i2] = 0xFF
    check(api, dev, new, kv, 4, 2, paged, True, first=first, cache=cache)
    i0, i2 = cache.slots(0, 200)
    cache.v[i0[190:], :, i2[190:], 5] = 0x7F
    q = W.randn_bf16((sum(new), 4, D), "cpu", 1, 7)
    out = torch.empty((sum(new), 4, D), device=dev)
    api.dr_prompt_attn(q.to(dev), cache.gpu(api, dev), starts(new).to(dev), i32(kv, dev), out, first_key=i32(first, dev))
    K, V = cache.rows(0, 200)
    pos = torch.arange(50, 200)
    ref, tol = attend(q[:150], K, torch.nan_to_num(V), torch.full((150,), 40), pos + 1, pos, fp8=True)
    sees, keep = pos >= 190, [d for d in range(D) if d != 5]
    assert_close(out[:150][~sees], ref[~sees], tol[~sees], "queries before")
    assert_close(out[:150][sees][..., keep], ref[sees][..., keep], tol[sees][..., keep], "other dimensions")
    assert torch.isnan(out[:150][sees][..., 5]).all()


@pytest.mark.parametrize("bad", [-1, 10 ** 6])
@pytest.mark.parametrize("fp8", [False, True])
def test_keys_of_a_missing_block_are_left_out(api, cuda_device, fp8, bad):
    dev, new, kv = cuda_device, [200, 1, 1], [300, 150, 70]
    cache = Cache(kv, 2, True, fp8, 3)
    q = W.randn_bf16((sum(new), 4, D), "cpu", 1, 7)
    rows = [cache.rows(b, L) for b, L in enumerate(kv)]
    cache.table[0, 3], cache.table[1, 5] = bad, bad
    out, err = torch.empty((sum(new), 4, D), device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    api.dr_prompt_attn(q.to(dev), cache.gpu(api, dev), starts(new).to(dev), i32(kv, dev), out, err_flag=err)
    assert int(err.item()) == api.DR_ERRF_BLOCK_ID
    at = 0
    for b, (n, L, gone) in enumerate(zip(new, kv, (3, 5, None))):
        K, V = rows[b]
        pos = torch.arange(L - n, L)
        hi = pos + 1
        if gone is not None:   # the keys without the block's, and how many of them each query sees
            keep = torch.tensor([j // PAGE != gone for j in range(L)])
            K, V = K[:, keep], V[:, keep]
            hi = torch.cat([torch.zeros(1, dtype=torch.long), keep.long().cumsum(0)])[hi]
        ref, tol = attend(q[at:at + n], K, V, torch.zeros(n, dtype=torch.long), hi, hi - 1, fp8=fp8)
        assert_close(out[at:at + n], ref, tol, f"row {b}")
        at += n


@pytest.mark.parametrize("fp8", [False, True])
def test_workspaces_of_any_size(api, cuda_device, fp8):
    dev, n, L, Hq, Hkv = cuda_device, 37, 5000, 6, 3
    cache = Cache([L], Hkv, True, fp8, 5)
    q = W.randn_bf16((n, Hq, D), "cpu", 2)
    K, V = cache.rows(0, L)
    pos = torch.arange(L - n, L)
    ref, tol = attend(q, K, V, torch.zeros(n, dtype=torch.long), pos + 1, pos, fp8=fp8)
    one, full = n * Hq * 66 * 4, api.dr_prompt_attn_workspace(n, 1, Hq, Hkv, L)
    assert full > 4 * one
    for size in (32, one, 2 * one - 1, 2 * one, 3 * one + 5, full):
        buf = torch.full((size + 64,), 0x7F, dtype=torch.uint8, device=dev)
        out = torch.empty((n, Hq, D), device=dev)
        api.dr_prompt_attn(q.to(dev), cache.gpu(api, dev), starts([n]).to(dev), i32([L], dev), out, workspace=buf[:size])
        assert_close(out, ref, tol, f"{size} bytes")
        assert (buf[size:] == 0x7F).all()


@pytest.mark.parametrize("prefix_fp8", [False, True])
def test_prefix_and_own_keys_of_different_formats(api, cuda_device, prefix_fp8):
    dev, P, own = cuda_device, 450, [0, 1, 33, 200]
    prefix, cache = Cache([P], 2, prefix_fp8, prefix_fp8, 4), Cache(own, 2, not prefix_fp8, not prefix_fp8, 5, valid=own)
    q = W.randn_bf16((len(own), 6, D), "cpu", 2)
    out = torch.empty((len(own), 6, D), device=dev)
    ws = torch.empty(api.dr_shared_prefix_attn_workspace(len(own), 6, 2, P), dtype=torch.uint8, device=dev)
    api.dr_shared_prefix_attn(q.to(dev), prefix.gpu(api, dev), i32([P], dev), out, ws, cache=cache.gpu(api, dev),
                              seq_len=i32(own, dev))
    ref, tol = shared_reference(prefix, P, cache, own, q, 0.0, None, False, torch.float32)
    assert_close(out, ref, tol, "mixed formats")


def test_graphs_on_another_stream_share_a_workspace(api, cuda_device):
    """Two graphs, captured on a side stream, that use the same workspace and are replayed in turn without a pause."""
    dev = cuda_device
    side, jobs = torch.cuda.Stream(), []
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=dev)
    for seed, (n, L) in enumerate(((40, 6000), (33, 9000))):
        cache = Cache([L], 2, True, False, 20 + seed).gpu(api, dev)
        q, out = W.randn_bf16((n, 4, D), dev, seed), torch.zeros((n, 4, D), device=dev)
        assert 0 < api.dr_prompt_attn_workspace(n, 1, 4, 2, L) <= ws.numel()
        args = (q, cache, starts([n]).to(dev), i32([L], dev))
        want = torch.zeros_like(out)
        api.dr_prompt_attn(*args, want, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            api.dr_prompt_attn(*args, out, workspace=ws)
        jobs.append((g, out, want, args))
    with torch.cuda.stream(side):
        for _ in range(50):
            for g, *_ in jobs:
                g.replay()
    torch.cuda.synchronize()
    for _, out, want, _ in jobs:
        assert torch.equal(out, want)
