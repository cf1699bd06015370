"""GPU checks of the tile kernel's bounded waits: a CTA whose keys never come gives up after about 2 s, flags it and ends
cleanly.  What it would have written stays as it was, or is NaN where key ranges are joined (never an earlier call's); every
other output is that of the undisturbed call, and later calls work."""
import pytest
import torch

from decode_attention_self_gb300 import workloads as W
from prompt_reference import Cache, D, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api(cuda_device):
    from decode_attention_self_gb300 import api as _api

    return _api


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("new,kv", [([40, 1, 90], [40, 300, 2000]),   # one key tile: nothing in flight
                                    ([200, 30], [900, 30])])          # more than the stages hold: copies in flight
def test_prompt(api, cuda_device, fp8, paged, new, kv):
    dev, Hq, Hkv, head = cuda_device, 4, 2, 1
    cache = Cache(kv, Hkv, paged, fp8, 11).gpu(api, dev)
    q = W.randn_bf16((sum(new), Hq, D), dev, 1)
    args = (q, cache, starts(new).to(dev), i32(kv, dev))
    want = api.dr_prompt_attn(*args, torch.empty((sum(new), Hq, D), device=dev))
    out, err = torch.full_like(want, 3.0), i32([0], dev)
    api.dr_prompt_attn_stall_test(head, *args, out, err_flag=err)
    assert int(err.item()) == api.DR_ERRF_TIMEOUT
    # the last 128 (token, query head) pairs of the first row's second key/value head: two query heads per token
    lost = torch.zeros((sum(new), Hq), dtype=torch.bool)
    first = ((new[0] * 2 - 1) // 128 * 128) // 2
    lost[first:new[0], 2:] = True
    lost = lost.to(dev)
    assert (out[lost] == 3.0).all() and torch.equal(out[~lost], want[~lost])
    err.zero_()
    assert torch.equal(api.dr_prompt_attn(*args, out, err_flag=err), want) and int(err.item()) == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_joined_key_ranges(api, cuda_device, fp8):
    """The workspace holds the states of an earlier call: none of them may pass for this one's."""
    dev, n, L, Hq, Hkv, head = cuda_device, 40, 9000, 4, 2, 0
    cache = Cache([L], Hkv, True, fp8, 12).gpu(api, dev)
    q = W.randn_bf16((n, Hq, D), dev, 1)
    ws = torch.empty(api.dr_prompt_attn_workspace(n, 1, Hq, Hkv, L), dtype=torch.uint8, device=dev)
    assert ws.numel() > 0
    args = (q, cache, starts([n]).to(dev), i32([L], dev))
    want = api.dr_prompt_attn(*args, torch.empty((n, Hq, D), device=dev), workspace=ws)
    out, err = torch.full_like(want, 3.0), i32([0], dev)
    api.dr_prompt_attn_stall_test(head, *args, out, workspace=ws, err_flag=err)
    assert int(err.item()) == api.DR_ERRF_TIMEOUT
    assert out[:, :2].isnan().all() and torch.equal(out[:, 2:], want[:, 2:])
    err.zero_()
    assert torch.equal(api.dr_prompt_attn(*args, out, workspace=ws, err_flag=err), want) and int(err.item()) == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("P", [60, 9000])
def test_shared_prefix(api, cuda_device, fp8, P):
    dev, own, Hq, Hkv, head = cuda_device, [5, 0, 300], 6, 2, 1
    prefix, cache = Cache([P], Hkv, True, fp8, 13).gpu(api, dev), Cache([5, 1, 300], Hkv, True, fp8, 14).gpu(api, dev)
    q = W.randn_bf16((3, Hq, D), dev, 1)
    ws = torch.empty(api.dr_shared_prefix_attn_workspace(3, Hq, Hkv, P), dtype=torch.uint8, device=dev)
    args, kw = (q, prefix, i32([P], dev)), dict(cache=cache, seq_len=i32(own, dev))
    want = api.dr_shared_prefix_attn(*args, torch.empty((3, Hq, D), device=dev), ws, **kw)
    out, err = torch.full_like(want, 3.0), i32([0], dev)
    api.dr_shared_prefix_attn_stall_test(head, *args, out, ws, err_flag=err, **kw)
    assert int(err.item()) == api.DR_ERRF_TIMEOUT
    assert out[:, 3:].isnan().all() and torch.equal(out[:, :3], want[:, :3])
    err.zero_()
    assert torch.equal(api.dr_shared_prefix_attn(*args, out, ws, err_flag=err, **kw), want) and int(err.item()) == 0


def test_hook_refusals(api, cuda_device):
    dev = cuda_device
    cache = Cache([64], 2, True, False, 4).gpu(api, dev)
    q = W.randn_bf16((2, 4, D), dev, 3)
    args = (q, cache, starts([2]).to(dev), i32([9], dev), torch.empty((2, 4, D), device=dev))
    for head in (-1, 2):
        with pytest.raises(api.DrError):
            api.dr_prompt_attn_stall_test(head, *args)
        with pytest.raises(api.DrError):
            api.dr_shared_prefix_attn_stall_test(head, q, cache, i32([9], dev), args[-1],
                                                 torch.empty(1 << 16, dtype=torch.uint8, device=dev))
    with pytest.raises(api.DrError):                     # single tokens: no tile kernel
        api.dr_prompt_attn_stall_test(0, q[:1], cache, starts([1]).to(dev), i32([9], dev), args[-1][:1])
