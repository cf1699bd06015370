"""GPU checks that single tokens over a bf16 cache keep their softmax weights to 16 bits for the product with V.

Tolerance: a weight is the sum of its upper 8 bits (a bf16, cut off) and the rest (below 2^-7 of it) rounded to bf16, off by
half a step of that: 2^-7 * 2^-9 = 2^-16 of the weight.  Both products are exact in fp32; the sums take a rounding of 2^-24
(the tensor cores may cut off: 2^-23) of sum p |v| for each 8 products (one instruction's) and join: at most L / 8 + 64 of
them.  Scores and exponentials as in prompt_reference.
"""
import pytest
import torch

from decode_attention_self_gb300 import workloads as W
from prompt_reference import Cache, D, assert_close, attend, starts
from test_gpu_shared_prefix import reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api(cuda_device):
    from decode_attention_self_gb300 import api as _api

    return _api


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def tighter(tol, weight, L):
    """prompt_reference's tolerance with 2^-8 for the weights replaced; weight: sum p |v|."""
    return tol - (2.0 ** -8 - 2.0 ** -16 - (L / 8 + 64) * 2.0 ** -23) * weight


@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (16, 2), (12, 1), (32, 2), (7, 1)])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("softcap", [0.0, 15.0])
def test_single_tokens(api, cuda_device, Hq, Hkv, paged, softcap):
    dev, kv = cuda_device, [1, 17, 200, 1111, 3000]
    cache = Cache(kv, Hkv, paged, False, 41)
    q = W.randn_bf16((len(kv), Hq, D), "cpu", 1, 7)
    out = torch.empty((len(kv), Hq, D), device=dev)
    api.dr_prompt_attn(q.to(dev), cache.gpu(api, dev), starts([1] * len(kv)).to(dev), i32(kv, dev), out, softcap=softcap)
    for b, L in enumerate(kv):
        K, V = cache.rows(b, L)
        at = (torch.zeros(1, dtype=torch.long), torch.tensor([L]), torch.tensor([L - 1]))
        ref, tol = attend(q[b:b + 1], K, V, *at, softcap=softcap)
        size, _ = attend(q[b:b + 1], K, V.abs(), *at, softcap=softcap)
        assert_close(out[b:b + 1], ref, tighter(tol, size, L), f"row {b}")


def test_own_keys_behind_an_empty_prefix(api, cuda_device):
    dev, own, Hq, Hkv = cuda_device, [5, 300, 2000], 8, 2
    prefix, cache = Cache([16], Hkv, True, False, 42), Cache(own, Hkv, True, False, 43)
    q = W.randn_bf16((3, Hq, D), "cpu", 1, 7)
    out = torch.empty((3, Hq, D), device=dev)
    ws = torch.empty(api.dr_shared_prefix_attn_workspace(3, Hq, Hkv, 16), dtype=torch.uint8, device=dev)
    api.dr_shared_prefix_attn(q.to(dev), prefix.gpu(api, dev), i32([0], dev), out, ws, cache=cache.gpu(api, dev),
                              seq_len=i32(own, dev))
    ref, tol = reference(prefix, 0, cache, own, q, 0.0, None, False, torch.float32)
    cache.v = cache.v.abs()
    size, _ = reference(prefix, 0, cache, own, q, 0.0, None, False, torch.float32)
    assert_close(out, ref, tighter(tol, size, 2000), "own")
