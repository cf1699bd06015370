"""GPU checks of queries with one element far above the others, over keys that are zero there: the other elements decide.

Tolerance: prompt_reference's.  e4m3 caches hold q in f16, scaled so that its largest element is below 2^15: an element keeps
its 8 bits down to 2^-17 (f16's last step is 2^-24), 2^-31 of the largest; the smallest here, 2^-8 * 2^-20, keep them all.
"""
import pytest
import torch

from decode_attention_self_gb300 import workloads as W
from prompt_reference import Cache, D, assert_close, attend, starts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [1, 140])
@pytest.mark.parametrize("outlier", [2.0 ** 12, 2.0 ** 20])
def test_other_elements_decide(cuda_device, fp8, n, outlier):
    from decode_attention_self_gb300 import api

    dev, L, Hq, Hkv = cuda_device, 500, 4, 2
    cache = Cache([L], Hkv, True, fp8, 61)
    cache.k[..., 7] = 0
    q = W.randn_bf16((n, Hq, D), "cpu", 1, n)
    q = torch.where(q.abs() < 2.0 ** -8, torch.zeros_like(q), q)
    q[..., 7] = outlier
    out = torch.empty((n, Hq, D), device=dev)
    api.dr_prompt_attn(q.to(dev), cache.gpu(api, dev), starts([n]).to(dev), torch.tensor([L], dtype=torch.int32, device=dev),
                       out)
    K, V = cache.rows(0, L)
    pos = torch.arange(L - n, L)
    ref, tol = attend(q, K, V, torch.zeros(n, dtype=torch.long), pos + 1, pos, fp8=fp8)
    assert_close(out, ref, tol, "outlier")
