"""GPU checks of rows in which one key outweighs each of thousands of others whose sum still counts: its value is zero, theirs
are not.

Tolerance: prompt_reference's, which takes each weight as good to 2^-8 (bf16 caches) or 2^-11 (e4m3) of itself.  f16, which
holds the weights over e4m3 caches, does so down to 2^-14 and has steps of 2^-24 below; the kernels hold weights 2^7 times as
large as their ratio to the row's largest (or more), so a weight is off by at most half a step, 2^-25 * 2^-7 = 2^-32 of the
largest.  L keys: 2^-32 * L * max |v| more.  The fp32 sums take at most one rounding of 2^-23 for each 8 keys.
"""
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


def lopsided(L, fp8, gap, where, seed):
    """A cache of L keys of score 28 - gap (for a query of 8 in dimension 0) and one, `where`, of score 28 and value 0."""
    cache = Cache([L], 1, True, fp8, seed, k_scale=1.0)
    i0, i2 = cache.slots(0, L)
    k, v = torch.zeros(L, D), W.randn_bf16((L, D), "cpu", seed, 9).float().abs()
    k[:, 0] = 28.0 - gap
    k[where, 0], v[where] = 28.0, 0.0
    if fp8:
        cache.k[i0, 0, i2] = W.to_e4m3_codes(k.to(torch.bfloat16), cache.k_scale)
        cache.v[i0, 0, i2] = W.to_e4m3_codes(v.to(torch.bfloat16), cache.v_scale)
    else:
        cache.k[i0, 0, i2], cache.v[i0, 0, i2] = k.to(torch.bfloat16), v.to(torch.bfloat16)
    return cache


def query(n):
    q = torch.zeros(n, 2, D, dtype=torch.bfloat16)
    q[..., 0] = 8.0
    return q


def compare(out, q, K, V, hi, fp8, what):
    L = K.shape[1]
    ref, tol = attend(q, K, V, torch.zeros(len(hi), dtype=torch.long), hi, hi - 1, fp8=fp8)
    size, _ = attend(q, K, V.abs(), torch.zeros(len(hi), dtype=torch.long), hi, hi - 1, fp8=fp8)
    tol = tol + L / 8 * 2.0 ** -23 * size + (2.0 ** -32 * L * float(V.abs().max()) if fp8 else 0.0)
    assert_close(out, ref, tol, what)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("gap", [12, 17, 20, 24])
@pytest.mark.parametrize("n", [1, 130])
def test_prompt(api, cuda_device, fp8, gap, n):
    dev, L = cuda_device, 20000
    for where in (0, 9990, L - n):
        cache = lopsided(L, fp8, gap, where, 3)
        q, out = query(n), torch.empty((n, 2, D), device=dev)
        nb = api.dr_prompt_attn_workspace(n, 1, 2, 1, L)
        for ws in (None, torch.empty(nb, dtype=torch.uint8, device=dev) if nb else None):
            api.dr_prompt_attn(q.to(dev), cache.gpu(api, dev), starts([n]).to(dev), i32([L], dev), out, workspace=ws)
            compare(out, q, *cache.rows(0, L), torch.arange(L - n + 1, L + 1), fp8, f"key {where}")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("gap", [12, 17, 20, 24])
def test_shared_prefix(api, cuda_device, fp8, gap):
    """The heavy key in the prefix, and in the row's own keys."""
    dev, P, own = cuda_device, 12000, 8000
    for where in ((5000, None), (None, 77)):
        parts = [lopsided(n, fp8, gap, x or 0, 4 + i) for i, (n, x) in enumerate(zip((P, own), where))]
        for c, x in zip(parts, where):
            if x is None:   # no heavy key here
                i0, i2 = c.slots(0, 2)
                c.k[i0[0], 0, i2[0]] = c.k[i0[1], 0, i2[1]]
        q, out = query(1), torch.empty((1, 2, D), device=dev)
        ws = torch.empty(api.dr_shared_prefix_attn_workspace(1, 2, 1, P), dtype=torch.uint8, device=dev)
        api.dr_shared_prefix_attn(q.to(dev), parts[0].gpu(api, dev), i32([P], dev), out, ws, cache=parts[1].gpu(api, dev),
                                  seq_len=i32([own], dev))
        K, V = (torch.cat(x, 1) for x in zip(parts[0].rows(0, P), parts[1].rows(0, own)))
        compare(out, q, K, V, torch.tensor([P + own]), fp8, str(where))
