"""GPU checks of the score cap over the whole documented range of caps, 1e-6 .. 1e30.

Tolerance, derived from the kernels' arithmetic before the first run; nothing in it grows with the cap.  The raw score is an
fp32 sum of exact products, off by at most 72 * 2^-23 * A (A the largest sum_d |q_d k_d| * scale of the row, prompt_reference);
a cap has a slope of at most 1, so that is passed on unchanged.  cap * tanh(s / cap): up to s / cap = 1/2 the score times a
polynomial in (s / cap)^2 whose value lies within 10% of 1 (2^-26 from tanh(u) / u; four fused steps, three products and two
quotients' roundings of 2^-24: below 2^-21); beyond, cap - 2 cap / (e^(2 s / cap) + 1), off by at most 2^-22 of the cap (the
exponential's and the reciprocal's 2^-22, each times a factor below 1/2) where the value is at least 0.46 of it.  Both stay
below 2^-20 of the score.  With the exponential's 2^-20,
    |got - ref| <= (eps_w + 2 * ((72 * 2^-23 + 2^-20) * A + 2^-20)) * sum_j p_j |v_j| + 2^-23 |ref|
eps_w: 2^-8 for bf16 caches, 2^-11 for e4m3 (prompt_reference).
"""
import pytest
import torch

from decode_attention_self_gb300 import workloads as W
from prompt_reference import Cache, D, assert_close, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api(cuda_device):
    from decode_attention_self_gb300 import api as _api

    return _api


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def capped(q, K, V, hi, cap, fp8, scale=D ** -0.5):
    """q [n, Hq, D], K, V [Hkv, L, D] float64, keys [0, hi[i]) -> (ref, tolerance)."""
    q, g = q.double(), q.shape[1] // K.shape[0]
    k, v = K.repeat_interleave(g, 0), V.repeat_interleave(g, 0)
    hidden = (torch.arange(K.shape[1])[None] >= hi[:, None])[:, None]                 # [n, 1, L]
    s = torch.einsum("nhd,hld->nhl", q, k) * scale
    mag = (torch.einsum("nhd,hld->nhl", q.abs(), k.abs()) * scale).masked_fill(hidden, 0.0).amax(-1)
    p = torch.softmax((cap * torch.tanh(s / cap)).masked_fill(hidden, -float("inf")), -1)
    ref, size = torch.einsum("nhl,hld->nhd", p, v), torch.einsum("nhl,hld->nhd", p, v.abs())
    rel = (2.0 ** -11 if fp8 else 2.0 ** -8) + 2 * ((72 * 2.0 ** -23 + 2.0 ** -20) * mag + 2.0 ** -20)
    return ref, rel[..., None] * size + 2.0 ** -23 * ref.abs() + 1e-30


CAPS = [1e-6, 0.02, 1.0, 30.0, 1e3, 1e4, 1e5, 1e6, 1e8, 1e12, 1e30]


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [1, 140])
def test_any_cap(api, cuda_device, cap, fp8, n):
    dev, L, Hq, Hkv = cuda_device, 1024, 4, 2
    cache = Cache([L], Hkv, True, fp8, 31)
    for gain in (1.0, 6.0):
        q = (W.randn_bf16((n, Hq, D), "cpu", 1, n).float() * gain).to(torch.bfloat16)
        out = torch.empty((n, Hq, D), device=dev)
        api.dr_prompt_attn(q.to(dev), cache.gpu(api, dev), starts([n]).to(dev), i32([L], dev), out, softcap=cap)
        ref, tol = capped(q, *cache.rows(0, L), torch.arange(L - n + 1, L + 1), cap, fp8)
        assert_close(out, ref, tol, f"gain {gain}")


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("fp8", [False, True])
def test_any_cap_behind_a_shared_prefix(api, cuda_device, cap, fp8):
    dev, P, own, Hq, Hkv = cuda_device, 700, [90, 0, 300], 4, 2
    prefix, cache = Cache([P], Hkv, True, fp8, 32), Cache([max(x, 1) for x in own], Hkv, True, fp8, 33)
    q = (W.randn_bf16((3, Hq, D), "cpu", 1).float() * 3).to(torch.bfloat16)
    out = torch.empty((3, Hq, D), device=dev)
    ws = torch.empty(api.dr_shared_prefix_attn_workspace(3, Hq, Hkv, P), dtype=torch.uint8, device=dev)
    api.dr_shared_prefix_attn(q.to(dev), prefix.gpu(api, dev), i32([P], dev), out, ws, cache=cache.gpu(api, dev),
                              seq_len=i32(own, dev), softcap=cap)
    for b, m in enumerate(own):
        K, V = (torch.cat(x, 1) for x in zip(prefix.rows(0, P), cache.rows(b, m)))
        ref, tol = capped(q[b:b + 1], K, V, torch.tensor([P + m]), cap, fp8)
        assert_close(out[b:b + 1], ref, tol, f"row {b}")


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_small_scores_beside_large_ones(api, cuda_device, fp8, bias):
    """Every other query of a tile reaches the cap; the others stay far below it.  (A bias of slope 0 takes the other way
    through the kernel.)"""
    dev, L, n, cap = cuda_device, 500, 200, 1e6
    cache = Cache([L], 1, True, fp8, 34)
    q = W.randn_bf16((n, 2, D), "cpu", 5)
    q[::2] *= 2.0 ** 24
    out = torch.empty((n, 2, D), device=dev)
    api.dr_prompt_attn(q.to(dev), cache.gpu(api, dev), starts([n]).to(dev), i32([L], dev), out, softcap=cap,
                       slopes=torch.zeros(2, device=dev) if bias else None)
    ref, tol = capped(q, *cache.rows(0, L), torch.arange(L - n + 1, L + 1), cap, fp8)
    assert_close(out[1::2], ref[1::2], tol[1::2], "small")
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [1, 130])
def test_infinite_and_nan_scores_under_a_cap(api, cuda_device, fp8, n):
    """An infinite score is the cap (or minus it), a score that is not a number stays one."""
    dev, L, cap = cuda_device, 260, 5.0
    cache = Cache([L], 1, True, fp8, 35)
    q = W.randn_bf16((n, 2, D), "cpu", 5)
    q[0, 0, 0] = float("inf")
    q[n - 1, 1, 2] = float("nan")
    i0, i2 = cache.slots(0, L)
    if fp8:
        zero = (cache.k[i0, :, i2, 0] & 0x7F) == 0          # inf * 0 is not a number
        assert not zero.any()
    out = torch.empty((n, 2, D), device=dev)
    api.dr_prompt_attn(q.to(dev), cache.gpu(api, dev), starts([n]).to(dev), i32([L], dev), out, softcap=cap)
    K, V = cache.rows(0, L)
    hi = torch.arange(L - n + 1, L + 1)
    ref, tol = capped(q, K, V, hi, cap, fp8)
    # A is infinite for the infinite query; its scores are +-cap exactly: weights' rounding and the exponentials' remain
    p = torch.softmax((cap * torch.sign(K[0, :hi[0], 0])), 0)
    size = p @ V[0, :hi[0]].abs()
    tol[0, 0] = ((2.0 ** -11 if fp8 else 2.0 ** -8) + 2 * (2.0 ** -20 * (cap + 1))) * size + 1e-30
    assert torch.isnan(out[n - 1, 1]).all() and torch.isfinite(out[0, 0]).all()
    keep = torch.ones(n, 2, dtype=torch.bool)
    keep[n - 1, 1] = False
    assert_close(out[keep.to(dev)], ref[keep], tol[keep], "others")
