"""An infinite or NaN weight in a gated product, by the formula: which outputs of its column are infinite, which NaN, which finite."""
import pytest
import torch

from layer_reference import act64, assert_within, linear64

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def api(cuda_device):
    from decode_attention_self_gb300 import api as _api

    return _api


def randn(shape, seed, scale=1.0, dtype=BF16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


@pytest.mark.parametrize("T", [1, 9, 18, 65, 260, 1900, 7000])
@pytest.mark.parametrize("act", [None, "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("half", [0, 1])
@pytest.mark.parametrize("out", [BF16, F32])
def test_infinite_weight_of_a_gated_product(api, T, act, half, out):
    # Column n's sum is x[t][k] * inf and finite terms: +-inf by the sign of x[t][k].  In the first half it is activated (inf, or the
    # limit at -inf) and multiplied by a finite factor, in the second it multiplies an activated one, which relu makes 0 at times: NaN.
    K, N, n, k = 200, 530, 77, 5
    x, W = randn((T, K), 1), randn((2 * N, K), 2, K ** -0.5)
    b, r = randn((2 * N,), 3, 0.5), randn((T, N), 4, 1.0, out)
    ref, tol = linear64(x, W, b, act, True, r, out)
    W[half * N + n, k] = float("inf")
    o = torch.empty((T, N), dtype=out, device="cuda")
    api.dr_linear(x.cuda(), W.cuda(), o, bias=b.cuda(), act=act, gated=True, residual=r.cuda())
    o = o.cpu()
    w_other = W[(1 - half) * N + n].double()
    other = x.double() @ w_other + b[(1 - half) * N + n].double()   # the finite factor's sum
    sure = other.abs() > K * 2.0 ** -23 * (x.double().abs() @ w_other.abs() + 1)   # of its sign, in fp32
    sign = x[:, k].double().sign()
    assert (sign != 0).all() and sure.sum() >= T - T // 500
    inf = sign * float("inf")
    if half == 0:
        limit = {None: -float("inf")}.get(act, 0.0)
        a = torch.where(sign > 0, inf, torch.full_like(inf, limit))
        want = a * other
    else:
        want = act64(other, act) * inf
    want = r[:, n].double() + want
    got = o[:, n].double()[sure]
    want = want[sure]
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got[want.isinf()], want[want.isinf()])
    finite = want.isfinite()
    assert torch.equal(got[finite], want[finite])   # the residual alone
    keep = torch.ones(N, dtype=torch.bool)
    keep[n] = False
    assert_within(o[:, keep], ref[:, keep], tol[:, keep], "the other columns")


@pytest.mark.parametrize("T", [9, 65, 1900, 7000])
@pytest.mark.parametrize("half", [0, 1])
def test_nan_weight_of_a_gated_product(api, T, half):
    K, N, n = 200, 530, 500
    x, W = randn((T, K), 1), randn((2 * N, K), 2, K ** -0.5)
    ref, tol = linear64(x, W, None, "silu", True, None, BF16)
    W[half * N + n, 5] = float("nan")
    o = torch.empty((T, N), dtype=BF16, device="cuda")
    api.dr_linear(x.cuda(), W.cuda(), o, act="silu", gated=True)
    o = o.cpu()
    assert o[:, n].isnan().all()
    keep = torch.ones(N, dtype=torch.bool)
    keep[n] = False
    assert_within(o[:, keep], ref[:, keep], tol[:, keep], "the other columns")
