"""dr_linear where the lanes of a warp have different amounts to do: rows, column groups and steps of K that end inside a warp."""
import pytest
import torch

from layer_reference import assert_within, linear64

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def api(cuda_device):
    from decode_attention_self_gb300 import api as _api

    return _api


def randn(shape, seed, scale=1.0, dtype=BF16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def check(api, T, K, N, gated, residual, out):
    x, W = randn((T, K), T), randn((2 * N if gated else N, K), T + 1, K ** -0.5)
    b, r = randn((W.shape[0],), T + 2, 0.5), randn((T, N), T + 3, 1.0, out) if residual else None
    ref, tol = linear64(x, W, b, "silu" if gated else None, gated, r, out)
    first = None
    for _ in range(5):
        o = torch.full((T, N), float("nan"), dtype=out, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        api.dr_linear(x.cuda(), W.cuda(), o, bias=b.cuda(), act="silu" if gated else None, gated=gated,
                      residual=None if r is None else r.cuda(), err_flag=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        assert_within(o, ref, tol, f"T={T} K={K} N={N} gated={gated}")
        first = o if first is None else first
        assert torch.equal(o, first)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T,K,N", [
    (104, 4096, 64),    # 8 CTAs of a cluster share K: 13 rows of each, 52 or 104 pieces of four columns
    (104, 4096, 63),    # and element by element
    (33, 2048, 200), (50, 1536, 24), (121, 1000, 129),
    (45, 512, 96), (77, 256, 1000), (109, 64, 4096),   # whole K in a CTA
    (1, 40, 20), (9, 72, 50), (13, 1000, 129), (27, 104, 63),   # steps of K and rows of both operands that end inside a warp
])
def test_warps_that_are_not_full(api, T, K, N, gated, out):
    check(api, T, K, N, gated, T % 2 == 0, out)


@pytest.mark.parametrize("T,K,N,gated,out", [(2011, 136, 1000, False, BF16), (1501, 264, 1034, True, BF16), (3001, 520, 1017, False, F32),
                                             (5003, 200, 1032, False, BF16), (5003, 200, 1032, True, F32)])
def test_prompts_whose_last_tiles_are_not_full(api, T, K, N, gated, out):
    check(api, T, K, N, gated, True, out)
