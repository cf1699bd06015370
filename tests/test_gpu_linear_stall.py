"""dr_linear's bounded waits where a pair of CTAs has several tiles, two sets of warps take them in turn, and residuals are on their way."""
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


def tile_place(i, T, N, cols):
    """First token and column of tile i of 256 tokens by `cols` columns: groups of 8 token tiles take all column tiles in turn."""
    token_tiles, col_tiles = -(-T // 256), -(-N // cols)
    g = i // (8 * col_tiles)
    r, n = i - g * 8 * col_tiles, min(8, token_tiles - g * 8)
    return (g * 8 + r % n) * 256, r // n * cols


@pytest.mark.parametrize("out,gated,residual,N", [(BF16, False, True, 2048), (BF16, False, False, 2048), (BF16, True, True, 1024),
                                                  (F32, False, True, 2048), (F32, True, True, 1024), (BF16, False, True, 2041)])
@pytest.mark.parametrize("before", [0, 1])
def test_wait_that_runs_out_among_several_tiles(api, out, gated, residual, N, before):
    T, K = 6000, 576
    pairs, cols = torch.cuda.get_device_properties(0).multi_processor_count // 2, 128 if gated else 256
    tiles = -(-T // 256) * -(-N // cols)
    assert tiles > 2 * pairs + 2
    x, W = randn((T, K), 1), randn((2 * N if gated else N, K), 2, K ** -0.5)
    b, r = randn((W.shape[0],), 3, 0.5), randn((T, N), 4, 1.0, out) if residual else None
    ref, tol = linear64(x, W, b, "silu" if gated else "gelu", gated, r, out)
    cuda = [None if t is None else t.cuda() for t in (x, W, b, r)]
    args = dict(bias=cuda[2], act="silu" if gated else "gelu", gated=gated, residual=cuda[3])
    o = torch.full((T, N), float("nan"), dtype=out, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    stalled = 1 + before * pairs   # the first or the second tile of the pair that starts with tile 1
    api.dr_linear_stall_test(stalled, cuda[0], cuda[1], o, err_flag=err, **args)
    torch.cuda.synchronize()
    assert int(err.item()) & api.DR_ERRF_TIMEOUT
    got = o.cpu()
    for i in range(stalled, tiles, pairs):   # the tile, and those that the pair would have taken after it
        t0, n0 = tile_place(i, T, N, cols)
        assert got[t0:t0 + 256, n0:n0 + cols].isnan().all(), i
        got[t0:t0 + 256, n0:n0 + cols] = ref[t0:t0 + 256, n0:n0 + cols].to(out)
    assert_within(got, ref, tol, "tiles that ran")
    for _ in range(2):
        err.zero_()
        o.fill_(float("nan"))
        api.dr_linear(cuda[0], cuda[1], o, err_flag=err, **args)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        assert_within(o, ref, tol, "the call after")
