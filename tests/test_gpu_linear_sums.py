"""dr_linear's sums, measured: errors of whole outputs in norm, and sums that are exact and so must come out bit for bit.

The elementwise bounds of layer_reference.py cover any order of any sum and widen with K; these do not.

Bound of an fp32 output's error in norm, relative to the products' norm:
  chains     the tensor cores cut sums off: short by 0.9e-9 (K = 256) to 1.03e-9 (K = 2048) of their value per term, measured; fp32
             outputs promise chains of at most 512 terms: 1.1e-9 min(K, 512)
  adding up  a rounded fp32 addition is off by 0.2887 steps of 2^-23 / m in the root mean square, m in [1, 2) spread over its logarithm
             (E[1 / m^2] = 0.541): 2.5e-8 of the sum; n chains added in turn, of sums that grow like a walk, sqrt(n / 2) of that, or
             sqrt(n) where chains are a quarter as long; bias and residual, both smaller than twice the products, and the output a
             rounding each: 3e-8 (sqrt(ceil(K / 512)) + 4)
A chain of 1024 is off by 1.0e-6 and breaks the bound at every K here (0.72e-6 to 0.85e-6), sums held in 16 bits break it a
thousandfold.  Of two gated factors each has such an error.
"""
import math

import pytest
import torch

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def api(cuda_device):
    from decode_attention_self_gb300 import api as _api

    return _api


def bound(K):
    return 1.1e-9 * min(K, 512) + 3e-8 * (math.ceil(K / 512) ** 0.5 + 4)


def randn(shape, seed, scale=1.0, dtype=BF16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def ints(shape, seed, most, dtype=BF16):
    return torch.randint(-most, most + 1, shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def rel(got, ref, scale):
    return ((got.double() - ref).norm() / scale.norm()).item()


# every kernel: up to 8, 16 and 32 tokens; CTAs of a cluster, alone, and with accumulators enough for chains of 1024 and 2048; tiles
# of all widths
SUMS = [(1, 1000, 1024), (8, 16384, 128), (13, 8192, 520), (16, 4096, 1000), (32, 1536, 1024), (27, 4096, 1089),
        (33, 16384, 256), (64, 1000, 512), (64, 4096, 4096), (128, 8192, 4096), (128, 16384, 2048), (100, 1024, 1089), (200, 4096, 2000),
        (701, 1000, 1089), (1024, 4096, 1024), (2048, 2048, 1024), (1500, 8192, 520), (600, 16384, 1024), (4099, 1032, 1000),
        (40, 2048, 9800)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N", SUMS)
@pytest.mark.parametrize("bias,residual", [(False, False), (True, True)])
def test_fp32_outputs(api, T, K, N, bias, residual):
    x, W = randn((T, K), K).cuda(), randn((N, K), K + 1, K ** -0.5).cuda()
    b = randn((N,), K + 2, 0.5).cuda() if bias else None
    r = randn((T, N), K + 3, 1.0, F32).cuda() if residual else None
    o = torch.empty((T, N), dtype=F32, device="cuda")
    api.dr_linear(x, W, o, bias=b, residual=r)
    product = x.double() @ W.double().T
    ref = product + (0 if b is None else b.double()) + (0 if r is None else r.double())
    assert rel(o, ref, product) <= bound(K)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N", [(5, 4096, 520), (24, 1536, 512), (64, 2048, 1000), (128, 8192, 1024), (1200, 2048, 1000), (3000, 1000, 520)])
def test_fp32_gated_outputs(api, T, K, N):
    x, W = randn((T, K), K).cuda(), randn((2 * N, K), K + 1, K ** -0.5).cuda()
    o = torch.empty((T, N), dtype=F32, device="cuda")
    api.dr_linear(x, W, o, gated=True)
    a = x.double() @ W.double().T
    ref = a[:, :N] * a[:, N:]
    # (a + da)(b + db) - a b = a db + b da, and the product's rounding; the two errors follow their factors' signs alike
    assert rel(o, ref, ref) <= 2 * bound(K) + 3e-8


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N", SUMS + [(2000, 1024, 1024), (5000, 4096, 1024), (16384, 1024, 512)])
@pytest.mark.parametrize("gated", [False, True])
def test_bf16_outputs_are_rounded_once(api, T, K, N, gated):
    # One rounding to bf16, and a chain that may span all of K: 1.1e-9 K of the value (of either factor) beside it.
    x, W = randn((T, K), K).cuda(), randn((2 * N if gated else N, K), K + 1, K ** -0.5).cuda()
    o = torch.empty((T, N), dtype=BF16, device="cuda")
    api.dr_linear(x, W, o, gated=gated)
    ref = x.double() @ W.double().T
    if gated:
        ref = ref[:, :N] * ref[:, N:]
    rounded = rel(ref.to(BF16), ref, ref)
    assert rel(o, ref, ref) <= rounded + (2 if gated else 1) * (1.1e-9 * K + bound(K))


EXACT = [(1, 8, 33), (3, 72, 64), (8, 16384, 64), (16, 1000, 1089), (20, 1536, 512), (32, 8192, 520), (33, 72, 200), (64, 16384, 64),
         (100, 4096, 4096), (128, 1000, 1000), (200, 520, 2000), (512, 1024, 2560), (701, 1000, 1089), (1900, 72, 1089), (3000, 4096, 520),
         (2500, 200, 2048), (6000, 1032, 1024), (17, 264, 9729), (33, 264, 16384), (64, 1000, 9729), (128, 264, 16384)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N", EXACT)
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("act,gated,residual", [(None, False, True), ("relu", False, False), (None, True, True), ("relu", True, False)])
def test_whole_numbers_are_exact(api, T, K, N, out, act, gated, residual):
    # Whole numbers up to 3: every sum is a whole number below 2^24, which fp32 holds in any order and cut off or not; a term lost or
    # counted twice, a chain that starts on old sums or a step in 16 bits shows.  bf16 outputs are its one rounding, to even.
    N = N // 2 if gated else N
    x, W = ints((T, K), 1, 3).cuda(), ints((2 * N if gated else N, K), 2, 3).cuda()
    b = ints((W.shape[0],), 3, 100).cuda()
    r = ints((T, N), 4, 100, out).cuda() if residual else None
    o = torch.full((T, N), float("nan"), dtype=out, device="cuda")
    api.dr_linear(x, W, o, bias=b, act=act, gated=gated, residual=r)
    a = x.double() @ W.double().T + b.double()
    assert torch.equal(a, a.round())
    v = a[:, :N].clamp_min(0) if act else a[:, :N]
    if gated:
        v = v * a[:, N:]
    if r is not None:
        v = r.double() + v
    assert v.abs().max() < 2 ** 24
    assert torch.equal(o, v.to(out))


@pytest.mark.parametrize("K", [1000, 4096, 16384])
def test_the_bound_finds_lost_terms_and_16_bit_steps(K):
    # planted in the reference: the bound must refuse them, and take fp32 sums
    x, W, r = randn((8, K), 1), randn((64, K), 2, K ** -0.5), randn((8, 64), 3, 1.0, F32)
    product = x.double() @ W.double().T
    ref = product + r.double()
    f = x.float() @ W.float().T
    assert rel(f + r, ref, product) <= bound(K)
    assert rel(f + r.to(BF16).float(), ref, product) > bound(K)          # a residual in 16 bits
    assert rel(f.to(BF16).float() + r, ref, product) > bound(K)          # sums in 16 bits
    assert rel((f + r).to(BF16), ref, product) > bound(K)                # outputs in 16 bits
    short = x[:, :K - 8].float() @ W[:, :K - 8].float().T
    assert rel(short + r, ref, product) > bound(K)                       # the last 8 of K
    assert 1.0e-9 * 1024 > bound(K)                                      # what a chain of 1024 is short by
