"""dr_residual_norm's statistics against bounds of the sums it really makes.

A row's sum passes through few roundings: up to 32 elements a thread, two at a time (16 additions and one that joins the two), 5 of a
warp's shuffles, and the row's warps in turn (256 elements or more each, at most 16): depth = 22 + min(16, ceil(D / 256)).  Of
U = 2^-24 each:
  mean      off by (depth + 2) U mean|v| (the sum, 1 / D, the product), and U of the difference
  variance  relative (depth + 4) U (the sum of squares, 1 / D, the product, eps), halved by the root; the root and its reciprocal
            2 U.  A mean off by d adds d^2 to it: second order
  y         three roundings: times the reciprocal root, weight, bias
Mean square less squared mean in fp32 has lost these differences where rows lie far from zero; that is checked here at every width.
"""
import math

import pytest
import torch

from layer_reference import U, assert_within, half_step

BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


@pytest.fixture(scope="module")
def api(cuda_device):
    from decode_attention_self_gb300 import api as _api

    return _api


def randn(shape, seed, dtype=BF16, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale + shift).to(dtype)


def norm_bound(v, dv, kind, weight, bias, dtype):
    """(norm in float64, tolerance) of rows v that are known to within dv."""
    D = v.shape[1]
    depth = 22 + min(16, math.ceil(D / 256))
    c, off = v, torch.zeros_like(v)
    if kind == "layer":
        c = v - v.mean(1, keepdim=True)
        off = (depth + 2) * U * v.abs().mean(1, keepdim=True) + U * c.abs() + dv.mean(1, keepdim=True)
    off = off + dv
    r = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + EPS)
    y = c * r
    moved = torch.sqrt((off * off).mean(1, keepdim=True)) * r            # of the root mean square, relative, by Cauchy and Schwarz
    dy = y.abs() * (((depth + 4) / 2 + 3) * U + moved) + off * r * (1 + moved)
    w, b = weight.double(), bias.double()
    dy = dy * w.abs() + U * (y * w).abs()
    y = y * w + b
    dy = dy + U * y.abs()
    return y, dy + half_step(dtype) * (y.abs() + dy) + 1e-30


def problem(T, D, kind, dtype, res):
    x, w, b = randn((T, D), D + 1, F32), randn((D,), D + 2, BF16, 0.3, 1.0), randn((D,), D + 3, BF16, 0.3)
    v = res.double() + x.double()
    y, tol = norm_bound(v, U * v.abs(), kind, w, b, dtype)
    return x, w, b, y, tol


def far(T, D, seed):
    return randn((T, D), seed, F32, 1.0, 1000.0)


def few_large(T, D, seed):
    res = randn((T, D), seed, F32)
    res[:, 5], res[:, D - 1] = 300.0, -900.0
    return res


WIDTHS = [64, 256, 1000, 1024, 2048, 4096, 5000, 8192, 16384]


@pytest.mark.gpu
@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("T", [7, 1201])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("rows", [far, few_large, lambda T, D, seed: randn((T, D), seed, F32, 2.0, 0.5)], ids=["far", "few large", "plain"])
def test_statistics(api, T, D, kind, rows):
    res = rows(T, D, D)
    for dtype in (F32, BF16):
        x, w, b, ref, tol = problem(T, D, kind, dtype, res)
        y = torch.full((T, D), float("nan"), dtype=dtype, device="cuda")
        api.dr_residual_norm(x.cuda(), y=y, pre=api.Norm(kind, EPS, w.cuda(), b.cuda()), residual=res.cuda())
        assert_within(y, ref, tol, f"{kind} T={T} D={D} {dtype}")


@pytest.mark.gpu
@pytest.mark.parametrize("D", WIDTHS)
def test_statistics_of_the_norm_after_a_block(api, D):
    x, w, b = far(9, D, D), randn((D,), D + 2, BF16, 0.3, 1.0), randn((D,), D + 3, BF16, 0.3)
    v = x.double()
    ref, tol = norm_bound(v, torch.zeros_like(v), "layer", w, b, F32)
    h = torch.full((9, D), float("nan"), dtype=F32, device="cuda")
    api.dr_residual_norm(x.cuda(), h=h, residual=torch.zeros((9, D), device="cuda"), post=api.Norm("layer", EPS, w.cuda(), b.cuda()))
    assert_within(h, ref, tol, f"D={D}")


@pytest.mark.parametrize("D", WIDTHS)
def test_the_bound_refuses_what_it_should(D):
    # planted in a float32 reference: it must be refused at every width, and the form in two passes taken
    res = far(7, D, D)
    x, w, b, ref, tol = problem(7, D, "layer", F32, res)
    v = res + x
    mean = v.mean(1, keepdim=True)

    def finish(c, var):
        return c / torch.sqrt(var + EPS) * w.float() + b.float()

    def off(y):
        return int(((y.double() - ref).abs() > tol).sum())

    assert off(finish(v - mean, ((v - mean) ** 2).mean(1, keepdim=True))) == 0
    assert off(finish(v - mean, (v * v).mean(1, keepdim=True) - mean ** 2)) > 0          # one pass
    assert off(finish(v - mean, ((v - mean) ** 2).mean(1, keepdim=True)).to(BF16)) > 0   # outputs in 16 bits
    short = v[:, :D - 8]
    m = short.sum(1, keepdim=True) / D
    assert off(finish(v - m, ((v - m) ** 2).mean(1, keepdim=True))) > 0                  # the last vector left out of the mean
