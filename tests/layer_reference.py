"""Plain float64 forms of the layer operators and the bounds of their fp32 arithmetic (test infrastructure).

Bounds, derived before any result was seen:
  sums        products of bf16 are exact in fp32; a K-term fp32 sum, cut off or rounded, in any order:
              (K - 1) * 2^-23 * sum_k |x_k w_k|
  bias        2^-24 of the sum
  activations slope at most 1.13 (gelu's steepest; silu 1.10, gelu_tanh 1.13), and an evaluation error of 5e-7 + 2^-21 |v|:
              the fits' 1e-6 of at most 0.17, exponentials of 2 ulp, reciprocals of 1 ulp, a rounded exponent of |a| 2^-24
  gating      |u| db + |b| du + du db
  residual    2^-24 of the sum;  outputs: half a step, 2^-24 or 2^-8 of the value
  norms       statistics of Dm terms: relative Dm * 2^-24 at the worst for the mean square; a mean off by
              Dm * 2^-24 * mean |v|, which is divided by the deviation like everything else
"""
import math

import torch

U = 2.0 ** -24


def act64(a, act):
    if act == "relu":
        return a.clamp_min(0)
    if act == "gelu":
        return a * 0.5 * torch.special.erfc(-a / math.sqrt(2))
    if act == "gelu_tanh":
        return a * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3))
    if act == "silu":
        return a * torch.sigmoid(a)
    return a


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def linear64(x, W, bias, act, gated, residual, out_dtype):
    """(reference, tolerance) of dr_linear, float64, on the CPU."""
    x, W = x.double().cpu(), W.double().cpu()
    K = x.shape[1]
    a = x @ W.T
    da = (K - 1) * 2 * U * (x.abs() @ W.abs().T)
    if bias is not None:
        a = a + bias.double().cpu()
        da = da + U * a.abs()
    N = W.shape[0] // 2 if gated else W.shape[0]
    if act in (None, "none"):
        v, dv = a[:, :N], da[:, :N]
    else:
        v = act64(a[:, :N], act)
        dv = 1.13 * da[:, :N] + 5e-7 + 8 * U * v.abs()
    if gated:
        b, db = a[:, N:], da[:, N:]
        dv = v.abs() * db + b.abs() * dv + dv * db + U * (v * b).abs()
        v = v * b
    if residual is not None:
        v = residual.double().cpu() + v
        dv = dv + U * v.abs()
    return v, dv + half_step(out_dtype) * (v.abs() + dv) + 1e-30


def norm64(v, kind, eps, weight, bias):
    """(value, bound of its fp32 arithmetic) of a norm of exact rows v."""
    D = v.shape[1]
    mag = v.abs().mean(1, keepdim=True)
    if kind == "layer":
        c = v - v.mean(1, keepdim=True)
        off = (D + 2) * U * mag          # the mean's error, and one rounding of the difference
    else:
        c = v
        off = torch.zeros_like(mag)
    var = (c * c).mean(1, keepdim=True)
    r = 1 / torch.sqrt(var + eps)
    y = c * r
    # relative error of the root mean square: the sum's, the shared offset's, and four roundings
    rel = (D + 4) * U + off * r
    dy = y.abs() * rel + off * r + U * y.abs() + U * v.abs() * r
    w = torch.ones(D, dtype=torch.float64) if weight is None else weight.double().cpu()
    dy = dy * w.abs() + U * (y * w).abs()
    y = y * w
    if bias is not None:
        y = y + bias.double().cpu()
        dy = dy + U * y.abs()
    return y, dy


def norm_slope(v, kind, eps, weight):
    """How far a change of d in every element of a row can move its norm, at most: 2 d max|weight| sqrt(D) / rms."""
    c = v - v.mean(1, keepdim=True) if kind == "layer" else v
    r = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + eps)
    w = 1.0 if weight is None else weight.double().abs().max().item()
    return 2 * w * r


def residual_norm64(x, post, gate, scale, residual, pre, h_dtype, y_dtype):
    """((h, tolerance), (y, tolerance)); post and pre are (kind, eps, weight, bias) or None."""
    v = x.double().cpu()
    dv = torch.zeros_like(v)
    if post is not None:
        v, dv = norm64(v, *post)
    if gate is not None:
        g = gate.double().cpu()
        v, dv = v * g, dv * g.abs() + U * (v * g).abs()
    v, dv = v * scale, dv * abs(scale) + U * (v * scale).abs()
    if residual is not None:
        v = residual.double().cpu() + v
        dv = dv + U * v.abs()
    h = (v, dv + half_step(h_dtype) * (v.abs() + dv) + 1e-30)
    if pre is None:
        return h, (v, dv + half_step(y_dtype) * (v.abs() + dv) + 1e-30)
    y, dy = norm64(v, *pre)
    # what h is off by moves the norm by its slope: directly, and through the statistics (at most the row's root mean square of it)
    carried = norm_slope(v, pre[0], pre[1], pre[2]) * (dv + (1 + y.abs()) * torch.sqrt((dv * dv).mean(1, keepdim=True)))
    dy = dy + carried
    return h, (y, dy + half_step(y_dtype) * (y.abs() + dy) + 1e-30)


def assert_within(got, ref, tol, what):
    g = got.detach().double().cpu()
    assert g.shape == ref.shape, (g.shape, ref.shape)
    bad = ~((g - ref).abs() <= tol)
    if bad.any():
        at = bad.nonzero()[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} elements off, first at {at}: {g[tuple(at)].item()} "
                             f"for {ref[tuple(at)].item()} +- {tol[tuple(at)].item()}")
