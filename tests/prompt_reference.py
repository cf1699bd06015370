"""64-bit references and seeded inputs for the prompt-side operators (test infrastructure).

Tolerances, derived before any GPU result was seen.  eps(t) is half a unit in the last place, relative: bf16 2^-9 of
the binade's top, taken as 2^-8 of the value to cover a value just above a power of two; f16 2^-11.

Attention.  The kernels round each weight once for its product with V (bf16 caches: 2^-8, e4m3 caches: 2^-11),
which moves the output by at most eps_w * sum_j p_j |v_j|.  Scores are fp32 sums of exact products: D + a few
roundings of at most 2^-24 (the tensor cores may truncate: 2^-23) of sum |q k| scale, and the exponentials are good to
about 2^-22; a score off by d moves the output by at most 2 d sum_j p_j |v_j|.  Together
    |got - ref| <= (eps_w + 2 * (72 * 2^-23 * A + E)) * sum_j p_j |v_j| + eps_out |ref|
with A the largest sum_d |q_d k_d| * scale of the row and E = 2^-20, plus, under a cap, the cap's own 2^-21 * cap, and
under a bias 2^-22 of the largest biased score that carries weight (at most 130 + the row's score range).

Rotation.  Table entries are given in fp32 (inputs).  Two products and a sum, each rounded to 2^-24:
    |got - ref| <= 3 * 2^-24 * (|x1| + |x2|) + eps_out |ref|
"""
from __future__ import annotations

import math

import numpy as np
import torch

from decode_attention_self_gb300 import workloads as W

D = 64
PAGE = 16


def to64(codes: torch.Tensor, scale: float) -> torch.Tensor:
    if codes.dtype == torch.uint8:
        return codes.view(torch.float8_e4m3fn).double() * scale
    return codes.double()


class Cache:
    """A cache on the CPU: rows of caps[b] keys; slots from valid[b] on hold `fill`."""

    def __init__(self, caps, Hkv, paged, fp8, seed, valid=None, fill=float("nan"), k_scale=1 / 64, v_scale=1 / 32):
        B = len(caps)
        if paged:
            nblk = [max(1, -(-int(c) // PAGE)) for c in caps]
            total = sum(nblk) + 3
            perm = np.random.default_rng(seed).permutation(total).astype(np.int32)
            table = np.full((B, max(nblk)), -1, np.int32)
            at = 0
            for b, n in enumerate(nblk):
                table[b, :n] = perm[at:at + n]
                at += n
            shape = (total, Hkv, PAGE, D)
            self.table = torch.from_numpy(table)
        else:
            shape = (B, Hkv, max(1, max(int(c) for c in caps)), D)
            self.table = None
        k, v = W.randn_bf16(shape, "cpu", seed, 1), W.randn_bf16(shape, "cpu", seed, 2)
        if valid is not None:
            keep = torch.zeros((shape[0], shape[2]), dtype=torch.bool)
            for b, n in enumerate(valid):
                i0, i2 = self.slots(b, int(n))
                keep[i0, i2] = True
            k.masked_fill_(~keep[:, None, :, None], fill)
            v.masked_fill_(~keep[:, None, :, None], fill)
        self.k_scale, self.v_scale = (k_scale, v_scale) if fp8 else (1.0, 1.0)
        if fp8:
            k, v = (W.to_e4m3_codes(torch.nan_to_num(x.float(), nan=0.0), s, torch.isnan(x))
                    for x, s in ((k, k_scale), (v, v_scale)))
        self.k, self.v = k, v

    def slots(self, b, n):
        j = torch.arange(n)
        if self.table is None:
            return torch.full_like(j, b), j
        return self.table[b].long()[j // PAGE], j % PAGE

    def rows(self, b, n):
        """(keys, values) 0..n-1 of row b, [Hkv, n, D] float64."""
        i0, i2 = self.slots(b, n)
        return (to64(self.k, self.k_scale)[i0, :, i2].transpose(0, 1) if n else torch.zeros(self.k.shape[1], 0, D).double(),
                to64(self.v, self.v_scale)[i0, :, i2].transpose(0, 1) if n else torch.zeros(self.k.shape[1], 0, D).double())

    def gpu(self, api, dev):
        return api.KVCache(self.k.to(dev), self.v.to(dev), None if self.table is None else self.table.to(dev),
                           self.k_scale, self.v_scale)


def attend(q, keys, vals, lo, hi, pos, scale=D ** -0.5, softcap=0.0, slopes=None, fp8=False, out_dtype=torch.float32):
    """q [n, Hq, D], keys/vals [Hkv, L, D] float64; visible keys [lo, hi) per query -> (ref, tolerance) [n, Hq, D]."""
    n, Hq, _ = q.shape
    Hkv, L, _ = keys.shape
    g = Hq // Hkv
    q = q.double()
    ref, tol = torch.zeros(n, Hq, D, dtype=torch.float64), torch.zeros(n, Hq, D, dtype=torch.float64)
    if L == 0:
        return ref, tol
    j = torch.arange(L)
    seen = (j[None] >= lo[:, None]) & (j[None] < hi[:, None])
    eps_w = 2.0 ** -11 if fp8 else 2.0 ** -8
    for h in range(Hq):
        K, V = keys[h // g], vals[h // g]
        # hidden keys may hold anything: keep them out of the products
        any_seen = seen.any(0)
        K, V = torch.where(any_seen[:, None], K, 0.0), torch.where(any_seen[:, None], V, 0.0)
        s = q[:, h] @ K.T * scale
        mag = (q[:, h].abs() @ K.abs().T * abs(scale)).masked_fill(~seen, 0.0).amax(1)
        extra = 0.0
        if softcap:
            s = softcap * torch.tanh(s / softcap)
            extra += 2.0 ** -21 * softcap
        if slopes is not None:
            s = s - slopes[h].double() * (pos[:, None] - j[None]).abs()
            extra += 2.0 ** -22 * (130.0 + 2.0 * float(mag.max()))
        s = s.masked_fill(~seen, -math.inf)
        ok = seen.any(1)
        p = torch.zeros_like(s)
        p[ok] = torch.softmax(s[ok], 1)
        ref[:, h] = p @ V
        d = 72 * 2.0 ** -23 * mag + 2.0 ** -20 + extra
        tol[:, h] = (eps_w + 2 * d)[:, None] * (p @ V.abs())
    if out_dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * ref.abs()
    return ref, tol + 2.0 ** -23 * ref.abs() + 1e-30


def assert_close(got, ref, tol, what=""):
    g = got.detach().double().cpu()
    assert g.shape == ref.shape
    bad = ~((g - ref).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} out of tolerance, first "
                           f"{bad.nonzero()[0].tolist()}: got {g[bad][0]:.6g} ref {ref[bad][0]:.6g} "
                           f"tol {tol[bad][0]:.3g}")


def starts(lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)
