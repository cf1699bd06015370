"""The work between a decoder layer's attention calls: real cases, plain forms, exact values.

Two operators on bf16 weights:
  linear         out = residual + act(x W^T + bias), plain or gated, columns in one output or in several (q, k, v)
  residual_norm  h = residual + scale * gate * post(x) and y = pre(h), post and pre being layer or RMS norms

`run` computes them with elementary torch operations in 32 bits, or (own = True) through the library's calls.
"""
from __future__ import annotations

import math

import torch

own = False

ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
NORMS = ["none", "layer", "rms"]
EPS = 1e-5


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------
def _linear(name, tokens, k, n, act="none", gated=False, bias=True, residual=False, out="bf16", split="", packed=False):
    return {"name": name, "op": "linear", "tokens": tokens, "k": k, "n": n, "act": act, "gated": gated, "bias": bias,
            "residual": residual, "out": out, "split": split, "packed": packed}


def _norm(name, tokens, dm, pre="layer", post="none", gate="none", scale=1.0, residual=True, stream="bf16", x="bf16",
          y="bf16", bias=True, store=True):
    return {"name": name, "op": "residual_norm", "tokens": tokens, "dm": dm, "pre": pre, "post": post, "gate": gate,
            "scale": scale, "residual": residual, "stream": stream, "x": x, "y": y, "bias": bias, "store": store}


def listed():
    return [
        # a batch-1 voice: attention output back into the residual stream; the smallest product, latency alone
        _linear("linear one token", 1, 1024, 1024, residual=True),
        # one step of 32 rows: queries, keys and values of grouped heads (16 and 4) from one projection
        _linear("linear qkv batch 32", 32, 1024, 1536, bias=False, split="1024,256,256"),
        # one step of a full batch: the two products of the MLP
        _linear("linear up batch 128", 128, 1024, 4096, act="gelu"),
        _linear("linear down batch 128", 128, 4096, 1024, residual=True),
        # text prompts of several rows, an odd count of tokens: an odd vocabulary's logits, fp32
        _linear("linear odd vocabulary", 701, 1000, 1089, bias=True, out="f32"),
        # a batch of ragged prompts through a gated MLP, x a slice of a wider buffer
        _linear("linear gated prompts", 2477, 1536, 4096, act="silu", gated=True, bias=False, packed=True),
        # one long prompt: the two products of the MLP, the second into an fp32 residual stream
        _linear("linear up long prompt", 16384, 1024, 4096, act="gelu"),
        _linear("linear down long prompt", 16384, 4096, 2048, residual=True, out="f32"),
        # a batch-1 voice: the norm before the next block
        _norm("residual_norm one token", 1, 1024),
        # a full batch: norms after and before a block, a gate per channel, a residual scale
        _norm("residual_norm batch 128", 128, 1536, pre="rms", post="rms", gate="channel", scale=0.5, bias=False),
        # ragged prompts, fp32 residual stream, a gate per token
        _norm("residual_norm prompts", 2477, 2048, gate="token", stream="f32"),
        # one long prompt: memory alone
        _norm("residual_norm long prompt", 65536, 1024, pre="rms", bias=False),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    if rng.random() < 0.65:
        k = 8 * _logint(rng, 8, 1024)
        if rng.random() < 0.5:
            k = max(64, k // 64 * 64)
        n = _logint(rng, 8, 8192)
        if rng.random() < 0.7:
            n = max(64, n // 64 * 64)
        gated = rng.random() < 0.25
        room = int(1.3e11 / (k * n * (2 if gated else 1)))
        # decode batches and prompts alike; a case stays below the largest listed one
        tokens = _logint(rng, 1, max(1, min(65536, room)))
        split = ""
        if not gated and n % 64 == 0 and n >= 192 and rng.random() < 0.4:
            heads = n // 64
            a = rng.randint(1, heads - 2)
            b = rng.randint(1, heads - a - 1)
            split = f"{64 * a},{64 * b},{64 * (heads - a - b)}"
        c = _linear("", tokens, k, n, rng.choice(ACTS[1:] if gated else ACTS), gated, rng.random() < 0.6,
                    not split and rng.random() < 0.4, rng.choice(["bf16", "bf16", "bf16", "f32"]), split,
                    rng.random() < 0.3)
    else:
        dm = 8 * _logint(rng, 8, 1024)
        tokens = _logint(rng, 1, max(1, min(65536, 64_000_000 // dm)))
        residual = rng.random() < 0.8
        c = _norm("", tokens, dm, rng.choice(NORMS[1:]), rng.choice(NORMS), rng.choice(["none", "none", "channel", "token"]),
                  rng.choice([1.0, 1.0, 0.5, 0.125]), residual, rng.choice(["bf16", "f32"]),
                  rng.choice(["bf16", "bf16", "f32"]), rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.5,
                  residual or rng.random() < 0.3)
    c.pop("name")
    return c


def _rows_of_w(case):
    return case["n"] * (2 if case["gated"] else 1)


def _size(kind):
    return 4 if kind == "f32" else 2


def work(case):
    t = case["tokens"]
    if case["op"] == "linear":
        k, n, w = case["k"], case["n"], _rows_of_w(case)
        e = _size(case["out"])
        return {"bytes": 2 * t * k + 2 * w * k + (2 * w if case["bias"] else 0) + t * n * e * (2 if case["residual"] else 1),
                "flops": 2 * t * k * w}
    dm = case["dm"]
    gate = {"none": 0, "channel": 2 * dm, "token": 2 * t * dm}[case["gate"]]
    streams = (1 if case["residual"] else 0) + (1 if case["store"] else 0)
    vectors = sum(2 * dm * (2 if case["bias"] and kind == "layer" else 1) for kind in (case["pre"], case["post"]) if kind != "none")
    return {"bytes": t * dm * (_size(case["x"]) + streams * _size(case["stream"]) + _size(case["y"])) + gate + vectors,
            "flops": t * dm * 10}


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------
def _type(kind):
    return torch.float32 if kind == "f32" else torch.bfloat16


def _randn(shape, g, kind="bf16", scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(_type(kind))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = case["tokens"]
    st = {"case": case}
    if case["op"] == "linear":
        k, n = case["k"], case["n"]
        if case["packed"]:
            # x is a slice of a wider buffer, as after a fused projection
            st["x"] = _randn((t, k + 64), g)[:, 64:]
        else:
            st["x"] = _randn((t, k), g)
        st["w"] = _randn((_rows_of_w(case), k), g, scale=1.0 / math.sqrt(k))
        st["bias"] = _randn((_rows_of_w(case),), g, scale=0.3) if case["bias"] else None
        st["residual"] = _randn((t, n), g, case["out"]) if case["residual"] else None
        widths = [int(w) for w in case["split"].split(",")] if case["split"] else [n]
        outs = [torch.zeros((t, w), dtype=_type(case["out"]), device="cuda") for w in widths]
        st["out"] = outs if case["split"] else outs[0]
        return st
    dm = case["dm"]

    def stream(kind):
        # a residual stream has a few channels far larger than the others
        x = torch.randn((t, dm), generator=g, device="cuda", dtype=torch.float32)
        big = torch.randint(0, dm, (3,), generator=g, device="cuda")
        x[:, big] = x[:, big] * 20.0 + 15.0
        return x.to(_type(kind))

    def params(kind):
        if kind == "none":
            return None, None
        w = (1.0 + 0.2 * torch.randn((dm,), generator=g, device="cuda")).to(torch.bfloat16)
        return w, _randn((dm,), g, scale=0.1) if case["bias"] and kind == "layer" else None

    st["x"] = stream(case["x"]) if not case["residual"] else _randn((t, dm), g, case["x"])
    st["residual"] = stream(case["stream"]) if case["residual"] else None
    st["gate"] = None
    if case["gate"] == "channel":
        st["gate"] = _randn((dm,), g)
    elif case["gate"] == "token":
        st["gate"] = _randn((t, dm), g)
    st["pre_w"], st["pre_b"] = params(case["pre"])
    st["post_w"], st["post_b"] = params(case["post"])
    st["h"] = torch.zeros((t, dm), dtype=_type(case["stream"]), device="cuda") if case["store"] else None
    st["y"] = torch.zeros((t, dm), dtype=_type(case["y"]), device="cuda")
    if own:
        from decode_attention_self_gb300 import api
        st["pre"] = api.Norm(case["pre"], EPS, st["pre_w"], st["pre_b"])
        st["post"] = None if case["post"] == "none" else api.Norm(case["post"], EPS, st["post_w"], st["post_b"])
    return st


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------
def _act(a, act):
    if act == "relu":
        return a.clamp_min(0.0)
    if act == "gelu":
        return 0.5 * a * torch.erfc(-a * math.sqrt(0.5))
    if act == "gelu_tanh":
        return 0.5 * a * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (a + 0.044715 * a * a * a)))
    if act == "silu":
        return a / (1.0 + torch.exp(-a))
    return a


def _plain_linear(st):
    case = st["case"]
    a = torch.matmul(st["x"].float(), st["w"].float().t())
    if st["bias"] is not None:
        a = a + st["bias"].float()
    if case["gated"]:
        v = _act(a[:, :case["n"]], case["act"]) * a[:, case["n"]:]
    else:
        v = _act(a, case["act"])
    if st["residual"] is not None:
        v = st["residual"].float() + v
    if not case["split"]:
        st["out"].copy_(v)
        return st["out"]
    at = 0
    for o in st["out"]:
        o.copy_(v[:, at:at + o.shape[1]])
        at += o.shape[1]
    return st["out"]


def _plain_norm(x, kind, w, b):
    if kind == "none":
        return x
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    return y if b is None else y + b.float()


def _plain_residual_norm(st):
    case = st["case"]
    v = _plain_norm(st["x"].float(), case["post"], st["post_w"], st["post_b"])
    if st["gate"] is not None:
        v = v * st["gate"].float()
    h = v * case["scale"]
    if st["residual"] is not None:
        h = h + st["residual"].float()
    if st["h"] is not None:
        st["h"].copy_(h)
    st["y"].copy_(_plain_norm(h, case["pre"], st["pre_w"], st["pre_b"]))
    return {"h": st["h"], "y": st["y"]}


def run(st):
    case = st["case"]
    if not own:
        return _plain_linear(st) if case["op"] == "linear" else _plain_residual_norm(st)
    from decode_attention_self_gb300 import api
    if case["op"] == "linear":
        return api.dr_linear(st["x"], st["w"], st["out"], bias=st["bias"], act=case["act"], gated=case["gated"],
                             residual=st["residual"])
    api.dr_residual_norm(st["x"], y=st["y"], pre=st["pre"], residual=st["residual"], h=st["h"], post=st["post"],
                         gate=st["gate"], scale=case["scale"])
    return {"h": st["h"], "y": st["y"]}


# ---------------------------------------------------------------------------------------------------------------
# exact values, from the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------
def _phi(z):
    """The normal distribution's share below z."""
    return torch.special.erfc(z * -(0.5 ** 0.5)) / 2


def _exact_act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return z * _phi(z)
    if act == "gelu_tanh":
        u = (2.0 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3)
        return z * torch.sigmoid(2 * u)      # (1 + tanh u) / 2
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def _exact_norm(rows, kind, w, b):
    if kind == "none":
        return rows
    if kind == "layer":
        var, mean = torch.var_mean(rows, dim=1, correction=0)
        rows = rows - mean[:, None]
    else:
        var = rows.pow(2).sum(1) / rows.shape[1]
    out = rows * torch.rsqrt(var + EPS)[:, None] * w.double()[None, :]
    return out if b is None else out + b.double()[None, :]


def exact(case, seed):
    if work(case)["flops"] > 6.0e11:
        return None
    st = prepare(case, seed)
    t = case["tokens"]
    if case["op"] == "linear":
        w = st["w"].double()
        bias = 0.0 if st["bias"] is None else st["bias"].double()
        n = case["n"]
        out = torch.empty((t, n), dtype=torch.float64, device="cuda")
        for i in range(0, t, 4096):
            z = torch.nn.functional.linear(st["x"][i:i + 4096].double(), w) + bias
            part = _exact_act(z[:, :n], case["act"])
            if case["gated"]:
                part = part * z[:, n:]
            if st["residual"] is not None:
                part = part + st["residual"][i:i + 4096].double()
            out[i:i + 4096] = part
        if not case["split"]:
            return out
        return list(torch.split(out, [int(s) for s in case["split"].split(",")], dim=1))
    rows = _exact_norm(st["x"].double(), case["post"], st["post_w"], st["post_b"]) * case["scale"]
    if st["gate"] is not None:
        rows = rows * st["gate"].double()
    if st["residual"] is not None:
        rows = rows + st["residual"].double()
    return {"h": rows if case["store"] else None, "y": _exact_norm(rows, case["pre"], st["pre_w"], st["pre_b"])}
