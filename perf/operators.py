"""Prompt-side and batch-shared attention operators: real cases, plain forms, exact values.

Three operators around the KV cache (head dimension 64, 16-key blocks, bf16 or e4m3):
  rope_append    rotate q and k by position and append k, v of ragged new tokens to the cache
  prompt_attn    ragged queries over the cache, with score cap, distance bias, causal / prefix / document mask
  shared_prefix  one query per row over a prefix that all rows share and the row's own keys

`run` computes them with elementary torch operations in 32 bits, or (own = True) through the library's calls.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

D = 64
PAGE = 16
K_SCALE, V_SCALE = 1.0 / 64.0, 1.0 / 32.0
ROPE_BASE = 10000.0


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------
def _rope(name, rows, new_lo, new_hi, start_hi, hq, hkv, kv="bf16", paged=True, rot=64, inter=False, offset=0,
          packed=True, lens_seed=1):
    return {"name": name, "op": "rope_append", "rows": rows, "new_lo": new_lo, "new_hi": new_hi, "start_hi": start_hi,
            "hq": hq, "hkv": hkv, "kv": kv, "paged": paged, "rot": rot, "inter": inter, "offset": offset,
            "packed": packed, "lens_seed": lens_seed}


def _prompt(name, rows, new_lo, new_hi, past_hi, hq, hkv, kv="bf16", paged=True, softcap=0.0, bias=False,
            mask="causal", lens_seed=1):
    return {"name": name, "op": "prompt_attn", "rows": rows, "new_lo": new_lo, "new_hi": new_hi, "past_hi": past_hi,
            "hq": hq, "hkv": hkv, "kv": kv, "paged": paged, "softcap": softcap, "bias": bias, "mask": mask,
            "lens_seed": lens_seed}


def _shared(name, rows, prefix, own_lo, own_hi, hq, hkv, kv="bf16", paged=True, softcap=0.0, lens_seed=1):
    return {"name": name, "op": "shared_prefix", "rows": rows, "prefix": prefix, "own_lo": own_lo, "own_hi": own_hi,
            "hq": hq, "hkv": hkv, "kv": kv, "paged": paged, "softcap": softcap, "lens_seed": lens_seed}


def listed():
    return [
        # one decode step of a batch-1 voice: the smallest call, latency alone
        _rope("rope_append one token", 1, 1, 1, 1024, 16, 16, paged=False, lens_seed=3),
        # one decode step of a full batch, q, k and v as slices of one projection
        _rope("rope_append batch 128", 128, 1, 1, 4095, 16, 16, lens_seed=4),
        # a batch of text prompts into an 8-bit cache, grouped heads, half of the dimensions rotated, past a shared prefix
        _rope("rope_append prompts e4m3", 37, 5, 1200, 64, 16, 4, kv="e4m3", rot=32, inter=True, offset=2048,
              lens_seed=5),
        # one long prompt into a static cache
        _rope("rope_append long prompt", 1, 65536, 65536, 0, 16, 16, paged=False, lens_seed=6),
        # one sentence of description text, causal: latency
        _prompt("prompt_attn one sentence", 1, 64, 64, 0, 16, 16, lens_seed=7),
        # single tokens of a ragged batch with capped scores: the decode form
        _prompt("prompt_attn single tokens capped", 32, 1, 1, 2047, 16, 4, softcap=30.0, lens_seed=8),
        # a ragged batch of packed documents with a distance bias
        _prompt("prompt_attn documents biased", 9, 17, 2100, 130, 16, 4, bias=True, mask="document", lens_seed=9),
        # the next chunk of long inputs in an 8-bit cache, after a two-way prefix
        _prompt("prompt_attn chunk e4m3 prefix", 3, 300, 700, 20000, 16, 16, kv="e4m3", mask="prefix", lens_seed=10),
        # one long prompt, causal: the compute bound
        _prompt("prompt_attn long prompt", 1, 16384, 16384, 0, 16, 16, lens_seed=11),
        # a few utterances of one voice: latency
        _shared("shared_prefix batch 8", 8, 500, 1, 64, 16, 16, lens_seed=12),
        # a full batch over one long description in an 8-bit cache, grouped heads
        _shared("shared_prefix batch 48 long e4m3", 48, 32777, 0, 300, 16, 4, kv="e4m3", lens_seed=13),
        # a full batch over one voice prompt, each row far into its own output
        _shared("shared_prefix batch 128", 128, 4096, 64, 2048, 16, 16, lens_seed=14),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope_append", "prompt_attn", "shared_prefix"])
    kv = rng.choice(["bf16", "bf16", "e4m3"])
    paged = rng.random() < 0.7
    hkv = rng.choice([1, 2, 4, 8, 16])
    hq = hkv * rng.choice([g for g in (1, 2, 3, 4, 7, 8, 16) if g * hkv <= 32])
    seed = rng.randrange(1, 1 << 30)
    if op == "rope_append":
        rows = _logint(rng, 1, 256)
        per = 8_000 * 48 // (hq + 2 * hkv)
        new_hi = 1 if rng.random() < 0.3 else _logint(rng, 1, max(1, min(65536, 4 * per // rows)))
        new_lo = 0 if new_hi > 4 and rng.random() < 0.3 else rng.randint(1, max(1, new_hi // 3))
        return {k: v for k, v in _rope("", rows, new_lo, new_hi, _logint(rng, 1, 4096), hq, hkv, kv, paged,
                                       rng.choice([0, 16, 32, 48, 64, 64, 64]), rng.random() < 0.4,
                                       rng.choice([0, 0, _logint(rng, 1, 100000)]), rng.random() < 0.6,
                                       seed).items() if k != "name"}
    if op == "prompt_attn":
        rows = _logint(rng, 1, 64)
        new_hi = 1 if rng.random() < 0.25 else _logint(rng, 2, min(8192, max(2, 60_000 // rows)))
        past = rng.choice([0, _logint(rng, 1, max(1, min(32768, 250_000_000 // (rows * new_hi), 250_000 // rows)))])
        mask = rng.choice(["causal", "causal", "document", "prefix", "none"])
        return {k: v for k, v in _prompt("", rows, max(1, new_hi // rng.choice([1, 3, 40])), new_hi, past, hq, hkv, kv,
                                         paged, rng.choice([0.0, 0.0, 15.0, 50.0]), rng.random() < 0.35, mask,
                                         seed).items() if k != "name"}
    rows = _logint(rng, 1, 256)
    own_hi = _logint(rng, 1, min(2048, max(1, 200_000 // rows)))
    own_lo = rng.choice([0, 1, max(1, own_hi // 4)])
    return {k: v for k, v in _shared("", rows, _logint(rng, 1, 32768), min(own_lo, own_hi), own_hi, hq, hkv, kv, paged,
                                     rng.choice([0.0, 0.0, 0.0, 30.0]), seed).items() if k != "name"}


def _lengths(case):
    """(first, second) per-row whole numbers of a case: they belong to the case, not to the inputs' seed."""
    r = np.random.default_rng([case["lens_seed"], case["rows"]])
    B = case["rows"]
    if case["op"] == "rope_append":
        new = r.integers(case["new_lo"], case["new_hi"], size=B, endpoint=True)
        return new, r.integers(0, case["start_hi"], size=B, endpoint=True)
    if case["op"] == "prompt_attn":
        new = r.integers(case["new_lo"], case["new_hi"], size=B, endpoint=True)
        return new, new + r.integers(case["past_hi"] // 3, case["past_hi"], size=B, endpoint=True)
    return r.integers(case["own_lo"], case["own_hi"], size=B, endpoint=True), None


def _intervals(case):
    """prompt_attn: the visible keys [lo, hi) of every query token, and the mask arrays a user passes."""
    new, kv = _lengths(case)
    r = np.random.default_rng([case["lens_seed"], 5])
    lo, hi, first, prefix = [], [], [], []
    for n, L in zip(new.tolist(), kv.tolist()):
        pos = np.arange(L - n, L)
        if case["mask"] == "document":
            # documents of about a third of the row: a query sees its own document from its first key on
            cuts = np.unique(np.concatenate([[0], r.integers(0, L, size=3)]))
            f = cuts[np.searchsorted(cuts, pos, side="right") - 1]
        else:
            f = np.zeros(n, np.int64)
        h = np.full(n, L) if case["mask"] == "none" else pos + 1
        if case["mask"] == "prefix":
            p = int(r.integers(0, L, endpoint=True))
            prefix.append(p)
            h = np.maximum(h, p)
        first.append(f)
        lo.append(f)
        hi.append(h)
    return np.concatenate(lo), np.concatenate(hi), np.concatenate(first), np.array(prefix, np.int32)


def work(case):
    e = 2 if case["kv"] == "bf16" else 1
    hq, hkv = case["hq"], case["hkv"]
    a, b = _lengths(case)
    if case["op"] == "rope_append":
        T = int(a.sum())
        return {"bytes": T * ((2 * hq + 2 * hkv) * D * 2 + 2 * hkv * D * e + case["rot"] * 4),
                "flops": T * (hq + hkv) * case["rot"] * 3}
    if case["op"] == "prompt_attn":
        lo, hi, _, _ = _intervals(case)
        T = int(a.sum())
        reached, at = 0, 0
        for n in a.tolist():
            if n:
                reached += int(hi[at:at + n].max()) - int(lo[at:at + n].min())
            at += n
        return {"bytes": 2 * T * hq * D * 2 + 2 * reached * hkv * D * e,
                "flops": 4 * D * hq * int(np.maximum(hi - lo, 0).sum())}
    B, P, S = case["rows"], case["prefix"], int(a.sum())
    return {"bytes": 2 * B * hq * D * 2 + 2 * (P + S) * hkv * D * e, "flops": 4 * D * hq * (B * P + S)}


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _stored(x, kv, scale):
    """bf16 values as the cache holds them: themselves, or e4m3 codes (uint8)."""
    if kv == "bf16":
        return x
    return (x.float() / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _cache(case, caps, valid, g, seed):
    """A cache of len(caps) rows for caps[b] keys each; with valid, slots from valid[b] on hold NaN."""
    B, hkv, kv = len(caps), case["hkv"], case["kv"]
    if case["paged"]:
        nblk = [max(1, -(-int(c) // PAGE)) for c in caps]
        total = sum(nblk) + 7
        perm = np.random.default_rng([seed, 99]).permutation(total).astype(np.int32)
        table = np.full((B, max(nblk)), -1, np.int32)
        at = 0
        for b, n in enumerate(nblk):
            table[b, :n] = perm[at:at + n]
            at += n
        shape = (total, hkv, PAGE, D)
    else:
        table = None
        shape = (B, hkv, max(1, int(max(caps))), D)
    k, v = _randn(shape, g), _randn(shape, g)
    if valid is not None:
        if case["paged"]:
            ok = np.zeros((shape[0], PAGE), bool)
            for b, n in enumerate(valid):
                for j in range(-(-int(n) // PAGE)):
                    ok[table[b, j], :min(PAGE, int(n) - PAGE * j)] = True
            bad = ~torch.from_numpy(ok).cuda().view(shape[0], 1, PAGE, 1)
        else:
            bad = torch.arange(shape[2], device="cuda").view(1, 1, -1, 1) >= torch.as_tensor(
                np.asarray(valid, np.int64), device="cuda").view(-1, 1, 1, 1)
        k.masked_fill_(bad, float("nan"))
        v.masked_fill_(bad, float("nan"))
    c = {"k": _stored(k, kv, K_SCALE), "v": _stored(v, kv, V_SCALE),
         "table": None if table is None else torch.from_numpy(table).cuda()}
    if own:
        from decode_attention_self_gb300 import api
        c["own"] = api.KVCache(c["k"], c["v"], c["table"], K_SCALE if kv == "e4m3" else 1.0,
                               V_SCALE if kv == "e4m3" else 1.0)
    return c


def _i32(a):
    return torch.as_tensor(np.asarray(a, np.int32), device="cuda")


def _starts(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32)


def prepare(case, seed):
    g = _gen(seed)
    hq, hkv, B = case["hq"], case["hkv"], case["rows"]
    a, b = _lengths(case)
    st = {"case": case, "new": a, "second": b}
    if case["op"] == "rope_append":
        T = max(1, int(a.sum()))
        st["cache"] = _cache(case, a + b, None, g, seed)
        if case["packed"]:
            qkv = _randn((T, (hq + 2 * hkv), D), g)
            st["q"], st["k"], st["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        else:
            st["q"], st["k"], st["v"] = _randn((T, hq, D), g), _randn((T, hkv, D), g), _randn((T, hkv, D), g)
        st["q_out"] = torch.zeros((T, hq, D), dtype=torch.bfloat16, device="cuda")
        st["row_start"], st["start_pos"] = _i32(_starts(a)), _i32(b)
        st["pos_offset"] = _i32([case["offset"]] * B) if case["offset"] else None
        st["table"] = None
        if case["rot"]:
            n = int((a + b).max()) + case["offset"]
            inv = ROPE_BASE ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda") / case["rot"])
            ang = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * inv
            st["table"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        return st
    if case["op"] == "prompt_attn":
        T = int(a.sum())
        st["q"] = _randn((T, hq, D), g)
        st["cache"] = _cache(case, b, b, g, seed)
        st["row_start"], st["kv_len"] = _i32(_starts(a)), _i32(b)
        lo, hi, first, prefix = _intervals(case)
        st["lo"], st["hi"] = _i32(lo), _i32(hi)
        st["first_key"] = _i32(first) if case["mask"] == "document" else None
        st["prefix_len"] = _i32(prefix) if case["mask"] == "prefix" else None
        st["slopes"] = None
        if case["bias"]:
            st["slopes"] = torch.as_tensor([2.0 ** (-8.0 * (i + 1) / hq) for i in range(hq)], dtype=torch.float32,
                                           device="cuda")
        st["out"] = torch.zeros((T, hq, D), dtype=torch.bfloat16, device="cuda")
        if own:
            from decode_attention_self_gb300 import api
            st["max_len"] = int(b.max())
            st["ws"] = torch.empty(api.dr_prompt_attn_workspace(T, B, hq, hkv, st["max_len"]), dtype=torch.uint8,
                                   device="cuda")
        return st
    P = case["prefix"]
    st["q"] = _randn((B, hq, D), g)
    st["prefix"] = _cache(case, [P], [P], g, seed)
    st["cache"] = _cache(case, np.maximum(a, 1), a, g, seed + 1)
    st["prefix_len"], st["seq_len"] = _i32([P]), _i32(a)
    st["out"] = torch.zeros((B, hq, D), dtype=torch.bfloat16, device="cuda")
    if own:
        from decode_attention_self_gb300 import api
        st["ws"] = torch.empty(api.dr_shared_prefix_attn_workspace(B, hq, hkv, P), dtype=torch.uint8, device="cuda")
    return st


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------
def _as_values(t, kv):
    return t if kv == "bf16" else t.view(torch.float8_e4m3fn)


def _rows(cache, b, n, kv, which):
    """Keys (or values) 0..n-1 of row b as [hkv, n, D] float32."""
    pool, scale = (cache["k"], K_SCALE) if which == "k" else (cache["v"], V_SCALE)
    if cache["table"] is None:
        x = pool[b, :, :n]
    else:
        blocks = cache["table"][b, :-(-n // PAGE)].long()
        x = pool[blocks].transpose(0, 1).reshape(pool.shape[1], -1, D)[:, :n]
    return x.float() if kv == "bf16" else x.view(torch.float8_e4m3fn).float() * scale


def _plain_rope_append(st):
    case, cache = st["case"], st["cache"]
    new, start = st["new"], st["second"]
    T, rot, kv = int(new.sum()), case["rot"], case["kv"]
    if T == 0:
        return {"q": st["q_out"], "k": _as_values(cache["k"], kv), "v": _as_values(cache["v"], kv)}
    starts, start_pos = st["row_start"].long(), st["start_pos"].long()
    tok = torch.arange(T, device="cuda")
    row = torch.searchsorted(starts[1:].contiguous(), tok, right=True)
    slot = start_pos[row] + tok - starts[row]
    q, k, v = st["q"][:T].float(), st["k"][:T].float(), st["v"][:T].float()
    if rot:
        pos = slot + (0 if st["pos_offset"] is None else st["pos_offset"].long()[row])
        cs = st["table"][pos]
        cos, sin = cs[:, None, :rot // 2], cs[:, None, rot // 2:]

        def turn(x):
            if case["inter"]:
                x1, x2 = x[..., 0:rot:2], x[..., 1:rot:2]
                y = torch.stack([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1).flatten(-2)
            else:
                x1, x2 = x[..., :rot // 2], x[..., rot // 2:rot]
                y = torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1)
            return torch.cat([y, x[..., rot:]], -1)

        q, k = turn(q), turn(k)
    st["q_out"][:T] = q.to(torch.bfloat16)
    for name, x, scale in (("k", k, K_SCALE), ("v", v, V_SCALE)):
        if kv == "bf16":
            y = x.to(torch.bfloat16)
        else:
            y = (x / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        if cache["table"] is None:
            cache[name][row, :, slot] = y
        else:
            cache[name][cache["table"].long()[row, slot // PAGE], :, slot % PAGE] = y
    return {"q": st["q_out"], "k": _as_values(cache["k"], kv), "v": _as_values(cache["v"], kv)}


def _plain_attend(q, k, v, lo, hi, pos, scale, softcap, slopes):
    """q [n, hq, D], k, v [hkv, L, D] float32; visible keys [lo, hi) per query -> [n, hq, D] float32."""
    n, hq, _ = q.shape
    hkv, L, _ = k.shape
    g = hq // hkv
    out = torch.empty_like(q)
    step = max(1, min(n, (1 << 28) // max(1, hq * L)))
    j = torch.arange(L, device=q.device)
    for i in range(0, n, step):
        m = min(step, n - i)
        qi = q[i:i + m].reshape(m, hkv, g, D).permute(1, 2, 0, 3).reshape(hkv, g * m, D)
        s = (torch.matmul(qi, k.transpose(1, 2)) * scale).view(hkv, g, m, L)
        if softcap:
            s = softcap * torch.tanh(s / softcap)
        if slopes is not None:
            s = s - slopes.view(hkv, g, 1, 1) * (pos[i:i + m, None] - j).abs().float()
        seen = (j >= lo[i:i + m, None]) & (j < hi[i:i + m, None])
        s = s.masked_fill(~seen, float("-inf"))
        top = s.amax(-1, keepdim=True).clamp_min(-3.0e38)
        p = torch.exp(s - top)
        total = p.sum(-1, keepdim=True)
        o = torch.matmul(p.view(hkv, g * m, L), v).view(hkv, g, m, D)
        o = torch.where(total > 0, o / total, torch.zeros_like(o))
        out[i:i + m] = o.permute(2, 0, 1, 3).reshape(m, hq, D)
    return out


def _plain_prompt_attn(st):
    case = st["case"]
    at = 0
    for b, (n, L) in enumerate(zip(st["new"].tolist(), st["second"].tolist())):
        if n == 0:
            continue
        k, v = _rows(st["cache"], b, L, case["kv"], "k"), _rows(st["cache"], b, L, case["kv"], "v")
        pos = torch.arange(L - n, L, device="cuda")
        o = _plain_attend(st["q"][at:at + n].float(), k, v, st["lo"][at:at + n], st["hi"][at:at + n], pos,
                          1.0 / math.sqrt(D), case["softcap"], st["slopes"])
        st["out"][at:at + n] = o.to(torch.bfloat16)
        at += n
    return st["out"]


def _plain_shared_prefix(st):
    case = st["case"]
    P, B, hkv, kv = case["prefix"], case["rows"], case["hkv"], case["kv"]
    q = st["q"].float()
    pk, pv = _rows(st["prefix"], 0, P, kv, "k"), _rows(st["prefix"], 0, P, kv, "v")
    for b, n in enumerate(st["new"].tolist()):
        k = torch.cat([pk, _rows(st["cache"], b, n, kv, "k")], 1) if n else pk
        v = torch.cat([pv, _rows(st["cache"], b, n, kv, "v")], 1) if n else pv
        s = torch.matmul(q[b].view(hkv, -1, D), k.transpose(1, 2)) * (1.0 / math.sqrt(D))
        if case["softcap"]:
            s = case["softcap"] * torch.tanh(s / case["softcap"])
        p = torch.exp(s - s.amax(-1, keepdim=True))
        st["out"][b] = (torch.matmul(p, v) / p.sum(-1, keepdim=True)).view(-1, D).to(torch.bfloat16)
    return st["out"]


def run(st):
    case = st["case"]
    if not own:
        return {"rope_append": _plain_rope_append, "prompt_attn": _plain_prompt_attn,
                "shared_prefix": _plain_shared_prefix}[case["op"]](st)
    from decode_attention_self_gb300 import api
    if case["op"] == "rope_append":
        api.dr_rope_append(st["cache"]["own"], st["k"], st["v"], st["row_start"], st["start_pos"], q=st["q"],
                           q_out=st["q_out"], table=st["table"], interleaved=case["inter"],
                           pos_offset=st["pos_offset"])
        c = st["cache"]
        return {"q": st["q_out"], "k": _as_values(c["k"], case["kv"]), "v": _as_values(c["v"], case["kv"])}
    if case["op"] == "prompt_attn":
        return api.dr_prompt_attn(st["q"], st["cache"]["own"], st["row_start"], st["kv_len"], st["out"],
                                  causal=case["mask"] != "none", softcap=case["softcap"], slopes=st["slopes"],
                                  prefix_len=st["prefix_len"], first_key=st["first_key"],
                                  max_len_hint=st["max_len"], workspace=st["ws"])
    return api.dr_shared_prefix_attn(st["q"], st["prefix"]["own"], st["prefix_len"], st["out"], st["ws"],
                                     cache=st["cache"]["own"], seq_len=st["seq_len"], softcap=case["softcap"],
                                     max_prefix_hint=case["prefix"], max_seq_len_hint=case["own_hi"])


# ---------------------------------------------------------------------------------------------------------------
# exact values, from the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------
def _wide(cache, kv, which):
    """The whole pool as float64 values."""
    if kv == "bf16":
        return cache[which].double()
    return cache[which].view(torch.float8_e4m3fn).double() * (K_SCALE if which == "k" else V_SCALE)


def _key_index(cache, b, n):
    """Where key j of row b lies: (first pool index, third pool index)."""
    j = torch.arange(n, device="cuda")
    if cache["table"] is None:
        return torch.full_like(j, b), j
    return cache["table"][b].long()[j // PAGE], j % PAGE


def _exact_softmax_sum(q, keys, vals, scale, softcap, slope, pos, lo, hi):
    """One head: q [n, D], keys, vals [L, D], all float64; the definition, row block by row block."""
    n, L = q.shape[0], keys.shape[0]
    res = torch.zeros((n, D), dtype=torch.float64, device=q.device)
    j = torch.arange(L, device=q.device, dtype=torch.int64)
    block = max(1, (1 << 26) // max(L, 1))
    for i in range(0, n, block):
        e = min(n, i + block)
        s = q[i:e] @ keys.T * scale
        if softcap:
            s = torch.tanh(s / softcap) * softcap
        if slope is not None:
            s = s - slope * torch.abs(j[None, :] - pos[i:e, None]).double()
        hidden = (j[None, :] < lo[i:e, None]) | (j[None, :] >= hi[i:e, None])
        s[hidden] = -math.inf
        some = ~hidden.all(1)
        if bool(some.any()):
            w = torch.softmax(s[some], dim=1)
            part = res[i:e]
            part[some] = w @ vals
            res[i:e] = part
    return res


def exact(case, seed):
    if work(case)["flops"] > 3.0e12:
        return None
    st = prepare(case, seed)
    new, second = st["new"].tolist(), None if st["second"] is None else st["second"].tolist()
    hq, hkv, kv = case["hq"], case["hkv"], case["kv"]
    g = hq // hkv
    if case["op"] == "rope_append":
        rot = case["rot"]
        cache = st["cache"]
        q_out = st["q_out"].double()
        pools = {w: (cache[w].double() if kv == "bf16" else cache[w].view(torch.float8_e4m3fn).double())
                 for w in ("k", "v")}
        freq = torch.tensor([ROPE_BASE ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64,
                            device="cuda") if rot else None
        first = torch.tensor([(2 * i if case["inter"] else i) for i in range(rot // 2)], dtype=torch.int64,
                             device="cuda")
        other = first + (1 if case["inter"] else rot // 2)
        at = 0
        for b, (n, start) in enumerate(zip(new, second)):
            if n == 0:
                continue
            slots = torch.arange(start, start + n, device="cuda")
            xs = {"q": st["q"][at:at + n].double(), "k": st["k"][at:at + n].double(),
                  "v": st["v"][at:at + n].double()}
            if rot:
                theta = (slots + case["offset"]).double()[:, None, None] * freq
                for w in ("q", "k"):
                    z = torch.complex(xs[w][..., first], xs[w][..., other]) * torch.polar(torch.ones_like(theta), theta)
                    xs[w][..., first], xs[w][..., other] = z.real, z.imag
            q_out[at:at + n] = xs["q"]
            i0, i2 = _key_index(cache, b, start + n)
            i0, i2 = i0[start:], i2[start:]
            for w, scale in (("k", K_SCALE), ("v", V_SCALE)):
                pools[w][i0, :, i2] = xs[w] if kv == "bf16" else (xs[w] / scale).clamp(-448.0, 448.0)
            at += n
        return {"q": q_out, "k": pools["k"], "v": pools["v"]}
    scale = D ** -0.5
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    if case["op"] == "prompt_attn":
        pk, pv = _wide(st["cache"], kv, "k"), _wide(st["cache"], kv, "v")
        at = 0
        for b, (n, L) in enumerate(zip(new, second)):
            if n == 0:
                continue
            i0, i2 = _key_index(st["cache"], b, L)
            pos = torch.arange(L - n, L, device="cuda")
            for h in range(hq):
                slope = None if st["slopes"] is None else st["slopes"][h].double()
                out[at:at + n, h] = _exact_softmax_sum(st["q"][at:at + n, h].double(), pk[i0, h // g, i2],
                                                       pv[i0, h // g, i2], scale, case["softcap"], slope, pos,
                                                       st["lo"][at:at + n].long(), st["hi"][at:at + n].long())
            at += n
        return out
    P, B = case["prefix"], case["rows"]
    i0, i2 = _key_index(st["prefix"], 0, P)
    k0, v0 = (_wide(st["prefix"], kv, w).transpose(0, 1)[:, i0, i2] for w in ("k", "v"))
    pools = [_wide(st["cache"], kv, w).transpose(0, 1) for w in ("k", "v")]
    for b, n in enumerate(new):
        i0, i2 = _key_index(st["cache"], b, n)
        keys = torch.cat([k0, pools[0][:, i0, i2]], 1).repeat_interleave(g, 0)
        vals = torch.cat([v0, pools[1][:, i0, i2]], 1).repeat_interleave(g, 0)
        s = (st["q"][b].double()[:, None, :] * keys).sum(-1) * scale
        if case["softcap"]:
            s = torch.tanh(s / case["softcap"]) * case["softcap"]
        out[b] = (torch.softmax(s, 1)[:, :, None] * vals).sum(1)
    return out
