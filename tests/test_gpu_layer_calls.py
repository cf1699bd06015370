"""The layer calls together, as they are used: a decoder layer's prompt and then its single-token steps, from the norm before the
attention to the MLP's residual, with only calls of the library on the device; the steps also captured in a graph.

The reference is the same layer in float64, rounded to bf16 where the layer hands bf16 on.  Bound: every quantity handed on is
rounded to bf16 on both sides from values that differ by fp32 arithmetic, so a rounding may fall the other way; such a flip is one
bf16 step (2^-7 of a value of order 1) in a few of the elements, spread over sums of hundreds of terms with weights of K^-0.5.
What is compared is the relative error of whole outputs: each of the eight roundings of the chain adds at most a relative
2^-8 in the norm on either side, 16 * 2^-8 together if none of them cancels, and far less as they are independent."""
import math

import pytest
import torch

from layer_reference import act64

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
D, HQ, HKV, DM, FF = 64, 16, 4, 1024, 4096
EPS = 1e-5


@pytest.fixture(scope="module")
def api(cuda_device):
    from decode_attention_self_gb300 import api as _api

    return _api


def randn(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(BF16).cuda()


def weights(gated):
    w = {"qkv": randn(((HQ + 2 * HKV) * D, DM), 1, DM ** -0.5), "o": randn((DM, HQ * D), 2, DM ** -0.5),
         "up": randn((FF * (2 if gated else 1), DM), 3, DM ** -0.5), "down": randn((DM, FF), 4, FF ** -0.5)}
    w["up_b"], w["down_b"] = randn((w["up"].shape[0],), 5, 0.1), randn((DM,), 6, 0.1)
    for i, n in enumerate(("n1", "n2")):
        w[n + "w"], w[n + "b"] = 1 + randn((DM,), 10 + i, 0.1), randn((DM,), 20 + i, 0.1)
    return w


def b16(t):
    return t.to(BF16).double()


def norm64(x, w, b):
    c = x - x.mean(1, keepdim=True)
    return c / torch.sqrt((c * c).mean(1, keepdim=True) + EPS) * w.double() + b.double()


def rotate64(x, pos):
    inv = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
    a = pos.double()[:, None, None] * inv
    x1, x2 = x[..., :D // 2], x[..., D // 2:]
    return torch.cat([x1 * a.cos() - x2 * a.sin(), x2 * a.cos() + x1 * a.sin()], -1)


class Layer64:
    """One row's layer in float64 with its keys and values kept; bf16 where the library's calls hand bf16 on."""

    def __init__(self, w, gated):
        self.w, self.gated, self.k, self.v = w, gated, None, None

    def __call__(self, h):
        w, T = self.w, h.shape[0]
        qkv = b16(b16(norm64(h, w["n1w"], w["n1b"])) @ w["qkv"].double().T).view(T, -1, D)
        past = 0 if self.k is None else self.k.shape[0]
        pos = torch.arange(past, past + T, device="cuda")
        q, k = b16(rotate64(qkv[:, :HQ], pos)), b16(rotate64(qkv[:, HQ:HQ + HKV], pos))
        v = qkv[:, HQ + HKV:]
        self.k = k if past == 0 else torch.cat([self.k, k])
        self.v = v if past == 0 else torch.cat([self.v, v])
        ks, vs = self.k.repeat_interleave(HQ // HKV, 1), self.v.repeat_interleave(HQ // HKV, 1)
        s = torch.einsum("thd,khd->htk", q, ks) / math.sqrt(D)
        s = s.masked_fill(torch.arange(past + T, device="cuda")[None, None, :] > pos[None, :, None], -math.inf)
        a = b16(torch.einsum("htk,khd->thd", torch.softmax(s, -1), vs)).reshape(T, -1)
        h = h + a @ w["o"].double().T
        z = b16(norm64(h, w["n2w"], w["n2b"])) @ w["up"].double().T + w["up_b"].double()
        u = act64(z[:, :FF], "silu") * z[:, FF:] if self.gated else act64(z, "gelu")
        return h + b16(u) @ w["down"].double().T + w["down_b"].double()


def rel(got, ref):
    return ((got.double() - ref).norm() / ref.norm()).item()


BOUND = 16 * 2.0 ** -8


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("lens", [(7,), (40, 1, 300), (600, 900)])
def test_prompts_and_steps(api, gated, lens):
    w = weights(gated)
    B, T, cap = len(lens), sum(lens), 1024
    cache = api.KVCache(torch.zeros((B, HKV, cap, D), dtype=BF16, device="cuda"), torch.zeros((B, HKV, cap, D), dtype=BF16, device="cuda"))
    table = api.dr_rope_table(torch.empty((cap, D), device="cuda"))
    n1, n2 = api.Norm("layer", EPS, w["n1w"], w["n1b"]), api.Norm("layer", EPS, w["n2w"], w["n2b"])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")

    def buffers(n):
        e = lambda *s: torch.empty(s, dtype=BF16, device="cuda")
        return {"x": e(n, DM), "q": e(n, HQ * D), "k": e(n, HKV * D), "v": e(n, HKV * D), "a": e(n, HQ, D), "u": e(n, FF)}

    def layer(h, b, row_start, start_pos, kv_len, ws):
        n = h.shape[0]
        api.dr_residual_norm(h, y=b["x"], pre=n1)
        api.dr_linear(b["x"], w["qkv"], [b["q"], b["k"], b["v"]], err_flag=err)
        q, k, v = b["q"].view(n, HQ, D), b["k"].view(n, HKV, D), b["v"].view(n, HKV, D)
        api.dr_rope_append(cache, k, v, row_start, start_pos, q=q, q_out=q, table=table, err_flag=err)
        api.dr_prompt_attn(q, cache, row_start, kv_len, b["a"], workspace=ws, err_flag=err)
        api.dr_linear(b["a"].view(n, HQ * D), w["o"], h, residual=h, err_flag=err)          # the fp32 stream in place
        api.dr_residual_norm(h, y=b["x"], pre=n2)
        api.dr_linear(b["x"], w["up"], b["u"], bias=w["up_b"], act="silu" if gated else "gelu", gated=gated, err_flag=err)
        api.dr_linear(b["u"], w["down"], h, bias=w["down_b"], residual=h, err_flag=err)

    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    h0 = torch.randn((T, DM), generator=torch.Generator().manual_seed(7)).cuda()
    refs = [Layer64(w, gated) for _ in lens]
    want = torch.cat([r(h0[a:b].double()) for r, a, b in zip(refs, starts, starts[1:])])
    h = h0.clone()
    ws = torch.empty(max(1, api.dr_prompt_attn_workspace(T, B, HQ, HKV, cap)), dtype=torch.uint8, device="cuda")
    layer(h, buffers(T), i32(starts), i32([0] * B), i32(list(lens)), ws)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert rel(h, want) <= BOUND

    # single tokens: the same buffers each step, the second and later steps replayed from a graph
    step, b = torch.empty((B, DM), device="cuda"), buffers(B)
    pos, length, one_each = i32(list(lens)), i32([n + 1 for n in lens]), i32(list(range(B + 1)))

    def one_step():
        layer(step, b, one_each, pos, length, None)
        pos.add_(1)
        length.add_(1)

    graph = None
    for i in range(4):
        x = torch.randn((B, DM), generator=torch.Generator().manual_seed(100 + i)).cuda()
        step.copy_(x)
        if i == 0:
            one_step()
        else:
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    one_step()
            graph.replay()
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        want = torch.cat([r(x[j:j + 1].double()) for j, r in enumerate(refs)])
        assert rel(step, want) <= BOUND, i


def test_norm_and_product_are_one_quantity_from_either_call(api):
    # the residual added in the product's epilogue, or by the norm call that follows: the same fp32 stream, bit for bit
    T = 50
    x, W, b, r = randn((T, 512), 1), randn((DM, 512), 2, 512 ** -0.5), randn((DM,), 3), torch.randn((T, DM), device="cuda")
    a, h = torch.empty((T, DM), device="cuda"), torch.empty((T, DM), device="cuda")
    api.dr_linear(x, W, a, bias=b, residual=r)
    v = torch.empty((T, DM), device="cuda")
    api.dr_linear(x, W, v, bias=b)
    api.dr_residual_norm(v, residual=r, h=h)
    assert torch.equal(a, h)
