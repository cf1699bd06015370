"""A whole layer from the library's calls, near enough to its reference that no bias or norm weight could be missing.

Bound: a rounding to bf16 is off by 2^-7 / sqrt(12) / m in the root mean square, m in [1, 2) spread over its logarithm (E[1 / m^2] = 0.541),
1.66e-3 of the value.  Eight quantities are rounded on the way (both norms' outputs, q/k/v, rotated q and k, softmax weights, attention's
output, the MLP's middle), on either side, from values that differ in the last bits: were all sixteen apart from one another,
sqrt(16) * 1.66e-3.  Leaving out any one bias or norm weight moves the outputs by 1.2 % at the least (in the reference, in 64 bits).
"""
import pytest
import torch

from test_gpu_layer_calls import BF16, DM, EPS, FF, HKV, HQ, D, Layer64, rel, weights

pytestmark = pytest.mark.gpu
BOUND = 4 * 1.66e-3


@pytest.fixture(scope="module")
def api(cuda_device):
    from decode_attention_self_gb300 import api as _api

    return _api


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("lens", [(7,), (40, 1, 300), (600, 900)])
def test_every_part_of_a_layer_counts(api, gated, lens):
    w = weights(gated)
    B, T, cap = len(lens), sum(lens), 1024
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    cache = api.KVCache(torch.zeros((B, HKV, cap, D), dtype=BF16, device="cuda"), torch.zeros((B, HKV, cap, D), dtype=BF16, device="cuda"))
    table = api.dr_rope_table(torch.empty((cap, D), device="cuda"))
    n1, n2 = api.Norm("layer", EPS, w["n1w"], w["n1b"]), api.Norm("layer", EPS, w["n2w"], w["n2b"])
    ws = torch.empty(max(1, api.dr_prompt_attn_workspace(T, B, HQ, HKV, cap)), dtype=torch.uint8, device="cuda")

    def layer(h, row_start, start_pos, kv_len):
        n = h.shape[0]
        e = lambda *s: torch.empty(s, dtype=BF16, device="cuda")
        x, q, k, v, a, u = e(n, DM), e(n, HQ * D), e(n, HKV * D), e(n, HKV * D), e(n, HQ, D), e(n, FF)
        api.dr_residual_norm(h, y=x, pre=n1)
        api.dr_linear(x, w["qkv"], [q, k, v])
        q, k, v = q.view(n, HQ, D), k.view(n, HKV, D), v.view(n, HKV, D)
        api.dr_rope_append(cache, k, v, row_start, start_pos, q=q, q_out=q, table=table)
        api.dr_prompt_attn(q, cache, row_start, kv_len, a, workspace=ws)
        api.dr_linear(a.view(n, HQ * D), w["o"], h, residual=h)
        api.dr_residual_norm(h, y=x, pre=n2)
        api.dr_linear(x, w["up"], u, bias=w["up_b"], act="silu" if gated else "gelu", gated=gated)
        api.dr_linear(u, w["down"], h, bias=w["down_b"], residual=h)
        return h

    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    prompt = torch.randn((T, DM), generator=torch.Generator().manual_seed(7)).cuda()
    step = torch.randn((B, DM), generator=torch.Generator().manual_seed(100)).cuda()

    def reference(w):
        rows = [Layer64(w, gated) for _ in lens]
        return (torch.cat([r(prompt[a:b].double()) for r, a, b in zip(rows, starts, starts[1:])]),
                torch.cat([r(step[j:j + 1].double()) for j, r in enumerate(rows)]))

    got = (layer(prompt.clone(), i32(starts), i32([0] * B), i32(list(lens))),
           layer(step.clone(), i32(list(range(B + 1))), i32(list(lens)), i32([n + 1 for n in lens])))
    for g, ref in zip(got, reference(w)):
        assert rel(g, ref) <= BOUND
    for name in w:
        without = dict(w)
        without[name] = torch.ones_like(w[name]) if name in ("n1w", "n2w") else torch.zeros_like(w[name])
        for g, ref in zip(got, reference(without)):
            assert rel(g, ref) > BOUND, name
