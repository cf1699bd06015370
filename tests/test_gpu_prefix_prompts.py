"""GPU check of a serving loop in which every row's prompt attends the shared prefix and itself: the prefix's blocks stand at
the head of each row's block table for the prompts, and apart from it for the single tokens that follow."""
import pytest
import torch

from decode_attention_self_gb300 import workloads as W
from prompt_reference import PAGE, Cache, D, assert_close, attend, starts

pytestmark = pytest.mark.gpu


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("P", [16, 80, 304])
def test_prompts_behind_a_shared_prefix(cuda_device, fp8, P):
    """Prefix, prompts and two steps; outputs are compared with 64-bit attention over prefix and own keys, position by
    position, and with a loop that holds everything in rows of their own."""
    from decode_attention_self_gb300 import api

    dev, Hq, Hkv, steps = cuda_device, 8, 2, 2
    prompts = [9, 33, 1, 20, 140]
    B, head = len(prompts), P // PAGE
    # row 0 of one pool is the prefix, rows 1.. the rows' own keys
    pool = Cache([P] + [n + steps for n in prompts], Hkv, True, fp8, 50, valid=[0] * (B + 1))
    apart = Cache([P + n + steps for n in prompts], Hkv, True, fp8, 51, valid=[0] * B)
    shared, own = pool.gpu(api, dev), apart.gpu(api, dev)
    width = pool.table.shape[1]
    pre = api.KVCache(shared.k, shared.v, pool.table[:1, :head].contiguous().to(dev), shared.k_scale, shared.v_scale)
    rows = api.KVCache(shared.k, shared.v, pool.table[1:].contiguous().to(dev), shared.k_scale, shared.v_scale)
    whole = api.KVCache(shared.k, shared.v, torch.cat([pool.table[:1, :head].expand(B, head), pool.table[1:]], 1).to(dev),
                        shared.k_scale, shared.v_scale)
    assert whole.block_table.shape == (B, head + width)
    table = torch.empty((512, 64), dtype=torch.float32, device=dev)
    api.dr_rope_table(table)
    err = i32([0], dev)

    def project(T, key):
        x = W.randn_bf16((T, Hq + 2 * Hkv, D), dev, 60, key)
        return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]

    def keys(b, n):
        """Prefix and the first n own keys of row b, from the pool."""
        pool.k, pool.v = shared.k.cpu(), shared.v.cpu()
        return (torch.cat(x, 1) for x in zip(pool.rows(0, P), pool.rows(1 + b, n)))

    # the prefix, once in the pool and once in every row of the other cache
    q, k, v = project(P, 1)
    qr, out = torch.empty((P, Hq, D), dtype=torch.bfloat16, device=dev), torch.empty((P, Hq, D), device=dev)
    api.dr_rope_append(pre, k, v, i32([0, P], dev), i32([0], dev), q=q, q_out=qr, table=table, err_flag=err)
    api.dr_prompt_attn(qr, pre, i32([0, P], dev), i32([P], dev), out, prefix_len=i32([P], dev), err_flag=err)
    api.dr_rope_append(own, k.repeat(B, 1, 1), v.repeat(B, 1, 1), starts([P] * B).to(dev), i32([0] * B, dev), table=table,
                       err_flag=err)

    # prompts: behind the prefix in rows that begin with its blocks
    T, rs = sum(prompts), starts(prompts).to(dev)
    q, k, v = project(T, 2)
    outs = []
    for cache in (whole, own):
        qr, out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=dev), torch.empty((T, Hq, D), device=dev)
        api.dr_rope_append(cache, k, v, rs, i32([P] * B, dev), q=q, q_out=qr, table=table, err_flag=err)
        api.dr_prompt_attn(qr, cache, rs, i32([P + n for n in prompts], dev), out, err_flag=err)
        outs.append(out)
    assert torch.equal(*outs)
    at = 0
    for b, n in enumerate(prompts):
        ref, tol = attend(qr[at:at + n].cpu(), *keys(b, n), torch.zeros(n, dtype=torch.long),
                          torch.arange(P + 1, P + n + 1), torch.arange(P, P + n), fp8=fp8)
        assert_close(out[at:at + n], ref, tol, f"prompt {b}")
        at += n

    # single tokens: the prefix read once for all rows, the rows' own keys from their own tables
    ws = torch.empty(api.dr_shared_prefix_attn_workspace(B, Hq, Hkv, P), dtype=torch.uint8, device=dev)
    one = starts([1] * B).to(dev)
    for i in range(steps):
        q, k, v = project(B, 3 + i)
        qr, out = torch.empty((B, Hq, D), dtype=torch.bfloat16, device=dev), torch.empty((B, Hq, D), device=dev)
        api.dr_rope_append(rows, k, v, one, i32([n + i for n in prompts], dev), q=q, q_out=qr, table=table,
                           pos_offset=i32([P] * B, dev), err_flag=err)
        api.dr_shared_prefix_attn(qr, pre, i32([P], dev), out, ws, cache=rows,
                                  seq_len=i32([n + i + 1 for n in prompts], dev), err_flag=err)
        for b, n in enumerate(prompts):
            L = P + n + i + 1
            ref, tol = attend(qr[b:b + 1].cpu(), *keys(b, n + i + 1), torch.zeros(1, dtype=torch.long), torch.tensor([L]),
                              torch.tensor([L - 1]), fp8=fp8)
            assert_close(out[b:b + 1], ref, tol, f"step {i}, row {b}")
    assert int(err.item()) == 0
