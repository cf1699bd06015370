"""dr_linear against the float64 product, over sizes, epilogues, layouts and what may stand in the inputs."""
import numpy as np
import pytest
import torch

from layer_reference import assert_within, half_step, linear64

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def api(cuda_device):
    from decode_attention_self_gb300 import api as _api

    return _api


def randn(shape, seed, scale=1.0, dtype=BF16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def problem(T, K, N, act=None, gated=False, bias=True, residual=False, out=BF16, seed=0):
    rows = 2 * N if gated else N
    x, W = randn((T, K), seed + 1), randn((rows, K), seed + 2, K ** -0.5)
    b = randn((rows,), seed + 3, 0.5) if bias else None
    r = randn((T, N), seed + 4, 1.0, out) if residual else None
    ref, tol = linear64(x, W, b, act, gated, r, out)
    cuda = [None if t is None else t.cuda() for t in (x, W, b, r)]
    return cuda, ref, tol


def run_and_check(api, T, K, N, act=None, gated=False, bias=True, residual=False, out=BF16, seed=0):
    (x, W, b, r), ref, tol = problem(T, K, N, act, gated, bias, residual, out, seed)
    o = torch.full((T, N), float("nan"), dtype=out, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.dr_linear(x, W, o, bias=b, act=act, gated=gated, residual=r, err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert_within(o, ref, tol, f"T={T} K={K} N={N} {act} gated={gated} residual={residual} {out}")


TOKENS = [1, 2, 3, 7, 8, 9, 15, 16, 17, 24, 31, 32, 33, 48, 63, 64, 65, 100, 127, 128, 129, 200, 255, 256, 257, 300, 513, 700,
          1030, 2700]


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("out", [BF16, F32])
def test_token_counts(api, T, out):
    run_and_check(api, T, 1024, 1024, "gelu", bias=True, residual=True, out=out, seed=T)


@pytest.mark.parametrize("T", [1, 5, 17, 30, 64, 130, 400, 2100, 19600])
@pytest.mark.parametrize("K,N", [(8, 1), (8, 64), (16, 7), (24, 9), (56, 63), (64, 8), (72, 65), (128, 100), (200, 127),
                                 (264, 129), (1000, 1089), (520, 257), (64, 2048)])
def test_odd_sizes(api, T, K, N):
    run_and_check(api, T, K, N, "silu", bias=True, out=BF16 if (T + N) % 2 else F32, seed=T + K)


@pytest.mark.parametrize("T", [1, 11, 27, 70, 500, 19600])
@pytest.mark.parametrize("N", [1, 7, 33, 63, 65, 129])
def test_odd_gated_sizes(api, T, N):
    run_and_check(api, T, 104, N, "gelu_tanh", gated=True, residual=True, out=F32 if (T + N) % 3 else BF16, seed=T + N)


@pytest.mark.parametrize("T", [1, 4, 20, 96, 128, 384])
@pytest.mark.parametrize("K,N", [(2048, 1536), (4096, 1024), (1024, 4096), (8192, 512), (6144, 64), (16384, 128)])
def test_model_sizes(api, T, K, N):
    run_and_check(api, T, K, N, "none", bias=False, residual=True, out=F32 if K > 4096 else BF16, seed=T)


@pytest.mark.parametrize("T,K,N", [(1024, 512, 512), (1500, 1024, 2048), (4099, 256, 1000), (3000, 2048, 600),
                                   (8192, 192, 512), (2304, 1024, 4096)])
@pytest.mark.parametrize("out,act,gated,residual", [(BF16, "gelu", False, False), (F32, None, False, True),
                                                    (BF16, "silu", True, False), (F32, "gelu_tanh", True, True),
                                                    (BF16, None, False, True)])
def test_prompt_sizes(api, T, K, N, out, act, gated, residual):
    run_and_check(api, T, K, N, act, gated=gated, residual=residual, out=out, seed=T)


@pytest.mark.parametrize("act", [None, "none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T", [3, 14, 25, 40, 1300, 5000])
def test_activations(api, act, gated, T):
    for bias, residual, out in ((True, True, F32), (False, False, BF16)):
        run_and_check(api, T, 320, 200, act, gated, bias, residual, out, seed=T)


@pytest.mark.parametrize("T", [1, 6, 20, 33, 150, 1500, 5000])
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("pad", [1, 3, 8, 64])
def test_slices_and_places(api, T, out, pad):
    # x, residual and output as slices of wider buffers, at strides that are and are not multiples of 16 bytes; what
    # stands around the output stays
    K, N = 264, 200
    (x, W, b, r), ref, tol = problem(T, K, N, "gelu", False, True, True, out, seed=T)
    xb = torch.full((T, K + 72), float("nan"), dtype=BF16, device="cuda")
    xb[:, 8:8 + K] = x
    rb = torch.full((T, N + pad + 5), float("nan"), dtype=out, device="cuda")
    rb[:, pad:pad + N] = r
    ob = torch.full((T + 2, N + 2 * pad), 7.0, dtype=out, device="cuda")
    o = ob[1:T + 1, pad:pad + N]
    api.dr_linear(xb[:, 8:8 + K], W, o, bias=b, act="gelu", residual=rb[:, pad:pad + N])
    torch.cuda.synchronize()
    assert_within(o, ref, tol, "slices")
    around = ob.clone()
    around[1:T + 1, pad:pad + N] = 7.0
    assert (around == 7.0).all()


@pytest.mark.parametrize("T", [1, 12, 31, 90, 1400, 6000])
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("widths", [(64,), (128, 64, 64), (64, 192, 64, 9), (1024, 256, 256), (320, 1), (64, 64, 64, 64)])
def test_outputs_share_the_columns(api, T, out, widths):
    N = sum(widths)
    (x, W, b, _), ref, tol = problem(T, 256, N, None, False, True, False, out, seed=N)
    outs = [torch.full((T, w), float("nan"), dtype=out, device="cuda") for w in widths]
    got = api.dr_linear(x, W, outs, bias=b)
    torch.cuda.synchronize()
    assert got is outs
    at = 0
    for o, w in zip(outs, widths):
        assert_within(o, ref[:, at:at + w], tol[:, at:at + w], f"output at {at}")
        at += w


@pytest.mark.parametrize("T", [1, 10, 29, 70, 300, 2000, 5000])
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("N", [512, 509])
def test_residual_in_place(api, T, out, N):
    (x, W, b, r), ref, tol = problem(T, 256, N, None, False, True, True, out, seed=T)
    assert api.dr_linear(x, W, r, bias=b, residual=r) is r
    torch.cuda.synchronize()
    assert_within(r, ref, tol, "in place")


@pytest.mark.parametrize("T,N", [(1, 256), (16, 256), (30, 256), (100, 256), (1000, 256), (1000, 1024), (5000, 256)])
def test_fp32_outputs_keep_long_sums(api, T, N):
    # A chain of tensor-core additions over K = 8192 drifts by 8e-6 of the value.  Broken every 512 of K it loses at most
    # one bit of the partial sum at each of 32 additions, two thirds of the value on average: 32 * 2/3 * 2^-23.
    x, W = randn((T, 8192), 1), randn((N, 8192), 2, 8192 ** -0.5)
    o = torch.empty((T, N), dtype=F32, device="cuda")
    api.dr_linear(x.cuda(), W.cuda(), o)
    ref = x.double() @ W.double().T
    assert ((o.double().cpu() - ref).norm() / ref.norm()).item() <= 32 * 2 / 3 * 2.0 ** -23


@pytest.mark.parametrize("T", [1, 9, 18, 65, 260, 1800, 7000])
@pytest.mark.parametrize("gated", [False, True])
def test_nan_and_infinity_stay_in_their_rows_and_columns(api, T, gated):
    K, N = 200, 130
    (x, W, b, r), ref, tol = problem(T, K, N, "silu" if gated else None, gated, True, True, F32, seed=5)
    t, n = T // 2, 77
    x2, W2, r2 = x.clone(), W.clone(), r.clone()
    x2[t, 3] = float("nan")
    W2[n, 5] = float("inf")
    r2[0, 1] = float("-inf")
    o = torch.empty((T, N), dtype=F32, device="cuda")
    api.dr_linear(x2, W2, o, bias=b, act="silu" if gated else None, gated=gated, residual=r2)
    o = o.cpu()
    assert o[t].isnan().all()
    assert not (o[:, n].isfinite()).any() if not gated else o[t, n].isnan()
    keep = torch.ones((T, N), dtype=torch.bool)
    keep[t], keep[:, n], keep[0, 1] = False, False, False
    assert_within(torch.where(keep, o, ref.float()), ref, tol + 1e-6 * ref.abs(), "the others")
    if t != 0:
        assert o[0, 1] == float("-inf")


@pytest.mark.parametrize("act,at_minus", [("relu", 0.0), ("gelu", 0.0), ("gelu_tanh", 0.0), ("silu", 0.0), (None, -np.inf)])
@pytest.mark.parametrize("T", [2, 24, 50, 1200, 19600])
def test_activations_at_the_ends(api, act, at_minus, T):
    # sums of exactly one product: +-inf, the largest and smallest bf16, signed zeros
    vals = torch.tensor([np.inf, -np.inf, 3e38, -3e38, 1e-38, -1e-38, 0.0, -0.0, 30.0, -30.0, 100.0, -100.0], dtype=BF16)
    K = 64
    x = torch.zeros((T, K), dtype=BF16)
    x[:, 0] = 1.0
    W = torch.zeros((vals.numel(), K), dtype=BF16)
    W[:, 0] = vals
    o = torch.empty((T, vals.numel()), dtype=F32, device="cuda")
    api.dr_linear(x.cuda(), W.cuda(), o, act=act)
    o = o.cpu()
    v = vals.double()
    from layer_reference import act64
    want = act64(v, act)
    want[1] = at_minus
    for i in range(vals.numel()):
        w = want[i].item()
        if np.isnan(w):       # a large negative argument whose exponential overflows in the plain form only
            w = 0.0
        if np.isinf(w):
            assert (o[:, i] == w).all(), (act, vals[i], o[:, i])
        else:
            # denormal arguments may be flushed
            assert ((o[:, i].double() - w).abs() <= 5e-7 + 2.0 ** -21 * abs(w)).all(), (act, vals[i], o[:, i], w)


def test_same_bits_from_call_to_call_on_two_streams_and_in_a_graph(api):
    s2 = torch.cuda.Stream()
    for T, K, N, out in ((1, 1024, 1024, BF16), (40, 2048, 512, F32), (128, 4096, 1024, BF16), (1500, 1024, 512, F32), (5000, 1024, 512, BF16),
                         (30, 1024, 512, BF16)):
        (x, W, b, r), ref, tol = problem(T, K, N, "gelu", False, True, True, out, seed=T)
        first = torch.empty((T, N), dtype=out, device="cuda")
        api.dr_linear(x, W, first, bias=b, act="gelu", residual=r)
        torch.cuda.synchronize()
        assert_within(first, ref, tol, "first")
        outs = [torch.empty_like(first) for _ in range(40)]
        for i, o in enumerate(outs):
            api.dr_linear(x, W, o, bias=b, act="gelu", residual=r, stream=s2 if i % 2 else None)
        torch.cuda.synchronize()
        assert all(torch.equal(o, first) for o in outs)
        o = torch.zeros_like(first)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            api.dr_linear(x, W, o, bias=b, act="gelu", residual=r)
            api.dr_linear(x, W, o, bias=b, act="gelu", residual=r)
        for _ in range(3):
            o.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, first)


def test_first_calls_of_a_process_in_a_capture():
    # what a kernel sets up once is set up during the capture
    import os
    import subprocess
    import sys

    code = """
import sys, torch
from decode_attention_self_gb300 import api
T, K, N = map(int, sys.argv[1:])
x = torch.randn(T, K, device='cuda').bfloat16()
W = (torch.randn(N, K, device='cuda') / K ** 0.5).bfloat16()
o, y = torch.zeros(T, N, device='cuda', dtype=torch.bfloat16), torch.zeros(T, N, device='cuda', dtype=torch.bfloat16)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    api.dr_linear(x, W, o)
    api.dr_residual_norm(o, y=y, pre=api.Norm('rms'))
g.replay()
torch.cuda.synchronize()
ref = x.double() @ W.double().T
assert ((o.double() - ref).norm() / ref.norm()).item() < 2 ** -8
ref = o.double() / (o.double() ** 2).mean(1, keepdim=True).add(1e-5).sqrt()
assert ((y.double() - ref).norm() / ref.norm()).item() < 2 ** -7
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    for size in ("4 512 512", "28 512 512", "200 2048 512", "2000 512 1024", "4000 512 1024"):
        subprocess.run([sys.executable, "-c", code, *size.split()], check=True, cwd=root, timeout=300)


def test_kernels_side_by_side_on_four_streams(api):
    # products of every kind, the LM head and a prompt's attention share the SMs and their tensor memory
    B, H, L = 2, 16, 700
    q = randn((B * L, H, 64), 50).cuda()
    cache = api.KVCache(randn((B, H, 1024, 64), 51).cuda(), randn((B, H, 1024, 64), 52).cuda())
    rs = torch.tensor([0, L, 2 * L], dtype=torch.int32, device="cuda")
    kl = torch.tensor([L, L], dtype=torch.int32, device="cuda")
    hid, head = randn((16, 1024), 53).cuda(), randn((9 * 1088, 1024), 54, 0.03).cuda()
    jobs = []
    for T, K, N, out in ((2600, 1024, 1024, BF16), (128, 4096, 1024, BF16), (700, 2048, 512, F32), (20, 1024, 1024, BF16),
                         (2000, 1024, 1024, BF16), (1200, 256, 1024, BF16)):
        x, W = randn((T, K), T).cuda(), randn((N, K), T + 1, K ** -0.5).cuda()
        jobs.append((lambda s, o, x=x, W=W: api.dr_linear(x, W, o, act="gelu", stream=s), (T, N), out))
    jobs.append((lambda s, o: api.dr_lm_head(hid, head, 9, o, stream=s), (16, 9, 1088), F32))
    jobs.append((lambda s, o: api.dr_prompt_attn(q, cache, rs, kl, o, stream=s), (B * L, H, 64), BF16))
    want = []
    for call, shape, dt in jobs:
        o = torch.empty(shape, dtype=dt, device="cuda")
        call(None, o)
        want.append(o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    rng = np.random.default_rng(0)
    runs = []
    for i in range(400):
        j = int(rng.integers(len(jobs)))
        call, shape, dt = jobs[j]
        s = streams[int(rng.integers(4))]
        with torch.cuda.stream(s):
            o = torch.empty(shape, dtype=dt, device="cuda")
        call(s, o)
        runs.append((j, o))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[j]) for j, o in runs)


def test_a_chain_of_products_reads_what_the_one_before_wrote(api):
    # launches overlap their predecessors' ends; each must still see all of its predecessor's output
    for T in (1, 24, 128, 1100, 3000, 4500):
        Ws = [randn((512, 512), 10 + i, 512 ** -0.5).cuda() for i in range(6)]
        x = randn((T, 512), 3).cuda()
        bufs = [torch.empty((T, 512), dtype=BF16, device="cuda") for _ in Ws]
        for _ in range(20):
            cur = x
            for W, o in zip(Ws, bufs):
                o.fill_(float("nan"))
            for W, o in zip(Ws, bufs):
                api.dr_linear(cur, W, o)
                cur = o
            torch.cuda.synchronize()
            cur = x
            for W, o in zip(Ws, bufs):
                ref, tol = linear64(cur, W, None, None, False, None, BF16)
                assert_within(o, ref, tol, f"chain T={T}")
                cur = o
            x = bufs[-1].clone()


def test_many_tokens_pass_32_bit_offsets(api):
    # 2^31 elements of output and more: the last rows and the first are right
    T, K, N = 1_050_000, 64, 2112
    x = torch.randn((T, K), device="cuda").to(BF16)
    W = randn((N, K), 1, 0.125)
    o = torch.empty((T, N), dtype=BF16, device="cuda")
    api.dr_linear(x, W.cuda(), o, act="relu")
    rows = torch.tensor([0, 1, 127, 128, 70000, 1_016_800, T - 130, T - 2, T - 1])
    ref, tol = linear64(x[rows.cuda()], W, None, "relu", False, None, BF16)
    assert_within(o[rows.cuda()], ref, tol, "far rows")
    del o
    # and of input
    T, K, N = 70_000, 64, 72
    wide = torch.empty((T, 32768), dtype=BF16, device="cuda")
    x = wide[:, 32000:32064]
    x.normal_()
    o = torch.empty((T, N), dtype=F32, device="cuda")
    W = randn((N, K), 2, 0.125)
    api.dr_linear(x, W.cuda(), o)
    rows = torch.tensor([0, 65535, 65537, T - 1])
    ref, tol = linear64(x[rows.cuda()], W, None, None, False, None, F32)
    assert_within(o[rows.cuda()], ref, tol, "far inputs")


@pytest.mark.parametrize("T,K,N", [(64, 1024, 512), (128, 4096, 256), (600, 512, 512), (2500, 512, 512), (6000, 576, 1024)])
def test_wait_that_runs_out(api, T, K, N):
    # Test hook: one output tile's CTAs never load their first K chunk; their waits give up after about 2 s, the tile is
    # left as it was, others are right, and the next call on the same context is right everywhere.
    (x, W, b, _), ref, tol = problem(T, K, N, None, False, True, False, F32, seed=T)
    o = torch.full((T, N), float("nan"), dtype=F32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.dr_linear_stall_test(1, x, W, o, bias=b, err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) & api.DR_ERRF_TIMEOUT
    got = o.cpu()
    hole = got.isnan()
    assert hole.any() and not hole.all()
    assert_within(torch.where(hole, ref.float(), got), ref, tol + half_step(F32) * ref.abs(), "tiles that ran")
    err.zero_()
    api.dr_linear(x, W, o, bias=b, err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert_within(o, ref, tol, "the call after")


# Tiles of 256 tokens by 128 weight rows, one for each pair of CTAs: bf16 outputs, more than a wave of smaller tiles, no more
# than a wave of these.
PAIRED = [(130, 64, 9600), (257, 8, 4000), (1900, 72, 1089), (2000, 1000, 1088), (1400, 1024, 1536), (512, 4096, 2560),
          (1025, 520, 1800), (2048, 320, 1024), (4600, 2048, 500)]


@pytest.mark.parametrize("T,K,N", PAIRED)
@pytest.mark.parametrize("act,gated,bias,residual", [(None, False, False, False), ("gelu", False, True, True), ("silu", True, True, False),
                                                     ("relu", True, False, True)])
def test_paired_sizes(api, T, K, N, act, gated, bias, residual):
    run_and_check(api, T, K, N // 2 if gated else N, act, gated, bias, residual, BF16, seed=T + N)


@pytest.mark.parametrize("T", [1300, 1900])
@pytest.mark.parametrize("pad", [1, 8, 16])
def test_paired_slices_in_place(api, T, pad):
    K, N = 264, 1000
    (x, W, b, r), ref, tol = problem(T, K, N, "gelu", False, True, True, BF16, seed=T)
    xb = torch.full((T, K + 72), float("nan"), dtype=BF16, device="cuda")
    xb[:, 8:8 + K] = x
    ob = torch.full((T + 2, N + 2 * pad), 7.0, dtype=BF16, device="cuda")
    o = ob[1:T + 1, pad:pad + N]
    o.copy_(r)
    api.dr_linear(xb[:, 8:8 + K], W, o, bias=b, act="gelu", residual=o)
    torch.cuda.synchronize()
    assert_within(o, ref, tol, "in place")
    ob[1:T + 1, pad:pad + N] = 7.0
    assert (ob == 7.0).all()


def test_paired_nan_and_infinity_stay_in_their_rows_and_columns(api):
    T, K, N = 1900, 200, 1030
    (x, W, b, r), ref, tol = problem(T, K, N, None, False, True, True, BF16, seed=6)
    x, W = x.clone(), W.clone()
    x[1000, 3] = float("nan")
    x[1899] = float("inf")
    W[77, 5] = float("nan")
    o = torch.empty((T, N), dtype=BF16, device="cuda")
    api.dr_linear(x, W, o, bias=b, residual=r)
    o = o.cpu()
    assert o[1000].isnan().all() and not o[1899].isfinite().any() and o[:, 77].isnan().all()
    keep = torch.ones((T, N), dtype=torch.bool)
    keep[1000], keep[1899], keep[:, 77] = False, False, False
    assert_within(torch.where(keep, o.float(), ref.float()), ref, tol + 1e-6 * ref.abs(), "the others")


def test_paired_same_bits_on_two_streams_and_in_a_graph(api):
    s2 = torch.cuda.Stream()
    (x, W, b, r), ref, tol = problem(1900, 1024, 1024, "gelu", False, True, True, BF16, seed=8)
    first = torch.empty((1900, 1024), dtype=BF16, device="cuda")
    api.dr_linear(x, W, first, bias=b, act="gelu", residual=r)
    torch.cuda.synchronize()
    assert_within(first, ref, tol, "first")
    outs = [torch.empty_like(first) for _ in range(40)]
    for i, o in enumerate(outs):
        api.dr_linear(x, W, o, bias=b, act="gelu", residual=r, stream=s2 if i % 2 else None)
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)
    g, o = torch.cuda.CUDAGraph(), torch.empty_like(first)
    with torch.cuda.graph(g):
        for _ in range(2):
            api.dr_linear(x, W, o, bias=b, act="gelu", residual=r)
    for _ in range(3):
        o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, first)


@pytest.mark.parametrize("T,K,N,tile", [(2048, 512, 1024, 1), (1900, 72, 1089, 71)])
def test_paired_wait_that_runs_out(api, T, K, N, tile):
    (x, W, b, _), ref, tol = problem(T, K, N, None, False, True, False, BF16, seed=T)
    o = torch.full((T, N), float("nan"), dtype=BF16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.dr_linear_stall_test(tile, x, W, o, bias=b, err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) & api.DR_ERRF_TIMEOUT
    got = o.cpu()
    t0, n0 = tile // -(-N // 128) * 256, tile % -(-N // 128) * 128
    assert got[t0:t0 + 256, n0:n0 + 128].isnan().all()   # both CTAs' halves
    got[t0:t0 + 256, n0:n0 + 128] = ref[t0:t0 + 256, n0:n0 + 128].to(BF16)
    assert_within(got, ref, tol, "tiles that ran")
    err.zero_()
    api.dr_linear(x, W, o, bias=b, err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert_within(o, ref, tol, "the call after")


def test_refusals_of_the_binding(api):
    x, W = torch.zeros((4, 64), dtype=BF16, device="cuda"), torch.zeros((32, 64), dtype=BF16, device="cuda")
    o = torch.full((4, 32), 7.0, dtype=BF16, device="cuda")
    bad = [dict(x=x.float()), dict(x=x.cpu()), dict(x=x[0]), dict(W=W[:, :32]), dict(W=W[:31]), dict(out=o[:3]),
           dict(out=o.half()), dict(out=[]), dict(out=[o, o]), dict(bias=torch.zeros(31, dtype=BF16, device="cuda")),
           dict(bias=torch.zeros(32, device="cuda")), dict(act="tanh"), dict(residual=o.float()), dict(residual=o[:, :16]),
           dict(gated=True), dict(x=x.t().contiguous().t()), dict(out=o.t().contiguous().t()),
           dict(err_flag=torch.zeros(1, device="cuda"))]
    for change in bad:
        args = dict(dict(x=x, W=W, out=o), **change)
        with pytest.raises(ValueError):
            api.dr_linear(**args)
    with pytest.raises(RuntimeError, match="invalid"):       # an expanded row
        api.dr_linear(x[:1].expand(4, 64), W, o)
    with pytest.raises(RuntimeError, match="invalid"):       # 20 is not a multiple of 8
        api.dr_linear(x[:, :20], W[:, :20].contiguous(), o)
    torch.cuda.synchronize()
    assert (o == 7.0).all()
