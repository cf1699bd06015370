"""dr_residual_norm against float64, over widths, types, parts that are left out, layouts and what may stand in the rows."""
import pytest
import torch

from layer_reference import assert_within, residual_norm64

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def api(cuda_device):
    from decode_attention_self_gb300 import api as _api

    return _api


def randn(shape, seed, dtype=BF16, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale + shift).to(dtype)


def cuda(t):
    return None if t is None else t.cuda()


def check(api, T, D, x_dtype=BF16, h_dtype=BF16, y_dtype=BF16, pre="layer", post=None, gate=None, scale=1.0, residual=True,
          store_h=True, store_y=True, weight=True, bias=True, eps=1e-5, seed=0, x=None, res=None):
    x = randn((T, D), seed + 1, x_dtype) if x is None else x
    r = (randn((T, D), seed + 2, h_dtype, 2.0, 0.5) if res is None else res) if residual else None
    g = None if gate is None else randn((D,) if gate == "channel" else (T, D), seed + 3)

    def norm(kind, at):
        if kind is None:
            return None, None
        w = randn((D,), seed + at, BF16, 0.3, 1.0) if weight else None
        b = randn((D,), seed + at + 1, BF16, 0.3) if bias else None
        return (kind, eps, w, b), api.Norm(kind, eps, cuda(w), cuda(b))

    pre64, pre_own = norm(pre, 10)
    post64, post_own = norm(post, 20)
    (h_ref, h_tol), (y_ref, y_tol) = residual_norm64(x, post64, g, scale, r, pre64, h_dtype, y_dtype)
    h = torch.full((T, D), float("nan"), dtype=h_dtype, device="cuda") if store_h else None
    y = torch.full((T, D), float("nan"), dtype=y_dtype, device="cuda") if store_y else None
    api.dr_residual_norm(x.cuda(), y=y, pre=pre_own, residual=cuda(r), h=h, post=post_own, gate=cuda(g), scale=scale)
    torch.cuda.synchronize()
    what = f"T={T} D={D} pre={pre} post={post} gate={gate}"
    if store_h:
        assert_within(h, h_ref, h_tol, "h " + what)
    if store_y:
        assert_within(y, y_ref, y_tol, "y " + what)


WIDTHS = [8, 16, 24, 64, 72, 128, 200, 256, 264, 504, 512, 768, 1000, 1024, 1032, 1536, 2048, 2056, 2560, 4096, 5000, 8192,
          8200, 12288, 16384]


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("T", [1, 3, 37])
def test_widths(api, D, T):
    check(api, T, D, pre="layer", post="rms", gate="token", scale=0.5, seed=D)
    check(api, T, D, pre="rms", post="layer", gate="channel", x_dtype=F32, h_dtype=F32, y_dtype=F32, seed=D)


@pytest.mark.parametrize("D", [8, 24, 40, 64, 104, 192, 384, 504, 768, 1000, 1152, 1280, 1536, 2304, 2560, 4608, 8192, 12288, 16384])
@pytest.mark.parametrize("x_dtype,h_dtype", [(BF16, BF16), (BF16, F32), (F32, BF16)])
def test_widths_of_many_rows(api, D, x_dtype, h_dtype):
    # rows of several elements a thread, one after the other or two in turn
    check(api, 1201, D, x_dtype, h_dtype, BF16, "layer", "rms", "token", 0.5, seed=D)
    if D <= 1536:
        check(api, 20011, D, x_dtype, h_dtype, F32, "rms", None, "channel", 1.0, seed=D)


@pytest.mark.parametrize("T", [1, 2, 5, 16, 127, 128, 129, 1000, 5001])
@pytest.mark.parametrize("D", [64, 1024, 2048])
def test_token_counts(api, T, D):
    check(api, T, D, pre="layer", seed=T)


@pytest.mark.parametrize("x_dtype", [BF16, F32])
@pytest.mark.parametrize("h_dtype", [BF16, F32])
@pytest.mark.parametrize("y_dtype", [BF16, F32])
@pytest.mark.parametrize("pre", [None, "layer", "rms"])
@pytest.mark.parametrize("post", [None, "layer", "rms"])
def test_types_and_norms(api, x_dtype, h_dtype, y_dtype, pre, post):
    for gate, residual, store_h, store_y in ((None, True, True, True), ("channel", False, False, True), ("token", True, True, False),
                                             (None, False, True, True)):
        check(api, 19, 384, x_dtype, h_dtype, y_dtype, pre, post, gate, 0.25, residual, store_h, store_y, seed=7)


@pytest.mark.parametrize("weight,bias", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_parameters_left_out(api, weight, bias, kind):
    check(api, 9, 512, pre=kind, post=kind, weight=weight, bias=bias)


@pytest.mark.parametrize("D", [256, 1024, 4096])
def test_rows_far_from_zero_keep_their_differences(api, D):
    # a mean a thousand deviations away: squares minus the squared mean would lose the variance altogether
    res = randn((7, D), 3, F32, 1.0, 1000.0)
    check(api, 7, D, h_dtype=F32, y_dtype=F32, pre="layer", x=torch.zeros((7, D), dtype=BF16), res=res)
    # and with a few channels far larger than the others
    res = randn((7, D), 4, F32)
    res[:, 5] = 300.0
    res[:, D - 1] = -900.0
    check(api, 7, D, h_dtype=F32, y_dtype=F32, pre="layer", res=res)
    check(api, 7, D, h_dtype=F32, y_dtype=F32, pre="rms", res=res)


def test_rows_without_spread(api):
    # all elements equal, or all zero: eps is all that is left under the root
    D = 512
    x = torch.full((3, D), 2.5, dtype=BF16)
    x[1] = 0.0
    for kind in ("layer", "rms"):
        y = torch.empty((3, D), dtype=F32, device="cuda")
        api.dr_residual_norm(x.cuda(), y=y, pre=api.Norm(kind, 1e-5))
        want = torch.zeros((3, D)) if kind == "layer" else x.float() / torch.sqrt(x.float() ** 2 + 1e-5)
        assert (y.cpu() - want).abs().max() <= 2.0 ** -20
        # without eps a row of zeros is 0 / 0, as the formula says, and the others are right
        api.dr_residual_norm(x.cuda(), y=y, pre=api.Norm(kind, 0.0))
        assert y[1].isnan().all()


@pytest.mark.parametrize("D", [40, 1024, 2048])
def test_nan_and_infinity_stay_in_their_tokens(api, D):
    T = 21
    x, r = randn((T, D), 1), randn((T, D), 2)
    y0, h0 = torch.empty((T, D), dtype=BF16, device="cuda"), torch.empty((T, D), dtype=BF16, device="cuda")
    pre, post = api.Norm("layer"), api.Norm("rms")
    api.dr_residual_norm(x.cuda(), y=y0, pre=pre, residual=r.cuda(), h=h0, post=post)
    x2, r2 = x.clone(), r.clone()
    x2[4, 7], r2[11, D - 1] = float("nan"), float("inf")
    y, h = torch.empty_like(y0), torch.empty_like(h0)
    api.dr_residual_norm(x2.cuda(), y=y, pre=pre, residual=r2.cuda(), h=h, post=post)
    ok = torch.ones(T, dtype=torch.bool)
    ok[4] = ok[11] = False
    assert torch.equal(y.cpu()[ok], y0.cpu()[ok]) and torch.equal(h.cpu()[ok], h0.cpu()[ok])
    assert y[4].isnan().all() and h[4].isnan().all() and y[11].isnan().all() and h[11, D - 1].isinf()


@pytest.mark.parametrize("D", [64, 520, 1024])
@pytest.mark.parametrize("pad", [8, 24])
def test_slices_and_places(api, D, pad):
    T = 13

    def sliced(t, fill=float("nan")):
        b = torch.full((T + 2, D + 2 * pad), fill, dtype=t.dtype, device="cuda")
        b[1:T + 1, pad:pad + D] = t.cuda()
        return b, b[1:T + 1, pad:pad + D]

    x, r, g = randn((T, D), 1), randn((T, D), 2, F32), randn((T, D), 3)
    (h_ref, h_tol), (y_ref, y_tol) = residual_norm64(x, None, g, 1.5, r, ("rms", 1e-6, None, None), F32, BF16)
    hb, h = sliced(torch.zeros((T, D), dtype=F32), 7.0)
    yb, y = sliced(torch.zeros((T, D), dtype=BF16), 7.0)
    api.dr_residual_norm(sliced(x)[1], y=y, pre=api.Norm("rms", 1e-6), residual=sliced(r)[1], h=h, gate=sliced(g)[1], scale=1.5)
    torch.cuda.synchronize()
    assert_within(h, h_ref, h_tol, "h")
    assert_within(y, y_ref, y_tol, "y")
    for b in (hb, yb):
        b[1:T + 1, pad:pad + D] = 7.0
        assert (b == 7.0).all()


@pytest.mark.parametrize("D", [128, 1024, 3200])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_in_place(api, D, dtype):
    T = 40
    x, r = randn((T, D), 1, dtype), randn((T, D), 2, dtype)
    pre = ("layer", 1e-5, None, None)
    (h_ref, h_tol), (y_ref, y_tol) = residual_norm64(x, None, None, 1.0, r, pre, dtype, dtype)
    own = api.Norm("layer")
    h = r.cuda()
    y = torch.empty_like(h)
    api.dr_residual_norm(x.cuda(), y=y, pre=own, residual=h, h=h)      # the residual stream in place
    assert_within(h, h_ref, h_tol, "h")
    assert_within(y, y_ref, y_tol, "y")
    h, y = r.cuda(), x.cuda()
    api.dr_residual_norm(y, y=y, pre=own, residual=h, h=h)             # and the block's output too
    assert_within(h, h_ref, h_tol, "h")
    assert_within(y, y_ref, y_tol, "y")
    y = r.cuda()
    api.dr_residual_norm(x.cuda(), y=y, pre=own, residual=y)
    assert_within(y, y_ref, y_tol, "y over the residual")


def test_many_tokens_pass_32_bit_offsets(api):
    T, D = 1_100_000, 2048
    x = torch.randn((T, D), device="cuda", dtype=BF16)
    y = torch.empty_like(x)
    api.dr_residual_norm(x, y=y, pre=api.Norm("rms"))
    rows = torch.tensor([0, 7, 524288, 1_048_577, T - 1]).cuda()
    _, (ref, tol) = residual_norm64(x[rows], None, None, 1.0, None, ("rms", 1e-5, None, None), BF16, BF16)
    assert_within(y[rows], ref, tol, "far rows")


def test_same_bits_on_two_streams_and_in_a_graph(api):
    s2 = torch.cuda.Stream()
    for T, D in ((1, 1024), (128, 1536), (3000, 2048)):
        x, r = randn((T, D), 1).cuda(), randn((T, D), 2).cuda()
        pre = api.Norm("layer", 1e-5, randn((D,), 3).cuda(), randn((D,), 4).cuda())
        first, h = torch.empty_like(x), torch.empty_like(x)
        api.dr_residual_norm(x, y=first, pre=pre, residual=r, h=h)
        torch.cuda.synchronize()
        outs = [torch.empty_like(x) for _ in range(20)]
        for i, o in enumerate(outs):
            api.dr_residual_norm(x, y=o, pre=pre, residual=r, stream=s2 if i % 2 else None)
        torch.cuda.synchronize()
        assert all(torch.equal(o, first) for o in outs)
        o = torch.zeros_like(x)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            api.dr_residual_norm(x, y=o, pre=pre, residual=r)
        o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, first)


def test_refusals_of_the_binding(api):
    x = torch.zeros((4, 64), dtype=BF16, device="cuda")
    y = torch.full((4, 64), 7.0, dtype=BF16, device="cuda")
    w32 = torch.ones(64, device="cuda")
    bad = [dict(x=x[0]), dict(x=x.half()), dict(x=x.cpu()), dict(y=y[:3]), dict(y=y[:, :32]), dict(y=y.half()),
           dict(residual=x[:2]), dict(residual=x, h=y.float()), dict(gate=x[0, :32]), dict(gate=x.float()),
           dict(pre=api.Norm("batch")), dict(pre=api.Norm("rms", 1e-5, w32)), dict(post=api.Norm("layer", 1e-5, None, w32)),
           dict(x=x.t().contiguous().t())]
    for change in bad:
        args = dict(dict(x=x, y=y, pre=api.Norm("layer")), **change)
        with pytest.raises(ValueError):
            api.dr_residual_norm(**args)
    with pytest.raises(RuntimeError, match="invalid"):
        api.dr_residual_norm(x)                               # nothing to write
    with pytest.raises(RuntimeError, match="invalid"):
        api.dr_residual_norm(x, y=y, h=y)                     # both outputs in one place
    torch.cuda.synchronize()
    assert (y == 7.0).all()
