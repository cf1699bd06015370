"""GPU checks of NaN in a query or in a key that is seen: the outputs that it reaches are NaN, whichever kernel, split and
workspace take the call, and no other output is touched.  Tolerances are those of prompt_reference."""
import pytest
import torch

from decode_attention_self_gb300 import workloads as W
from prompt_reference import Cache, D, assert_close, attend, starts
from test_gpu_shared_prefix import reference as shared_reference

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(scope="module")
def api(cuda_device):
    from decode_attention_self_gb300 import api as _api

    return _api


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def spoil_keys(cache, b, keys, head):
    i0, i2 = cache.slots(b, max(keys) + 1)
    for j in keys:
        cache.k[i0[j], head, i2[j], 3] = 0x7F if cache.k.dtype == torch.uint8 else NAN


def same(got, ref, tol, what):
    """NaN exactly where the reference has it, the rest within tolerance."""
    nan = ref.isnan()
    assert torch.equal(got.cpu().isnan(), nan), what
    assert nan.any() and not nan.all(), what
    assert_close(got[~nan.to(got.device)], ref[~nan], tol[~nan], what)


def prompt(api, dev, cache, q, new, kv, Hkv, fp8, first=None, workspace=True, what=""):
    T, Hq = q.shape[:2]
    out = torch.full((T, Hq, D), 3.0, device=dev)
    nb = api.dr_prompt_attn_workspace(T, len(new), Hq, Hkv, max(kv)) if workspace else 0
    ws = torch.full((nb,), 0x11, dtype=torch.uint8, device=dev) if nb else None
    api.dr_prompt_attn(q.to(dev), cache.gpu(api, dev), starts(new).to(dev), i32(kv, dev), out, max_len_hint=max(kv),
                       first_key=None if first is None else i32(first, dev), workspace=ws)
    refs, tols, at = [], [], 0
    for b, (n, L) in enumerate(zip(new, kv)):
        pos = torch.arange(L - n, L)
        lo = torch.zeros(n, dtype=torch.long) if first is None else torch.tensor(first[at:at + n])
        K, V = cache.rows(b, L)
        r, t = attend(q[at:at + n], K, V, lo, pos + 1, pos, fp8=fp8)
        refs.append(r)
        tols.append(t)
        at += n
    same(out, torch.cat(refs), torch.cat(tols), what)
    return nb


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new,kv", [([1, 1], [60, 33]),           # one CTA per row and head
                                    ([1, 1], [3000, 700]),        # eight
                                    ([40, 1], [200, 90]), ([40], [9000])])
@pytest.mark.parametrize("workspace", [False, True])
def test_a_query_that_is_not_a_number(api, cuda_device, fp8, new, kv, workspace):
    cache = Cache(kv, 2, True, fp8, 3)
    q = W.randn_bf16((sum(new), 4, D), "cpu", 1, 7)
    q[0, 1, 5] = NAN
    q[sum(new) - 1, 2, 63] = NAN
    nb = prompt(api, cuda_device, cache, q, new, kv, 2, fp8, workspace=workspace)
    assert (nb > 0) == (workspace and kv == [9000])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [1, 2, 40])
def test_the_only_visible_key_is_not_a_number(api, cuda_device, fp8, new):
    """The first token of row 0 sees key 0 alone; where there are more, they see the others alone."""
    kv = [new, 50]
    cache = Cache(kv, 2, False, fp8, 4)
    spoil_keys(cache, 0, [0], 1)
    first = [0] + [1] * (new - 1) + [0]
    prompt(api, cuda_device, cache, W.randn_bf16((new + 1, 4, D), "cpu", 2, 7), [new, 1], kv, 2, fp8, first=first)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("at", ["first", "middle", "last"])
def test_a_run_of_keys_that_are_not_numbers(api, cuda_device, fp8, new, at):
    """Long enough that one of the CTAs that share a row has no other key, first or last among them."""
    L = 9000
    cache = Cache([L], 2, True, fp8, 5)
    lo, hi = {"first": (0, 2600), "middle": (3000, 6000), "last": (6400, L - 40)}[at]
    spoil_keys(cache, 0, range(lo, hi), 0)
    assert prompt(api, cuda_device, cache, W.randn_bf16((new, 4, D), "cpu", 2, 7), [new], [L], 2, fp8) > 0 or new == 1


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("P,own", [(300, [5, 0, 70]), (9000, [5, 0, 70]), (40, [3000, 10, 0])])
@pytest.mark.parametrize("where", ["query", "prefix", "own"])
def test_shared_prefix(api, cuda_device, fp8, P, own, where):
    dev, B, Hq, Hkv = cuda_device, len(own), 4, 2
    prefix, cache = Cache([P], Hkv, True, fp8, 6), Cache([max(n, 1) for n in own], Hkv, True, fp8, 7)
    q = W.randn_bf16((B, Hq, D), "cpu", 2)
    if where == "query":
        q[0, 3, 1] = q[1, 0, 0] = NAN
    elif where == "prefix":
        spoil_keys(prefix, 0, range(0, min(P, 2600)), 1)
    else:
        spoil_keys(cache, 0, range(own[0]), 0)
    out = torch.full((B, Hq, D), 3.0, device=dev)
    ws = torch.full((api.dr_shared_prefix_attn_workspace(B, Hq, Hkv, P),), 0x11, dtype=torch.uint8, device=dev)
    api.dr_shared_prefix_attn(q.to(dev), prefix.gpu(api, dev), i32([P], dev), out, ws, cache=cache.gpu(api, dev),
                              seq_len=i32(own, dev), max_prefix_hint=P)
    ref, tol = shared_reference(prefix, P, cache, own, q, 0.0, None, fp8, torch.float32)
    same(out, ref, tol, where)


def test_no_prefix_and_one_own_key_that_is_not_a_number(api, cuda_device):
    dev = cuda_device
    prefix, cache = Cache([16], 2, False, False, 6), Cache([4, 4, 4], 2, False, False, 7)
    spoil_keys(cache, 1, [0], 0)
    q = W.randn_bf16((3, 4, D), "cpu", 2)
    out = torch.full((3, 4, D), 3.0, device=dev)
    ws = torch.empty(api.dr_shared_prefix_attn_workspace(3, 4, 2, 16), dtype=torch.uint8, device=dev)
    api.dr_shared_prefix_attn(q.to(dev), prefix.gpu(api, dev), i32([0], dev), out, ws, cache=cache.gpu(api, dev),
                              seq_len=i32([0, 1, 3], dev))
    ref, tol = shared_reference(prefix, 0, cache, [0, 1, 3], q, 0.0, None, False, torch.float32)
    same(out, ref, tol, "own")
    assert (out[0] == 0).all()
