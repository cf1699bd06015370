"""GPU check of the positions behind a shared prefix where a row's length is outside its cache: it counts as clamped, for the
biases on the prefix's keys as for those on its own.  Tolerances are those of prompt_reference."""
import pytest
import torch

from decode_attention_self_gb300 import workloads as W
from prompt_reference import Cache, D, assert_close
from test_gpu_shared_prefix import reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_lengths_outside_are_clamped_for_the_bias_too(cuda_device, paged, fp8):
    from decode_attention_self_gb300 import api

    dev, P, cap, Hq, Hkv = cuda_device, 200, 32, 4, 2
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    given = [32, 33, 500, 2 ** 31 - 1, -1, -2 ** 31, 0]
    own = [min(max(n, 0), cap) for n in given]
    prefix, cache = Cache([P], Hkv, paged, fp8, 1), Cache([cap] * len(own), Hkv, paged, fp8, 2)
    q = W.randn_bf16((len(own), Hq, D), "cpu", 3)
    slopes = torch.tensor([0.01, 0.02, 0.03, 0.05])
    out, err = torch.empty((len(own), Hq, D), device=dev), i32([0])
    ws = torch.empty(api.dr_shared_prefix_attn_workspace(len(own), Hq, Hkv, P), dtype=torch.uint8, device=dev)
    api.dr_shared_prefix_attn(q.to(dev), prefix.gpu(api, dev), i32([P]), out, ws, cache=cache.gpu(api, dev),
                              seq_len=i32(given), slopes=slopes.to(dev), err_flag=err)
    assert int(err.item()) == api.DR_ERRF_SEQ_LEN
    ref, tol = reference(prefix, P, cache, own, q, 0.0, slopes, fp8, torch.float32)
    assert_close(out, ref, tol, "clamped")
