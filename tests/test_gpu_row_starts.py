"""GPU checks that dr_rope_append flags every row_start that does not rise from 0 to at most T, wherever it does not."""
import pytest
import torch

from decode_attention_self_gb300 import workloads as W
from prompt_reference import Cache, D

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api(cuda_device):
    from decode_attention_self_gb300 import api as _api

    return _api


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def flag(api, dev, row_start, T):
    B = len(row_start) - 1
    cache = Cache([16] * B, 2, False, False, seed=6).gpu(api, dev)
    k, v, q = (W.randn_bf16((T, 2, D), dev, i) for i in range(3))
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    api.dr_rope_append(cache, k, v, i32(row_start, dev), i32([0] * B, dev), q=q, q_out=torch.empty_like(q), err_flag=err)
    return int(err.item())


@pytest.mark.parametrize("row_start,T", [([0, 5, 3, 8], 8), ([0, 8, 0, 8], 8), ([0, 3, -1, 8], 8), ([0, 9, 8], 8),
                                         ([0, 2, 1, 1], 1), ([1, 2, 3], 3), ([0, 4], 3),
                                         ([0] * 200 + [4] + [2] * 100 + [4], 4),      # far more rows than tokens
                                         (list(range(300)) + [298, 300], 300),
                                         ([0] * 63 + [-5] + [0, 2], 2)])
def test_a_fall_anywhere_is_flagged(api, cuda_device, row_start, T):
    assert flag(api, cuda_device, row_start, T) == api.DR_ERRF_ROW_START


@pytest.mark.parametrize("row_start,T", [([0, 5, 8], 8), ([0, 0, 0, 8, 8], 9), ([0] * 300 + [4], 4), ([0, 0], 3),
                                         (list(range(301)), 300), ([0] * 40 + [7] * 300, 7)])
def test_rising_rows_are_not(api, cuda_device, row_start, T):
    assert flag(api, cuda_device, row_start, T) == 0
