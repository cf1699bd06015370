"""Limits of dr_linear: a K whose products would outlast the kernels' bounded waits is refused before a launch."""
import pytest

from test_layer_host import lib, linear   # noqa: F401  (lib: fixture)


@pytest.mark.parametrize("T", [1, 20, 64, 4096])
@pytest.mark.parametrize("od", [0, 1])
@pytest.mark.parametrize("K", [2 ** 24 + 8, 2 ** 25, 2 ** 29, 2 ** 30])
def test_k_beyond_the_waits_is_refused(lib, T, od, K):   # noqa: F811
    assert linear(lib, xs=K, K=K, T=T, od=od) == 1
