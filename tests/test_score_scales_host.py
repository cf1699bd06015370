"""Host-side refusals of scales whose products, which the kernels compute with, are not finite in fp32."""
import pytest

from test_prompt_host import GOOD, lib, prompt, shared  # noqa: F401

INVALID = 1
CODES = dict(GOOD, kv_dtype=1, v_scale=1.0)


@pytest.mark.parametrize("bad", [
    dict(scale=3e38),                                                # times log2 e
    dict(cache=dict(CODES, k_scale=1e30), scale=1e9),                # times k_scale
    dict(scale=1e33, opts=dict(causal=1, softcap=1e-6)),             # over the cap
    dict(cache=dict(CODES, k_scale=1e34), opts=dict(causal=1, softcap=1e-6)),
])
def test_products_that_overflow_are_refused(lib, bad):  # noqa: F811
    assert prompt(lib, **bad) == INVALID
    opts = {k: v for k, v in bad.get("opts", {}).items() if k != "causal"} or None
    given = dict(scale=bad.get("scale", 0.0), opts=opts)
    assert shared(lib, prefix=bad.get("cache"), **given) == INVALID
    assert shared(lib, own=bad.get("cache"), **given) == INVALID

