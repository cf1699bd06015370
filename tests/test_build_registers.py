"""The build refuses a tile kernel whose registers per thread are not those that its register split counts on."""
import pytest

from decode_attention_self_gb300 import build

LINE = """ptxas info    : Compiling entry function '_ZN2dr17attn_tiles_kernelILb{0}EEEv' for 'sm_103a'
ptxas info    : Function properties for _ZN2dr17attn_tiles_kernelILb{0}EEEv
    24 bytes stack frame, 52 bytes spill stores, 76 bytes spill loads
ptxas info    : Used {1} registers, used 1 barriers, 24 bytes cumulative stack size
"""
OTHER = """ptxas info    : Compiling entry function '_ZN2dr16attn_join_kernelEv' for 'sm_103a'
ptxas info    : Used 48 registers, used 0 barriers
"""


def test_registers_that_the_split_counts_on():
    build.check_registers("attn_tiles.cu", LINE.format(0, 128) + OTHER + LINE.format(1, 128))


@pytest.mark.parametrize("report", [LINE.format(0, 128) + LINE.format(1, 126), LINE.format(0, 168) + OTHER, OTHER, ""])
def test_others_are_refused(report):
    with pytest.raises(RuntimeError):
        build.check_registers("attn_tiles.cu", report)
