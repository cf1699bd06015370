"""Tensor-memory loads of the matrix products are waited for in the statement that issues them.

A load's registers hold nothing before its wait; the compiler takes a statement's outputs for there when the statement ends, and may
copy or spill them between a load and a later wait, as it does where values cross a loop's edge.
"""
import glob
import os
import re

import pytest

from decode_attention_self_gb300 import build

FILES = sorted(glob.glob(os.path.join(build.CSRC, "linear*.cu*")))


@pytest.mark.parametrize("path", FILES, ids=[os.path.basename(f) for f in FILES])
def test_no_load_is_left_in_flight(path):
    text = open(path).read()
    loads = re.findall(r"\btc::(ld\d+\w*)", text)
    assert all(name.endswith("_wait") for name in loads), sorted(set(loads))
    assert "tcgen05.ld" not in text and "wait_ld" not in text   # only by way of those


def test_waiting_loads_wait_in_their_statement():
    text = open(os.path.join(build.CSRC, "dr_tc.cuh")).read()
    bodies = re.findall(r"void (ld\d+\w*_wait)(\(.*?\n}\n)", text, flags=re.S)
    assert bodies
    for name, body in bodies:
        assert body.count("asm volatile") == 1, name
        assert body.rindex("tcgen05.wait::ld.sync.aligned") > body.rindex("tcgen05.ld.sync.aligned"), name
        assert re.search(r"E8\(q", body) and "R8(" not in body, name   # outputs apart from the inputs
