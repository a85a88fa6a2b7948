"""Warps that meet on a named barrier beside bounded waits: the source shows that one that gives up lets the other go (a wait
that runs out in such a kernel is not made to happen on a GPU)."""
import pathlib
import re

import pytest

CSRC = pathlib.Path(__file__).resolve().parent.parent / "block_sparse_long_kv_gb300" / "csrc"


def meeting():
    return sorted(p.name for p in CSRC.glob("*.cu") if "named_barrier(" in p.read_text() and "wait::" in p.read_text())


def test_there_are_such_kernels():
    assert "bsa_shared.cu" in meeting() and "bsa_selftest.cu" in meeting()


@pytest.mark.parametrize("name", meeting())
def test_a_warp_that_gives_up_lets_its_partner_go(name):
    text = re.sub(r"//[^\n]*", "", (CSRC / name).read_text())
    barriers = set(re.findall(r"named_barrier\((\w+),", text))
    left = set(re.findall(r"leave_pair\((\w+)\)", text))
    assert barriers and left == barriers
