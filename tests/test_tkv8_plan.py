"""The sizes of tests/tkv8_plan.py take the paths that they are there for, so that a change of the plan's constants does not
empty the tests that go by them.  On the CPU: the host half with launchers that print."""
import os
import shutil

import pytest

from tests import tkv8_plan

pytestmark = pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists("/opt/rocm/include/hip"),
                                reason="g++ or the HIP headers not available")


def test_windows_that_are_dealt_evenly(tmp_path):
    cases = tkv8_plan.EVEN_WINDOWS
    plans = tkv8_plan.plans(cases, tmp_path)
    assert len(plans) == len(cases)
    for c, p in zip(cases, plans):
        assert p.even and p.window == c.window and p.row_tile <= 32, (c, p)
    for bits in (8, 4):
        some = [p for c, p in zip(cases, plans) if c.bits == bits]
        assert {p.row_tile for p in some} == {16, 32} and any(p.row_blocks > 1 for p in some)


def test_many_rows_in_several_chunks(tmp_path):
    cases = tkv8_plan.MANY_ROWS + tkv8_plan.MANY_CHUNKS
    plans = tkv8_plan.plans(cases, tmp_path)
    assert len(plans) == len(cases)
    for c, p in zip(cases, plans):
        assert not p.even and p.row_tile >= 64 and p.window == c.window, (c, p)
        assert p.n_split > 16 if c in tkv8_plan.MANY_CHUNKS else 1 < p.n_split <= 16, (c, p)
    assert {(c.bits, p.row_tile) for c, p in zip(cases, plans)} == {(8, 128), (4, 64), (4, 128)}
    assert any(p.row_blocks > 1 for p in plans) and {p.n_split <= 4 for p in plans} == {True, False}
