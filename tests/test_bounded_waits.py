"""Bounded waits of the attention kernels, read from the source (a wait that runs out is not provoked on a GPU): where
warps meet behind waits that each of them times for itself, they have to meet whatever the waits said."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "transformer_layer_pre_b200", "csrc")


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_warps_that_gave_up_still_meet_at_the_named_barriers():
    code = _code("attention_tc.cu")
    assert not re.search(r"\bnamed_barrier\s*\(", code)          # tells nobody that another warp gave up
    assert len(re.findall(r"if \(!\(ok = named_barrier_all\(1, 128, ok\)\)\) break;", code)) == 2


@pytest.mark.parametrize("begin", ["if (ok && (ok = wait_warp<0>(pv_done", "ok = wait_warp<kPauseStore>(&st_full[slot]"])
def test_no_warp_leaves_between_its_last_wait_and_the_barrier(begin):
    code = _code("attention_tc.cu")
    at = code.index(begin)
    part = code[at:code.index("named_barrier_all", at)]
    assert "break" not in part and "return" not in part and "continue" not in part


def test_pairs_of_warps_of_the_long_layer_attention_leave_together():
    code = _code("attn_tc.cu")
    at = code.index("const int bar_id = 1 + quarter;")
    part = code[at:code.index("tmem_dealloc", at)]
    assert len(re.findall(r"ok = named_barrier_all\(bar_id, 64, true\)\)\) break;", part)) == 2
    # a wait that ran out leads to one of these barriers before the warp leaves
    waits = re.findall(r"mbar_wait_warp\([^;]*\)\) (.*)", part)
    assert len(waits) == 5 and all(w.startswith("{ gave_up(); break; }") for w in waits)
    assert len(re.findall(r"[^_]named_barrier\(bar_id, 64\)", part)) == 1
