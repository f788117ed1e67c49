"""The product that a bounded wait of the Newton-Schulz kernel records (no GPU).

Every wait inside a tile knows the tile's product and records it; the waits of
the tile rings alone, which wait for a tile, have none and record 0.  In
launches with narrow tiles the scheduler waits for a tile's dependency beside
its producer, and whichever runs out first writes the status word: a wait that
recorded 0 there would name the wrong product, once in a few runs.
"""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_waits_for_a_dependency_record_their_product():
    with open(os.path.join(ROOT, "matrix_optimizers_under_gb300", "csrc", "ns_gemm.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    codes = re.findall(r"wait_code\(\s*([\w.]+)\s*,\s*(kRole\w+)\s*\)", text)
    assert len(codes) >= 15                                   # the waits are still written this way
    without = {role for phase, role in codes if phase == "0"}
    assert without <= {"kRoleTileFree", "kRoleTileFull"}, without
    assert "kRoleDependency" in {role for phase, role in codes if phase == "tl.phase"}
