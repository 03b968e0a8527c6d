"""The package without its library: the entry points are there, and calls raise."""
import os
import subprocess
import sys

import pytest

pytest.importorskip("torch")
ROOT = os.path.join(os.path.dirname(__file__), "..")

PROGRAM = """
import bit_quantized_expert_moe_gb300 as M
real, M.LIB_PATH = M.LIB_PATH, "/nowhere/libmoe_w4.so"
names = ["combine", "grouped_mm", "grouped_mm_dx", "grouped_mm_dw", "swiglu", "swiglu_backward", "block_norm",
         "block_norm_backward"]
assert all(hasattr(M, n) for n in names) and not hasattr(M, "grouped")
from bit_quantized_expert_moe_gb300 import swiglu
for fn in (swiglu, M.grouped_mm):
    try:
        fn()
    except RuntimeError as e:
        assert "/nowhere/libmoe_w4.so is missing" in str(e), e
    else:
        raise AssertionError("a call without the library")
"""


def test_entry_points_are_there_and_calls_raise():
    subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, check=True)
