"""CPU: the host planner runs where PyTorch is absent (a process that only plans calls
does not pay for loading it either)."""
import subprocess
import sys

import invariant_rmsnorm_fwd_gb300 as rb
from conftest import ROOT

PROGRAM = """
import sys
sys.modules["torch"] = None                     # any import of it raises
import numpy as np
import invariant_rmsnorm_fwd_gb300 as rb
plan, items, whole, spill = rb.plan_build(np.arange(70, dtype=np.int32), 1, 100)
assert (items, whole, spill) == (2, 1, 6), (items, whole, spill)
assert rb.plan_capacity(70, 1) >= items * rb.PLAN_ITEM_BYTES
assert rb.kernel_launches() == 0
"""


def test_planning_needs_no_torch():
    rb._load()                                  # built before the other process looks
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
