"""torch.compile of a function whose first call of the package is the compiled one, in a process of its own, on the CPU:
the package's refusal comes through, as from the eager call."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CHILD = """
import torch
import linear_cross_entropy_tiled_amd as flce
if {recorded}:
    fn = lambda x: flce.layer_norm(-x) * 2
else:
    fn = lambda x: flce.embedding_backward(-x, torch.zeros(4, dtype=torch.int64), 10) * 2
for f in (torch.compile(fn, backend="eager"), fn):
    try:
        f(torch.randn(4, 8))
    except ValueError as e:
        assert "GPU" in str(e), e
    else:
        raise SystemExit("not refused")
print("refused twice")
"""


@pytest.mark.parametrize("recorded", [True, False])
def test_a_first_call_under_the_compiler(recorded):
    r = subprocess.run([sys.executable, "-W", "ignore", "-c", CHILD.format(recorded=recorded)], cwd=ROOT,
                       stdout=subprocess.PIPE, stderr=subprocess.STDOUT, timeout=300)
    out = r.stdout.decode(errors="replace")
    assert r.returncode == 0 and out.strip().endswith("refused twice"), out[-2000:]
