"""Plans at the numbers of slots where their shared memory passes what a kernel may have without asking."""
import subprocess
import sys
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PLAN = """
import sys, torch
import serving_q8_encode_gb300 as pk
A = int(sys.argv[1])
t = pk.PageTable(A, 2, 2 * A, 16)
new = torch.arange(A, dtype=torch.int32, device="cuda") % 3
for _ in range(2):
    plan = t.plan(new, 2 * A)
starts = torch.cat([new.new_zeros(1), new.cumsum(0).int()])
assert torch.equal(plan.starts, starts), "starts"
assert torch.equal(plan.after, torch.where(new > 0, 2 * new, -1)), "after"
assert torch.equal(t.counts.cpu(), torch.tensor([int((new > 0).sum()), 2 * A])) and t.status() == 0
"""


@pytest.mark.parametrize("A", [2559, 2560, 2561, 3061, 3062, 3063, 3067, 3071, 3073])
def test_first_plan_of_a_process(A):
    """Each in a process of its own: an earlier and larger plan would have asked for all that comes after it."""
    import __graft_entry__
    __graft_entry__.build()
    r = subprocess.run([sys.executable, "-c", PLAN, str(A)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
