"""The library and torch share one HIP runtime, whichever is asked for first
(no GPU: the process's mapped libraries tell)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LOOK = "print(len({l.split()[-1] for l in open('/proc/self/maps') if 'libamdhip64' in l}))"


@pytest.mark.parametrize("first,second", [("import binary_rank_linear_amd as b; b.load()", "import torch"),
                                          ("import torch", "import binary_rank_linear_amd as b; b.load()")])
def test_one_runtime(first, second):
    r = subprocess.run([sys.executable, "-c", f"{first}\n{second}\n{LOOK}"], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.split() == ["1"], r.stdout + r.stderr


def test_sizes_without_torch():
    """A machine without torch can still ask for sizes and status texts."""
    code = "import sys; sys.modules['torch'] = None\nimport binary_rank_linear_amd as b\n" \
           "assert b.blr_workspace_bytes(64, 256, 256, 128) > 0 and b.status_string(-2)"
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
