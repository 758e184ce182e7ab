"""The entry script run as a program: its main block comes last, behind everything that smoke() calls."""
import ast
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SCRIPT = os.path.join(ROOT, "__graft_entry__.py")


def test_main_block_is_last():
    with open(SCRIPT) as f:
        body = ast.parse(f.read()).body
    mains = [i for i, n in enumerate(body) if isinstance(n, ast.If) and "__name__" in ast.dump(n.test)]
    assert mains == [len(body) - 1]


@pytest.mark.gpu
def test_smoke_as_a_program():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    done = subprocess.run([sys.executable, SCRIPT, "--smoke"], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and "smoke ok" in done.stdout, done.stderr[-2000:]
