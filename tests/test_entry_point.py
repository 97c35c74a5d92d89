"""The entry points' file run as a script."""
import ast
import os
import subprocess
import sys

import pytest

from conftest import ROOT

PATH = os.path.join(ROOT, "__graft_entry__.py")


def test_script_runs_after_its_functions():
    """The block that a script's run enters stands after every function it may call."""
    with open(PATH) as f:
        body = ast.parse(f.read()).body
    runs = [i for i, node in enumerate(body) if isinstance(node, ast.If) and "__name__" in ast.unparse(node.test)]
    assert len(runs) == 1
    late = [node.name for node in body[runs[0]:] if isinstance(node, ast.FunctionDef)]
    assert not late, f"defined after the script has run: {late}"


@pytest.mark.gpu
def test_smoke_as_a_script():
    r = subprocess.run([sys.executable, PATH, "smoke"], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "smoke ok" in r.stdout, r.stderr[-2000:]
