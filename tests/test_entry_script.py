"""The build and smoke file run as a script."""
import ast
import os
import subprocess
import sys

import pytest

from tests._gpu_util import require_gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FILE = os.path.join(ROOT, "__graft_entry__.py")


def test_script_has_all_functions_when_it_calls_smoke():
    """smoke() in place of which the names that are there by then are noted."""
    with open(FILE) as f:
        tree = ast.parse(f.read())
    functions = [n for n in tree.body if isinstance(n, ast.FunctionDef)]
    for n in functions:
        if n.name == "smoke":
            n.body = ast.parse("seen.update(globals())").body
    seen = {}
    exec(compile(ast.fix_missing_locations(tree), FILE, "exec"), {"__name__": "__main__", "__file__": FILE, "seen": seen})
    assert seen and all(n.name in seen for n in functions)


@pytest.mark.gpu
def test_script_runs():
    require_gpu()
    r = subprocess.run([sys.executable, FILE], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "smoke ok" in r.stdout, r.stderr[-2000:]
