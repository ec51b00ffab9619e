"""The entry points at the repository's root, run as a program."""
import os
import subprocess
import sys

import pytest
import torch

from shared_prefix_grouped_gb300.build import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

NAMES = """
import runpy
calls = []
import shared_prefix_grouped_gb300.build as b
b.build = lambda *a, **k: calls.append("build")
m = runpy.run_path("__graft_entry__.py", run_name="entry")
import ast
tree = ast.parse(open("__graft_entry__.py").read())
assert isinstance(tree.body[-1], ast.If), "what runs as a program comes after all it calls"
names = {n.func.id for n in ast.walk(tree) if isinstance(n, ast.Call) and isinstance(n.func, ast.Name)}
assert {n for n in names if n.startswith("_smoke")} <= set(m)
"""


def test_what_the_program_calls_stands_before_it():
    subprocess.run([sys.executable, "-c", NAMES], check=True, cwd=ROOT)


@pytest.mark.gpu
def test_smoke_as_a_program():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()
    out = subprocess.run([sys.executable, "__graft_entry__.py", "smoke"], cwd=ROOT, capture_output=True, text=True)
    assert out.returncode == 0 and "smoke ok" in out.stdout, out.stderr[-2000:]
