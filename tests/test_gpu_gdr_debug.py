"""The bounds-checked build under the tests of the one-decay rule and of the backward passes of the
prologue and the output epilogue: no false alarms, unchanged results.  A child pytest process with
KDA_LIB=debug, as in test_gpu_debug_build.py.
"""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(os.environ.get("KDA_LIB") == "debug", reason="already the debug-build process")
def test_training_operators_on_the_debug_build():
    lib = os.path.join(ROOT, "gated_delta_rule_prologue_b200", "libkda_debug.so")
    assert os.path.exists(lib), "libkda_debug.so is missing: run __graft_entry__.build()"
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
           "tests/test_gpu_gdr.py", "tests/test_gpu_gdr_paths.py", "tests/test_gpu_training_path.py"]
    r = subprocess.run(cmd, cwd=ROOT, env=dict(os.environ, KDA_LIB="debug"), capture_output=True,
                       text=True, timeout=1200)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
    assert " passed" in r.stdout and "failed" not in r.stdout, r.stdout[-3000:]
