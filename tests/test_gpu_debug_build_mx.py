"""The GQ_DEBUG build of the router and the products of microscaled blocks (GPU only): built beside the normal
library, run in a child process, correct results and a clean status word (tests/debug_build_mx_checks.py)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_debug_build_runs_clean():
    from quantized_skinny_matmul_gb300 import _build
    env = dict(os.environ, GQ_LIBRARY=_build.build(debug=True))
    res = subprocess.run([sys.executable, os.path.join(HERE, "debug_build_mx_checks.py")], env=env,
                         capture_output=True, text=True, timeout=900)
    assert res.returncode == 0, res.stdout[-2000:] + res.stderr[-4000:]
    assert "debug build clean" in res.stdout
