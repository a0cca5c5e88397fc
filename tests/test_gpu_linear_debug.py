"""Linear attention and layer norm in the index-checked build: no access of
theirs fails its check, and the results are those of the definition.  In a child
process, because a process loads one library."""
from __future__ import annotations

import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_no_check_fails():
    from ssd_chunked_forward_b200.build import build
    build(debug=True)
    env = dict(os.environ, SSD_DEBUG_CHECKS="1")
    res = subprocess.run([sys.executable, "-m", "tests.linear_debug_child"], capture_output=True, text=True, env=env,
                         cwd=ROOT, timeout=600)
    assert res.returncode == 0, res.stderr[-3000:]
    got = json.loads(res.stdout.strip().splitlines()[-1])
    assert got["record"] == [0, 0, 0, 0]
    for name, worst in got["worst"].items():
        # linear attention: in units of its bound; norms: of the largest value, bf16's rounding
        assert worst <= (2 ** -7 if "norm" in name else 1.0), (name, worst)
