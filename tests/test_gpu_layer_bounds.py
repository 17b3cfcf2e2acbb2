"""The debug-bounds build on the operators around the mixer: every computed index of their global
stores stays inside its buffer, and the outputs are the release build's bit for bit.  Each build
runs in a process of its own (tests/layer_bounds_run.py)."""
import json
import os
import subprocess
import sys

import pytest

from delta_rule_recurrent_osdn_b200 import build as B

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(lib, out):
    subprocess.run([sys.executable, "-m", "tests.layer_bounds_run", str(out)], cwd=ROOT,
                   env=dict(os.environ, OSDN_LIBRARY=lib), check=True, timeout=600)
    with open(out) as f:
        return json.load(f)


def test_debug_bounds_build_matches_release(tmp_path):
    B.build()
    B.build(debug_bounds=True)
    rel = run(B.LIB, tmp_path / "release.json")
    dbg = run(B.DEBUG_LIB, tmp_path / "debug.json")
    assert rel.pop("library") == B.LIB and dbg.pop("library") == B.DEBUG_LIB
    assert rel.keys() == dbg.keys()
    for case in rel:
        assert rel[case]["status"] == 0, (case, "release", rel[case]["status"])
        assert dbg[case]["status"] == 0, (case, "debug-bounds", dbg[case]["status"])
        assert dbg[case]["outputs"] == rel[case]["outputs"], case
