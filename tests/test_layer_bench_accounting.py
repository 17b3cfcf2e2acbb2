"""The byte counts that the benchmark's layer workloads are divided by, against hand counts: each of
a step's three calls reads its inputs and writes its outputs once."""
import json
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import bench  # noqa: E402

V = 16 * 128 * 2  # bytes of a token's values (x, y, gate), and of its b or c


def test_forward_bytes():
    # conv 2 values and 3 rows of state; scan x, b, c, y, dt and S_T; norm 3 values
    tokens = 4 * 4096
    want = tokens * (2 * V + 4 * V + 64 + 3 * V) + 4 * 3 * V + 4 * 16 * 65536
    assert bench.layer_bytes("layer", tokens, 4, 16, 128, 128, 4) == want


def test_backward_bytes():
    # norm 5 values; scan reads x, b, c, dt, dy, writes dx, db, dc, ddt; conv 3 values
    tokens = 4 * 4096
    want = tokens * (5 * V + 7 * V + 128 + 3 * V)
    assert bench.layer_bytes("layer_bwd", tokens, 4, 16, 128, 128, 4) == want


def test_step_bytes():
    # both states read and written: 3 rows of the convolution's, 64 KB a head of the scan's
    want = 256 * (2 * V + 6 * V + 4 * V + 64 + 2 * 16 * 65536 + 3 * V)
    assert bench.layer_bytes("layer_step", 256, 256, 16, 128, 128, 4) == want


@pytest.mark.parametrize("workload", sorted(bench.LAYER_DESC))
def test_reference_arm_says_why_it_has_none(workload, capsys):
    assert bench.main(["--impl", "reference", "--workload", workload]) == 0
    line = json.loads(capsys.readouterr().out)
    assert line["impl"] == "reference" and line["unavailable"]
