"""The bounds that the scan's step gradients are tested with (tests/step_gradient_bounds.py), on the
CPU: what a kernel could leave out of ddt, dA or ddt_bias does not pass them."""
import numpy as np
import pytest
import torch

from tests import test_gpu_layer_ops as ops
from tests.step_gradient_bounds import bounds, chunk_sums


@pytest.fixture()
def on_cpu(monkeypatch):
    def dev(a, io="f32"):
        return None if a is None else torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(ops.DT[io])
    monkeypatch.setattr(ops, "dev", dev)


@pytest.mark.parametrize("case", [s for s in ops.SCANS if max(s[1]) > 1], ids=lambda s: f"{s[0]}-{s[1]}-{s[3]}")
def test_bounds_tell_missing_terms(on_cpu, case):
    io, lens, _, H, G, Dk, Dv, D, bias, state, softplus = case
    a, rng = ops.scan_inputs(io, lens, H, G, Dk, Dv, D, bias, state, softplus, seed=41)
    dy = ops.rounded(rng.standard_normal(a["x"].shape), io)
    dST = ops.rounded(0.3 * rng.standard_normal((len(lens), H, Dv, Dk)), "f32") if state else None
    want = ops.scan_ref(a, softplus, lens, dy=dy, dST=dST)
    lim = bounds(a, io, softplus, lens, dy, dST)
    # zeros: the bound is a small part of the gradient's own norm (a head's dA or ddt_bias, one number
    # each, can be small by chance: less than half there, a small part of the heads' norm)
    assert np.all(lim["ddt"] < 1e-3 * np.linalg.norm(want["ddt"], axis=0))
    for name in ("dA", "ddt_bias"):
        assert np.all(lim[name] < 0.5 * np.abs(want[name])), name
        assert np.linalg.norm(lim[name]) < 0.05 * np.linalg.norm(want[name]), name
    # without the sums' share of what follows the block
    block = 128 if io == "bf16" else 64
    full, inner = chunk_sums(a, softplus, lens, dy, dST, block)
    missing = np.linalg.norm(full - inner, axis=0)
    assert np.all(missing > 10 * lim["ddt"]) or (max(lens) <= block and dST is None), missing / lim["ddt"]
    # without the factor of softplus, and without A
    if softplus:
        raw = a["dt"] + (0.0 if a["dt_bias"] is None else a["dt_bias"])
        wrong = np.linalg.norm(want["ddt"] / ops.R.sigmoid(raw) - want["ddt"], axis=0)
        assert np.all(wrong > 10 * lim["ddt"])


def test_chunk_sums_differ_by_one_number_a_block(on_cpu):
    """What the form without <G, S> lacks is A <G, S> for each token of a block: constant over it."""
    a, rng = ops.scan_inputs("f32", [150], 2, 1, 64, 64, False, False, True, False, seed=3)
    dy = rng.standard_normal(a["x"].shape)
    full, inner = chunk_sums(a, False, [150], dy, None, 64)
    for t0 in (0, 64, 128):
        d = (full - inner)[t0:t0 + 64]
        np.testing.assert_allclose(d, np.broadcast_to(d[:1], d.shape), rtol=1e-9, atol=1e-9 * np.abs(full).max())
