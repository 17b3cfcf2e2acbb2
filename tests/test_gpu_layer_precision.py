"""Accuracy of the layer operators where it is easily lost: small residual scales, tokens that make
the state forget, gradients of steps.  Against the 64-bit statements of tests/layer_ref.py.

E = 2^-24 is half a step of fp32, relative; U that of the io type.  Tolerances count roundings, and
are stated at each test.
"""
import numpy as np
import pytest
import torch

from tests import layer_ref as R
from tests.test_gpu_layer_ops import E, U, close, dev, finish, norm_inputs, osdn, rounded  # noqa: F401

pytestmark = pytest.mark.gpu


# ====================================================================================== norm
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("res,gate", [(False, False), (False, True), (True, False)])
@pytest.mark.parametrize("scale", [1e-3, 1e-4, 1e-6, 2e-8, 0.0, -1e-5])
def test_norm_gradients_at_small_scales(osdn, io, res, gate, scale):  # noqa: F811
    """Without the first norm, scale * f alone is what the second norm sees (with a residual, a part
    of it).  A gradient's terms pass at most 16 products and the sums over a row (D) and, for the
    weights, over the rows: k = 16 + D (+ R) roundings of the sum of the terms' magnitudes."""
    Rr, D, eps = 40, 96, 1e-5
    a, rng = norm_inputs(io, Rr, D, gate, False, res, True, seed=21)
    dxo, dh = (rounded(rng.standard_normal((Rr, D)), io) for _ in range(2))
    s32 = float(np.float32(scale))
    want = R.norm(a["f"], a["x"], a["gate"], None, a["w_next"], "silu", False, s32, eps, dxo, dh)
    d = {k: dev(v, "f32" if k.startswith("w") else io) for k, v in a.items()}
    kw = dict(scale=scale, eps=eps)
    xo, h = osdn.osdn_norm_fwd(d["f"], d["x"], d["gate"], None, d["w_next"], **kw)
    g = osdn.osdn_norm_bwd(d["f"], dev(dxo, io), dev(dh, io), d["x"], d["gate"], None, d["w_next"], **kw)
    finish(osdn)
    act = 1.0 if a["gate"] is None else a["gate"] * R.sigmoid(a["gate"])
    u = np.abs(s32 * a["f"] * act) + (0.0 if a["x"] is None else np.abs(a["x"]))  # |x'| or more
    xp = want["x_out"]
    rn = 1 / np.sqrt((xp * xp).mean(-1, keepdims=True) + eps)
    dn = np.abs(dh * a["w_next"])
    mag = np.abs(dxo) + rn * (dn + u * rn * (dn * u * rn).mean(-1, keepdims=True))
    k = (16 + D) * E
    close(xo, want["x_out"], U[io] * np.abs(xp) + k * u, "x_out")
    close(h, want["h"], U[io] * np.abs(want["h"]) + k * u * rn * np.abs(a["w_next"]), "h")
    close(g["dw_next"], want["dw_next"], (16 + D + Rr) * E * (np.abs(dh) * u * rn).sum(0), "dw_next")
    close(g["df"], want["df"], U[io] * np.abs(want["df"]) + k * np.abs(s32) * 1.1 * mag * (
        1.0 if a["gate"] is None else np.maximum(1.0, np.abs(act))), "df")
    if res:
        close(g["dx"], want["dx"], U[io] * np.abs(want["dx"]) + k * mag, "dx")
    if gate:
        close(g["dgate"], want["dgate"], U[io] * np.abs(want["dgate"]) + k * np.abs(s32) * 2 * mag *
              np.abs(a["f"]) * np.maximum(1.0, np.abs(a["gate"])), "dgate")
