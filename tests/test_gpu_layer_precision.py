"""Accuracy of the layer operators where it is easily lost: small residual scales, tokens that make
the state forget, gradients of steps.  Against the 64-bit statements of tests/layer_ref.py.

E = 2^-24 is half a step of fp32, relative; U that of the io type.  Tolerances count roundings, and
are stated at each test.
"""
import numpy as np
import pytest
import torch

from tests import layer_ref as R
from tests.step_gradient_bounds import bounds, relative_error
from tests.test_gpu_layer_ops import (E, NORMS, SCANS, U, close, dev, finish, norm_inputs,  # noqa: F401
                                      osdn, rounded, scan_bwd, scan_dev, scan_fwd, scan_inputs,
                                      scan_ref)

pytestmark = pytest.mark.gpu


def relative_l2(got, want):
    want = np.asarray(want).reshape(got.shape)
    return np.linalg.norm(got.detach().double().cpu().numpy() - want) / max(np.linalg.norm(want), 1e-300)


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


@pytest.mark.parametrize("io,Rr,D,gate,first,act,post,res,nxt", NORMS)
def test_norm_by_norm(osdn, io, Rr, D, gate, first, act, post, res, nxt):  # noqa: F811
    """Every result in L2 norm: bf16 to its own rounding, fp32 to 2^-18 (gradients 2^-17).  A value passes
    some 16 products (2^-24 each); a sigmoid is good to 2^-21 (e^-z and a quotient of 2^-22, and z's own
    rounding, |z| < 5); a row's sum of squares adds 16 values a thread one after another and the threads
    in a tree, 32 x 2^-24 at most, of which the root takes half: (16 + 8 + 16) 2^-24 < 2^-18.  Gradients
    pass both a norm's products and its sum twice.  Rows of one value: df = dn (1 - n^2) / rms with
    1 - n^2 = eps / (f^2 + eps), formed as dn - n (dn n) from products off by 2^-24 of dn each, four of them
    at most: 4 x 2^-24 (f^2 + eps) / eps more.  Weight gradients sum the rows' terms in fp32, Rr of
    them, with random signs: another sqrt(Rr) 2^-24."""
    a, rng = norm_inputs(io, Rr, D, gate, post, res, nxt, seed=22)
    dxo = rounded(rng.standard_normal((Rr, D)), io)
    dh = rounded(rng.standard_normal((Rr, D)), io) if nxt else None
    want = R.norm(a["f"], a["x"], a["gate"], a["w_post"], a["w_next"], act, first, 0.5, 1e-5, dxo, dh)
    d = {k: dev(v, "f32" if k.startswith("w") else io) for k, v in a.items()}
    kw = dict(gate_act=act, gate_first=first, scale=0.5, eps=1e-5)
    xo, h = osdn.osdn_norm_fwd(d["f"], d["x"], d["gate"], d["w_post"], d["w_next"], **kw)
    g = osdn.osdn_norm_bwd(d["f"], dev(dxo, io), dev(dh, io), d["x"], d["gate"], d["w_post"], d["w_next"], **kw)
    finish(osdn)
    half = 1.9e-3 if Rr * D > 500 else 2.0 ** -8
    for name, got, lim in (("x_out", xo, 2.0 ** -18), ("h", h, 2.0 ** -18), ("df", g["df"], 2.0 ** -17),
                           ("dx", g["dx"], 2.0 ** -17), ("dgate", g["dgate"], 2.0 ** -17)):
        if got is not None:
            lim = half if io == "bf16" else lim
            if name == "df" and D == 1:
                lim += 4 * E * (a["f"].max() ** 2 + 1e-5) / 1e-5
            assert relative_l2(got, want[name]) <= lim, name
    for name in ("dw_post", "dw_next"):
        if g[name] is not None and D > 1:
            assert relative_l2(g[name], want[name]) <= 2.0 ** -17 + Rr ** 0.5 * E, name


# ====================================================================================== scan
def near(got, want, tol, name):
    """Per head (the axis in front of the last two, the last of 1- and 2-d results): the L2 norm of the
    difference is within tol (an absolute norm, or a number relative to that of `want`)."""
    got = np.asarray(got if isinstance(got, np.ndarray) else got.detach().double().cpu().numpy())
    want = np.asarray(want).reshape(got.shape)
    axes = tuple(i for i in range(got.ndim) if i != (got.ndim - 1 if got.ndim < 3 else got.ndim - 3))
    norm = lambda t: np.sqrt((t * t).sum(axes)) if axes else np.abs(t)  # noqa: E731
    lim = tol * norm(want) if np.ndim(tol) == 0 else tol
    assert np.all(np.isfinite(got)), name
    assert np.all(norm(got - want) <= lim + 1e-30), (name, norm(got - want), lim)


def step_gradients(g, want, a, io, softplus, lens, dy, dST):
    """ddt, dA and ddt_bias within the norms of tests/step_gradient_bounds.py."""
    lim = bounds(a, io, softplus, lens, dy, dST)
    H = a["A"].size
    near(g["ddt"].reshape(-1, H), want["ddt"].reshape(-1, H), lim["ddt"], "ddt")
    near(g["dA"], want["dA"], lim["dA"], "dA")
    if g["ddt_bias"] is not None:
        near(g["ddt_bias"], want["ddt_bias"], lim["ddt_bias"], "ddt_bias")


RESETS = [  # io, lens, packed, H, G, Dk, Dv
    ("bf16", [300], False, 2, 1, 64, 64),
    ("bf16", [5, 300, 64], True, 2, 2, 128, 64),
    ("bf16", [1100], False, 2, 1, 64, 128),     # cut into segments
    ("bf16", [3200], False, 2, 1, 64, 64),      # ... in the backward pass too
    ("f32", [300], False, 2, 1, 64, 64),
]


@pytest.mark.parametrize("io,lens,packed,H,G,Dk,Dv", RESETS)
@pytest.mark.parametrize("every", [True, False])
@pytest.mark.parametrize("dt", [40.0, 1e3, 1e4])
def test_scan_behind_tokens_that_forget(osdn, io, lens, packed, H, G, Dk, Dv, every, dt):  # noqa: F811
    """Tokens with steps of 40 to 10,000 (log2 decays down to -230,000 for one head, -1 to -290 for the
    other): what follows them decays among itself as if they were not there.  One such token in every
    16, or one 10 tokens before the end.  bf16 states come from values as two bf16 terms (2^-17 at
    most) and two exponentials (2^-22 each); dS0 from three terms and as many exponentials as chunks."""
    a, rng = scan_inputs(io, lens, H, G, Dk, Dv, True, True, True, True, seed=31)
    a["A"][:] = rounded([-16.0, -0.02], "f32")
    if every:
        a["dt"][1::16] = dt
    else:
        a["dt"][-10] = dt
    dy = rounded(rng.standard_normal(a["x"].shape), io)
    dST = rounded(0.3 * rng.standard_normal(a["S0"].shape), "f32")
    want = scan_ref(a, True, lens, dy=dy, dST=dST)
    t = scan_dev(a, io, lens, packed)
    y, ST = scan_fwd(osdn, t)
    g = scan_bwd(osdn, t, dev(dy, io).reshape(t["x"].shape), dev(dST))
    finish(osdn)
    near(ST, want["ST"], 2.0 ** -17 + 2.0 ** -20 if io == "bf16" else 2 * relative_error(io, max(lens)), "ST")
    near(g["dS0"], want["dS0"], 2.0 ** -19 if io == "bf16" else 2 * relative_error(io, max(lens)), "dS0")
    for name in ("dx", "db", "dc"):  # the result's own rounding, and two bf16 terms' 2^-16
        l2 = relative_l2(g[name], want[name])
        assert l2 <= (2.0 ** -8 + 2.0 ** -14 if io == "bf16" else 2 * relative_error(io, max(lens))), (name, l2)
    step_gradients(g, want, a, io, True, lens, dy, dST)


# Rounding a value x in [2^e, 2^(e+1)) to bf16 is off by up to 2^-8 2^e, evenly: in L2 norm 2^-8 / sqrt(3)
# times the root of sum 2^2e / sum x^2: 1.53e-3 for values spread evenly in log x, 1.66e-3 for normal ones.
# What else a kernel adds stays below what a second rounding of that size would (2.35e-3 together).
ROUNDED = 1.9e-3


@pytest.mark.parametrize("case", SCANS, ids=lambda s: f"{s[0]}-{'.'.join(map(str, s[1]))}-H{s[3]}G{s[4]}k{s[5]}v{s[6]}")
@pytest.mark.parametrize("kind", ["plain", "slow", "extreme"])
def test_scan_gradients_by_norm(osdn, case, kind):  # noqa: F811
    """Every gradient in L2 norm: dx, db, dc to their own rounding, the step gradients within the norms
    of tests/step_gradient_bounds.py, which zeros and gradients without the <G, S> terms fail
    (tests/test_step_gradient_bounds.py).  slow: states that hardly decay.  extreme: masked tokens
    (dt = -inf), tokens that forget, a head that never decays."""
    io, lens, packed, H, G, Dk, Dv, D, bias, state, softplus = case
    a, rng = scan_inputs(io, lens, H, G, Dk, Dv, D, bias, state, softplus, seed=41)
    n, N = sum(lens), len(lens)
    if kind == "slow":
        a["A"][:] = rounded(-np.geomspace(0.002, 0.05, H), "f32")
    if kind == "extreme":
        if softplus:
            a["dt"][3:8] = -np.inf
        a["dt"][n // 2] = 40.0
        a["A"][-1] = 0.0
    dy = rounded(rng.standard_normal((n, H, Dv)), io)
    dST = rounded(0.3 * rng.standard_normal((N, H, Dv, Dk)), "f32") if state else None
    with np.errstate(invalid="ignore"):
        want = scan_ref(a, softplus, lens, dy=dy, dST=dST)
    t = scan_dev(a, io, lens, packed)
    g = scan_bwd(osdn, t, dev(dy, io).reshape(t["x"].shape), dev(dST), softplus)
    finish(osdn)
    for name in ("dx", "db", "dc"):
        l2 = relative_l2(g[name], want[name])
        assert l2 <= (ROUNDED if io == "bf16" else 2 * relative_error(io, max(lens))), (name, l2)
    step_gradients(g, want, a, io, softplus, lens, dy, dST)


@pytest.mark.parametrize("io,lens", [("bf16", [150, 150]), ("bf16", [3200]), ("f32", [90, 90])])
@pytest.mark.parametrize("given", ["S0", "dST"])
def test_step_gradients_with_one_of_the_states(osdn, io, lens, given):  # noqa: F811
    a, rng = scan_inputs(io, lens, 2, 1, 64, 64, True, True, given == "S0", True, seed=43)
    a["A"][:] = rounded([-0.01, -4.0], "f32")
    dy = rounded(rng.standard_normal(a["x"].shape), io)
    dST = rounded(rng.standard_normal((len(lens), 2, 64, 64)), "f32") if given == "dST" else None
    want = scan_ref(a, True, lens, dy=dy, dST=dST)
    t = scan_dev(a, io, lens, False)
    g = scan_bwd(osdn, t, dev(dy, io).reshape(t["x"].shape), dev(dST))
    finish(osdn)
    step_gradients(g, want, a, io, True, lens, dy, dST)


# two more: chunks alone, with no state in front of them
ALONE = [("bf16", [128, 128], False, 4, 2, 128, 128, False, True, False, True),
         ("bf16", [100, 5, 61], True, 2, 1, 64, 128, False, True, False, True)]


@pytest.mark.parametrize("case", [s for s in SCANS if s[0] == "bf16"] + ALONE,
                         ids=lambda s: f"{'.'.join(map(str, s[1]))}-H{s[3]}G{s[4]}k{s[5]}v{s[6]}")
@pytest.mark.parametrize("forget", [False, True])
def test_scan_outputs_by_norm(osdn, case, forget):  # noqa: F811
    """y in L2 norm, without D (which would make up most of y), and ST to the two bf16 terms of the
    values it is a sum of.  Within a chunk y is as good as its own rounding.  What an earlier state adds
    is a sum over key channels of elements rounded to bf16 each, independently: relative to that part of
    y another 1.66e-3 (as ROUNDED above), and sqrt(1.66^2 + 1.66^2) = 2.35e-3 together where it is all
    of y; 2.5e-3 leaves both 6%.  forget: one token dominates those behind it."""
    io, lens, packed, H, G, Dk, Dv, _, bias, state, softplus = case
    a, rng = scan_inputs(io, lens, H, G, Dk, Dv, False, bias, state, softplus, seed=44)
    if forget:
        a["dt"][sum(lens) // 3] = 1e3
    want = scan_ref(a, softplus, lens)
    y, ST = scan_fwd(osdn, scan_dev(a, io, lens, packed), softplus)
    finish(osdn)
    assert relative_l2(y, want["y"]) <= (2.5e-3 if state or max(lens) > 128 else ROUNDED)
    near(ST, want["ST"], 2.0 ** -17 + 2.0 ** -20, "ST")


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_scan_of_tokens_that_are_not_finite(osdn, io, bad):  # noqa: F811
    """What a later token of the same sequence holds does not reach y: b, c and dt not at all, x (of
    bf16 tokens) only its own head and value channel, within its chunk of 128 tokens."""
    H, G, D, at, v = 2, 1, 64, 150, 5
    a, _ = scan_inputs(io, [300], H, G, D, D, True, True, True, True, seed=51)
    t = scan_dev(a, io, [300], False)
    y0, _ = scan_fwd(osdn, t)
    for name in ("b", "c", "dt"):
        u = dict(t, **{name: t[name].clone()})
        u[name][0, at, 0] = bad
        y1, _ = scan_fwd(osdn, u)
        assert torch.equal(y1[:, :at], y0[:, :at]), name
        assert not torch.isfinite(y1[:, at, 0].float()).all(), name
    u = dict(t, x=t["x"].clone())
    u["x"][0, at, 1, v] = bad
    y1, _ = scan_fwd(osdn, u)
    finish(osdn)
    clean = 128 if io == "bf16" else at
    assert torch.equal(y1[:, :clean], y0[:, :clean])
    assert not torch.isfinite(y1[:, at:, 1, v].float()).any()
    y1[0, clean:, 1, v] = y0[0, clean:, 1, v]
    assert torch.equal(y1, y0)


@pytest.mark.parametrize("T", [1100, 3200])
def test_scan_of_one_sequence_with_offsets(osdn, T):  # noqa: F811
    """Offsets that say what the shape says: the same segments, the same bits."""
    a, rng = scan_inputs("bf16", [T], 2, 1, 64, 64, True, True, True, True, seed=52)
    t, p = scan_dev(a, "bf16", [T], False), scan_dev(a, "bf16", [T], True)
    dy = dev(rng.standard_normal(t["x"].shape), "bf16")
    for x, y in zip(scan_fwd(osdn, t), scan_fwd(osdn, p)):
        assert torch.equal(x, y)
    g, h = scan_bwd(osdn, t, dy), scan_bwd(osdn, p, dy)
    finish(osdn)
    assert all(torch.equal(g[k], h[k]) for k in g)
