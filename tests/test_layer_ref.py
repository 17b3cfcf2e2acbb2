"""The 64-bit statements of the layer operators (tests/layer_ref.py): their gradients against
central differences of their own forward values, and their state chaining."""
import numpy as np
import pytest

from tests import layer_ref as R

STEP = 1e-6
# central differences in 64 bits: truncation ~ STEP^2 times third derivatives of order one, and
# rounding ~ 1e-16 / STEP times the loss (|loss| < 1e3 here): 1e-7 bounds both
TOL = 1e-6


def check(value, arrays, grads):
    """value(arrays) -> loss; grads by name against central differences at a few elements."""
    rng = np.random.default_rng(0)
    for name, g in grads.items():
        a = arrays[name]
        for i in rng.choice(a.size, min(6, a.size), replace=False):
            idx = np.unravel_index(i, a.shape)
            keep = a[idx]
            a[idx] = keep + STEP
            hi = value()
            a[idx] = keep - STEP
            lo = value()
            a[idx] = keep
            want = (hi - lo) / (2 * STEP)
            assert abs(g[idx] - want) <= TOL * max(1.0, abs(want), np.abs(g).max()), (name, idx)


@pytest.mark.parametrize("silu", [False, True])
def test_conv_gradient(silu):
    rng = np.random.default_rng(1)
    lens, C, W = [5, 0, 1, 7], 3, 4
    a = dict(x=rng.standard_normal((13, C)), weight=rng.standard_normal((C, W)),
             bias=rng.standard_normal(C), state0=rng.standard_normal((4, W - 1, C)))
    dy, dst = rng.standard_normal((13, C)), rng.standard_normal((4, W - 1, C))

    def loss():
        o = R.conv(a["x"], a["weight"], a["bias"], a["state0"], silu, lens)
        return (o["y"] * dy).sum() + (o["stateT"] * dst).sum()

    o = R.conv(a["x"], a["weight"], a["bias"], a["state0"], silu, lens, dy, dst)
    check(loss, a, dict(x=o["dx"], weight=o["dweight"], bias=o["dbias"], state0=o["dstate0"]))


@pytest.mark.parametrize("use_softplus", [False, True])
def test_scan_gradient(use_softplus):
    rng = np.random.default_rng(2)
    lens, H, G, Dk, Dv = [4, 0, 1, 6], 4, 2, 3, 2
    n = sum(lens)
    a = dict(x=rng.standard_normal((n, H, Dv)), dt=rng.uniform(0.1, 0.8, (n, H)),
             A=-rng.uniform(0.2, 2, H), b=rng.standard_normal((n, G, Dk)),
             c=rng.standard_normal((n, G, Dk)), D=rng.standard_normal(H),
             dt_bias=rng.standard_normal(H), S0=rng.standard_normal((4, H, Dv, Dk)))
    dy, dST = rng.standard_normal((n, H, Dv)), rng.standard_normal((4, H, Dv, Dk))

    def run(**kw):
        return R.scan(a["x"], a["dt"], a["A"], a["b"], a["c"], a["D"], a["dt_bias"], use_softplus,
                      a["S0"], lens, **kw)

    def loss():
        o = run()
        return (o["y"] * dy).sum() + (o["ST"] * dST).sum()

    o = run(dy=dy, dST=dST)
    check(loss, a, {k: o["d" + k] for k in a})


@pytest.mark.parametrize("gate_first", [False, True])
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("post,res,nxt", [(True, True, True), (True, False, False),
                                          (False, True, True), (False, False, False)])
def test_norm_gradient(gate_first, act, post, res, nxt):
    rng = np.random.default_rng(3)
    Rr, D = 4, 5
    a = dict(f=rng.standard_normal((Rr, D)), gate=rng.standard_normal((Rr, D)))
    if res:
        a["x"] = rng.standard_normal((Rr, D))
    if post:
        a["w_post"] = rng.standard_normal(D)
    if nxt:
        a["w_next"] = rng.standard_normal(D)
    dxo, dh = rng.standard_normal((Rr, D)), rng.standard_normal((Rr, D)) if nxt else None

    def run(*g):
        return R.norm(a["f"], a.get("x"), a["gate"], a.get("w_post"), a.get("w_next"), act,
                      gate_first, 0.7, 1e-5, *g)

    def loss():
        o = run()
        return (o["x_out"] * dxo).sum() + ((o["h"] * dh).sum() if nxt else 0.0)

    o = run(dxo, dh)
    names = dict(f="df", gate="dgate", x="dx", w_post="dw_post", w_next="dw_next")
    check(loss, a, {k: o[names[k]] for k in a})


def test_states_chain():
    rng = np.random.default_rng(4)
    C, W = 3, 4
    x, w = rng.standard_normal((9, C)), rng.standard_normal((C, W))
    whole = R.conv(x, w, None, None, True, [9])
    first = R.conv(x[:2], w, None, None, True, [2])
    rest = R.conv(x[2:], w, None, first["stateT"], True, [7])
    np.testing.assert_allclose(np.concatenate([first["y"], rest["y"]]), whole["y"], rtol=1e-13)
    np.testing.assert_array_equal(rest["stateT"], whole["stateT"])
