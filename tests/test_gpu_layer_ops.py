"""The layer operators around the mixer on the GPU (short causal convolution, selective scan,
block norm; prompts, single tokens, gradients) against their 64-bit statements.

Tolerances, per element.  U is half a rounding step of the stored type (bf16 2^-8, fp32 2^-24,
relative), E = 2^-24 that of fp32 arithmetic, and M the sum of the magnitudes of the terms that
make up the element (the 64-bit statement run on absolute values): an fp32 evaluation with k
roundings on the way to a term is off by at most k E M.
  conv   k <= 80: W + 2 fused multiply-adds, and silu through e^z and a fast division, whose
         documented errors are 2 + 1.2 |z| and 2 units in the last place (|z| < 20 here).
  scan   k = 4 T + Dk + 64: four roundings per token that a state passes, and a dot product.  With
         bf16 tokens the scores and the state enter a product rounded to bf16 (2^-8 each), and
         what leads to fp32 results as two bf16 terms (2^-16 each): y, dx, db, dc add 3 * 2^-8 M,
         states and step gradients 4 * 2^-16 M.
  norm   k <= 64 + D against the largest magnitude of the row.
"""
import numpy as np
import pytest
import torch

from tests import layer_ref as R

pytestmark = pytest.mark.gpu

U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
E = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def osdn():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.set_device(0)
    from delta_rule_recurrent_osdn_b200 import osdn as m
    return m


def dev(a, io="f32"):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(
        "cuda", DT[io])


def host(t):
    return None if t is None else t.detach().float().cpu().numpy().astype(np.float64)


def rounded(a, io):
    return host(dev(a, io)) if a is not None else None


def close(got, want, tol, name):
    got = host(got) if isinstance(got, torch.Tensor) else got
    want = np.asarray(want).reshape(got.shape)
    tol = np.broadcast_to(np.asarray(tol), want.size and np.shape(tol) or ()).reshape(
        got.shape) if np.size(tol) > 1 else tol
    assert np.all(np.isfinite(got)), name
    bad = np.abs(got - want) - tol
    assert not got.size or bad.max() <= 1e-30, (name, bad.max(), np.unravel_index(bad.argmax(), bad.shape))


def offsets(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32), device="cuda")


def finish(osdn):
    torch.cuda.synchronize()
    assert osdn.osdn_get_device_status() == osdn.OSDN_OK


# =============================================================================== convolution
CONVS = [  # io, lens, packed, C, W, bias, state, silu
    ("bf16", [1], False, 8, 4, True, True, True),
    ("bf16", [3, 3], False, 64, 4, False, False, True),
    ("bf16", [70, 70, 70], False, 264, 4, True, True, True),
    ("bf16", [5, 0, 1, 2, 130, 33, 0], True, 128, 4, True, True, True),
    ("bf16", [5, 0, 1, 2, 130, 33, 0], True, 132, 3, False, True, False),
    ("bf16", [17, 2, 41], True, 77, 2, True, False, True),
    ("f32", [257], False, 516, 4, True, True, True),
    ("f32", [2, 1, 0, 64, 9], True, 1001, 3, True, True, True),
    ("f32", [31, 1], True, 20, 2, False, True, False),
    ("f32", [4, 4], False, 3, 4, True, True, True),
]


def conv_inputs(io, lens, C, W, bias, state, seed=0):
    rng = np.random.default_rng(seed)
    n = sum(lens)
    a = dict(x=rounded(rng.standard_normal((n, C)), io),
             weight=rounded(rng.standard_normal((C, W)) * W ** -0.5, "f32"),
             bias=rounded(0.3 * rng.standard_normal(C), "f32") if bias else None,
             state0=rounded(rng.standard_normal((len(lens), W - 1, C)), io) if state else None)
    return a, rng


def lead(lens, packed):
    return (1, sum(lens)) if packed else (len(lens), lens[0])


@pytest.mark.parametrize("io,lens,packed,C,W,bias,state,silu", CONVS)
def test_conv_fwd(osdn, io, lens, packed, C, W, bias, state, silu):
    a, _ = conv_inputs(io, lens, C, W, bias, state)
    args = (a["x"], a["weight"], a["bias"], a["state0"], silu, lens)
    want, mag = R.conv(*args), R.conv(*args, absolute=True)
    y, st = osdn.osdn_conv_fwd(dev(a["x"], io).reshape(*lead(lens, packed), C), dev(a["weight"]),
                               dev(a["bias"]), dev(a["state0"], io), "silu" if silu else None,
                               offsets(lens) if packed else None)
    finish(osdn)
    close(y.reshape(-1, C), want["y"], U[io] * np.abs(want["y"]) + 80 * E * mag["y"], "y")
    np.testing.assert_array_equal(host(st), want["stateT"])


@pytest.mark.parametrize("io,C,W,bias", [("bf16", 128, 4, True), ("bf16", 77, 3, False),
                                         ("bf16", 12, 2, True), ("f32", 260, 4, True),
                                         ("f32", 5, 3, True)])
def test_conv_steps_are_the_prompt(osdn, io, C, W, bias):
    """Token by token from a state: the same bits as one prompt call, y and state."""
    N, T = 5, 6
    a, rng = conv_inputs(io, [T] * N, C, W, bias, True, seed=1)
    x, w, bs = dev(a["x"], io).reshape(N, T, C), dev(a["weight"]), dev(a["bias"])
    y, st = osdn.osdn_conv_fwd(x, w, bs, dev(a["state0"], io))
    state = dev(a["state0"], io)
    for t in range(T):
        got = osdn.osdn_conv_step(x[:, t].clone(), w, state, bs)
        assert torch.equal(got, y[:, t]), t
    finish(osdn)
    assert torch.equal(state, st)


@pytest.mark.parametrize("io,lens,packed,C,W,bias,state,silu", CONVS)
@pytest.mark.parametrize("dy_io", ["same", "f32"])
def test_conv_bwd(osdn, io, lens, packed, C, W, bias, state, silu, dy_io):
    gio = io if dy_io == "same" else "f32"
    a, rng = conv_inputs(io, lens, C, W, bias, state, seed=2)
    n, N = sum(lens), len(lens)
    dy = rounded(rng.standard_normal((n, C)), gio)
    dst = rounded(rng.standard_normal((N, W - 1, C)), "f32") if state else None
    args = (a["x"], a["weight"], a["bias"], a["state0"], silu, lens, dy, dst)
    want, mag = R.conv(*args), R.conv(*args, absolute=True)
    shape = (*lead(lens, packed), C)
    g = osdn.osdn_conv_bwd(dev(a["x"], io).reshape(shape), dev(a["weight"]),
                           dev(dy, gio).reshape(shape), dev(a["bias"]), dev(a["state0"], io),
                           dev(dst), "silu" if silu else None, offsets(lens) if packed else None)
    finish(osdn)
    close(g["dx"].reshape(-1, C), want["dx"], U[io] * np.abs(want["dx"]) + 80 * E * mag["dx"], "dx")
    close(g["dweight"], want["dweight"], (80 + n) * E * mag["dweight"], "dweight")
    assert (g["dbias"] is None) == (not bias) and (g["dstate0"] is None) == (not state)
    if bias:
        close(g["dbias"], want["dbias"], (80 + n) * E * mag["dbias"], "dbias")
    if state:
        close(g["dstate0"], want["dstate0"], 80 * E * mag["dstate0"], "dstate0")


def test_conv_keeps_sequences_apart(osdn):
    """Inf and NaN in one packed sequence stay there, forward and backward."""
    lens, C, W = [40, 50, 3, 60], 64, 4
    a, rng = conv_inputs("bf16", lens, C, W, True, True, seed=3)
    x = dev(a["x"], "bf16").reshape(1, -1, C)
    dy = torch.randn_like(x)
    for n, bad in ((1, float("nan")), (2, float("inf"))):
        lo = sum(lens[:n])
        z, dz = x.clone(), dy.clone()
        z[:, lo:lo + lens[n]] = bad
        dz[:, lo:lo + lens[n]] = bad
        args = dev(a["weight"]), dev(a["bias"]), dev(a["state0"], "bf16")
        y0, _ = osdn.osdn_conv_fwd(x, *args, cu_seqlens=offsets(lens))
        y1, _ = osdn.osdn_conv_fwd(z, *args, cu_seqlens=offsets(lens))
        g0 = osdn.osdn_conv_bwd(x, args[0], dy, *args[1:], cu_seqlens=offsets(lens))
        g1 = osdn.osdn_conv_bwd(z, args[0], dz, *args[1:], cu_seqlens=offsets(lens))
        keep = torch.ones(sum(lens), dtype=torch.bool, device="cuda")
        keep[lo:lo + lens[n]] = False
        assert torch.equal(y0[:, keep], y1[:, keep])
        assert torch.equal(g0["dx"][:, keep], g1["dx"][:, keep])
    finish(osdn)


# ====================================================================================== scan
SCANS = [  # io, lens, packed, H, G, Dk, Dv, D, bias, state, softplus
    ("f32", [1], False, 1, 1, 64, 64, True, True, True, True),
    ("f32", [65, 65], False, 2, 2, 128, 64, True, True, False, True),
    ("f32", [5, 1, 130, 0, 64, 17], True, 4, 2, 64, 128, True, True, True, True),
    ("f32", [200], False, 3, 1, 128, 128, False, False, True, False),
    # long enough for the few heads that sequences are cut into segments
    ("f32", [300, 300], False, 2, 1, 64, 128, True, True, True, True),
    ("f32", [5, 400, 0, 129, 128, 1], True, 2, 2, 128, 64, True, True, True, True),
    ("bf16", [1], False, 1, 1, 128, 128, True, True, True, True),
    ("bf16", [127, 127], False, 2, 1, 128, 128, True, True, False, True),
    ("bf16", [128], False, 2, 2, 64, 64, False, True, True, True),
    ("bf16", [129, 129], False, 3, 3, 128, 64, True, False, True, False),
    ("bf16", [5, 1, 300, 0, 64, 129, 2], True, 4, 2, 64, 128, True, True, True, True),
    ("bf16", [3, 257, 0, 0, 128, 1], True, 4, 1, 128, 128, True, True, True, True),
    ("bf16", [40, 1, 200], True, 6, 3, 64, 64, True, True, False, True),
    ("bf16", [600], False, 2, 1, 128, 64, True, True, True, True),
    # long enough for the few heads that sequences are cut into segments
    ("bf16", [1100], False, 2, 1, 64, 128, True, True, True, True),
    ("bf16", [1400, 3, 0, 512, 200], True, 2, 2, 128, 64, True, True, True, True),
    ("bf16", [1, 1025], True, 3, 1, 128, 128, False, True, False, True),
    # ... in the backward pass too
    ("bf16", [3200], False, 1, 1, 128, 64, True, True, True, True),
    ("bf16", [3109], True, 2, 1, 64, 64, True, True, True, True),
    ("bf16", [3081, 3081], False, 1, 1, 64, 128, False, True, False, True),
]
SCAN_IDS = [f"{s[0]}-{'.'.join(map(str, s[1]))}-H{s[3]}G{s[4]}k{s[5]}v{s[6]}" for s in SCANS]


def scan_inputs(io, lens, H, G, Dk, Dv, D, bias, state, softplus, seed=0):
    rng = np.random.default_rng(seed)
    n, N = sum(lens), len(lens)
    f = "f32"
    a = dict(x=rounded(rng.standard_normal((n, H, Dv)), io),
             dt=rounded(0.5 * rng.standard_normal((n, H)) if softplus else
                        rng.uniform(0.0, 0.2, (n, H)), f),
             A=rounded(-rng.uniform(0.5, 16.0, H), f),
             b=rounded(0.5 * rng.standard_normal((n, G, Dk)), io),
             c=rounded(0.5 * rng.standard_normal((n, G, Dk)), io),
             D=rounded(1 + 0.1 * rng.standard_normal(H), f) if D else None,
             dt_bias=rounded(rng.uniform(-6, -2, H), f) if bias and softplus else None,
             S0=rounded(0.5 * rng.standard_normal((N, H, Dv, Dk)), f) if state else None)
    return a, rng


def scan_ref(a, softplus, lens, **kw):
    return R.scan(a["x"], a["dt"], a["A"], a["b"], a["c"], a["D"], a["dt_bias"], softplus, a["S0"],
                  lens, **kw)


def scan_dev(a, io, lens, packed):
    ld = lead(lens, packed)
    t = {k: dev(a[k], io) for k in ("x", "b", "c")}
    t = {k: v.reshape(*ld, *v.shape[1:]) for k, v in t.items()}
    t["dt"] = dev(a["dt"]).reshape(*ld, -1)
    t.update({k: dev(a[k]) for k in ("A", "D", "dt_bias", "S0")})
    t["cu"] = offsets(lens) if packed else None
    return t


def scan_fwd(osdn, t, softplus=True, **kw):
    return osdn.osdn_ssm_fwd(t["x"], t["dt"], t["A"], t["b"], t["c"], t["D"], t["dt_bias"], softplus,
                             t["S0"], t["cu"], **kw)


def scan_bwd(osdn, t, dy, dST=None, softplus=True, **kw):
    return osdn.osdn_ssm_bwd(t["x"], t["dt"], t["A"], t["b"], t["c"], dy, t["D"], t["dt_bias"],
                             softplus, t["S0"], dST, t["cu"], **kw)


def scan_factors(io, lens, Dk):
    k = (4 * max(lens) + Dk + 64) * E
    return (k + 3 * 2.0 ** -8, k + 4 * 2.0 ** -16) if io == "bf16" else (k, k)


@pytest.mark.parametrize("io,lens,packed,H,G,Dk,Dv,D,bias,state,softplus", SCANS, ids=SCAN_IDS)
def test_scan_fwd(osdn, io, lens, packed, H, G, Dk, Dv, D, bias, state, softplus):
    a, _ = scan_inputs(io, lens, H, G, Dk, Dv, D, bias, state, softplus)
    want, mag = scan_ref(a, softplus, lens), scan_ref(a, softplus, lens, absolute=True)
    y, ST = scan_fwd(osdn, scan_dev(a, io, lens, packed), softplus)
    finish(osdn)
    coarse, fine = scan_factors(io, lens, Dk)
    close(y.reshape(want["y"].shape), want["y"], U[io] * np.abs(want["y"]) + coarse * mag["y"], "y")
    close(ST, want["ST"], fine * mag["ST"], "ST")


@pytest.mark.parametrize("io,lens,packed,H,G,Dk,Dv,D,bias,state,softplus", SCANS, ids=SCAN_IDS)
def test_scan_bwd(osdn, io, lens, packed, H, G, Dk, Dv, D, bias, state, softplus):
    a, rng = scan_inputs(io, lens, H, G, Dk, Dv, D, bias, state, softplus, seed=1)
    n, N = sum(lens), len(lens)
    dy = rounded(rng.standard_normal((n, H, Dv)), io)
    dST = rounded(0.3 * rng.standard_normal((N, H, Dv, Dk)), "f32") if state else None
    want = scan_ref(a, softplus, lens, dy=dy, dST=dST)
    mag = scan_ref(a, softplus, lens, dy=dy, dST=dST, absolute=True)
    t = scan_dev(a, io, lens, packed)
    g = scan_bwd(osdn, t, dev(dy, io).reshape(t["x"].shape), dev(dST), softplus)
    finish(osdn)
    coarse, fine = scan_factors(io, lens, max(Dk, Dv))
    for name in ("dx", "db", "dc"):
        close(g[name].reshape(want[name].shape), want[name],
              U[io] * np.abs(want[name]) + coarse * mag[name], name)
    step = (np.abs(a["A"]) * mag["cancel"] + mag["ddt"]) * fine
    close(g["ddt"].reshape(n, H), want["ddt"], step, "ddt")
    close(g["dA"], want["dA"], fine * (mag["reach"] + mag["dA"]), "dA")
    for name, inp, tol in (("dD", "D", (n + Dv) * E * mag["dD"]), ("ddt_bias", "dt_bias", step.sum(0)),
                           ("dS0", "S0", fine * mag["dS0"])):
        assert (g[name] is None) == (a[inp] is None)
        if a[inp] is not None:
            close(g[name], want[name], tol, name)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("N,H,G,Dk,Dv,D", [(1, 1, 1, 64, 64, True), (5, 6, 2, 128, 64, False),
                                           (3, 4, 4, 64, 128, True), (2, 3, 1, 128, 128, True)])
def test_scan_steps(osdn, io, N, H, G, Dk, Dv, D):
    T = 4
    a, _ = scan_inputs(io, [T] * N, H, G, Dk, Dv, D, True, True, True, seed=2)
    want = scan_ref(a, True, [T] * N)
    mag = scan_ref(a, True, [T] * N, absolute=True)
    t = scan_dev(a, io, [T] * N, False)
    S = t["S0"].clone()
    ys = [osdn.osdn_ssm_step(*(t[k][:, i].clone() for k in ("x", "dt")), t["A"],
                             *(t[k][:, i].clone() for k in ("b", "c")), S, t["D"], t["dt_bias"])
          for i in range(T)]
    finish(osdn)
    y = host(torch.stack(ys, 1)).reshape(want["y"].shape)
    k = (4 * T + Dk + 64) * E
    close(y, want["y"], U[io] * np.abs(want["y"]) + k * mag["y"], "y")
    close(S, want["ST"], k * mag["ST"], "S")


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_scan_chains_through_states(osdn, io):
    """Two halves joined by the state against the whole, within the tolerance of each side."""
    T, cut, H, G, Dk, Dv = 333, 150, 2, 1, 128, 64
    a, _ = scan_inputs(io, [T], H, G, Dk, Dv, True, True, True, True, seed=3)
    mag = scan_ref(a, True, [T], absolute=True)
    t = scan_dev(a, io, [T], False)
    y, ST = scan_fwd(osdn, t)
    u = {k: (v[:, :cut].contiguous() if k in ("x", "b", "c", "dt") else v) for k, v in t.items()}
    y0, S = scan_fwd(osdn, u)
    u = {k: (v[:, cut:].contiguous() if k in ("x", "b", "c", "dt") else v) for k, v in t.items()}
    y1, S1 = scan_fwd(osdn, dict(u, S0=S))
    finish(osdn)
    coarse, fine = scan_factors(io, [T], Dk)
    both = host(torch.cat([y0, y1], 1)).reshape(-1, H, Dv)
    close(both, host(y).reshape(-1, H, Dv), 2 * (U[io] + coarse) * mag["y"], "y")
    close(S1, host(ST), 2 * fine * mag["ST"], "ST")


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_scan_keeps_sequences_apart(osdn, io):
    """NaN and infinities in one packed sequence (a padded batch's leftovers) reach no other."""
    lens, H, G, Dk, Dv = [70, 130, 1, 200], 2, 1, 128, 128
    a, rng = scan_inputs(io, lens, H, G, Dk, Dv, True, True, True, True, seed=4)
    t = scan_dev(a, io, lens, True)
    dy = dev(rng.standard_normal(t["x"].shape), io)
    y0, S0 = scan_fwd(osdn, t)
    g0 = scan_bwd(osdn, t, dy)
    for n, bad in ((1, float("nan")), (2, float("inf")), (0, -float("inf"))):
        lo = sum(lens[:n])
        u = {k: (v.clone() if k in ("x", "b", "c", "dt") else v) for k, v in t.items()}
        dz = dy.clone()
        for v in (u["x"], u["b"], u["c"], u["dt"], dz):
            v[:, lo:lo + lens[n]] = bad
        y1, S1 = scan_fwd(osdn, u)
        g1 = scan_bwd(osdn, u, dz)
        keep = torch.ones(sum(lens), dtype=torch.bool, device="cuda")
        keep[lo:lo + lens[n]] = False
        other = [i for i in range(len(lens)) if i != n]
        assert torch.equal(y0[:, keep], y1[:, keep]) and torch.equal(S0[other], S1[other])
        for k in ("dx", "db", "dc", "ddt"):
            assert torch.equal(g0[k][:, keep], g1[k][:, keep]), k
        assert torch.equal(g0["dS0"][other], g1["dS0"][other])
    finish(osdn)


@pytest.mark.parametrize("io,lens,packed", [("bf16", [1100], False), ("bf16", [700, 900, 1], True),
                                            ("bf16", [3200], False),
                                            ("f32", [150], False), ("f32", [301, 7, 290], True)])
def test_scan_slow_decay(osdn, io, lens, packed):
    """States that hardly decay: what a sequence starts from, and every segment and chunk, reaches
    all of what follows."""
    H, G, Dk, Dv = 2, 1, 64, 64
    a, rng = scan_inputs(io, lens, H, G, Dk, Dv, True, True, True, True, seed=6)
    a["A"][:] = rounded([-0.002, -0.05], "f32")
    a["S0"] *= 8
    dy = rounded(rng.standard_normal(a["x"].shape), io)
    dST = rounded(rng.standard_normal(a["S0"].shape), "f32")
    want = scan_ref(a, True, lens, dy=dy, dST=dST)
    mag = scan_ref(a, True, lens, dy=dy, dST=dST, absolute=True)
    t = scan_dev(a, io, lens, packed)
    y, ST = scan_fwd(osdn, t)
    g = scan_bwd(osdn, t, dev(dy, io).reshape(t["x"].shape), dev(dST))
    finish(osdn)
    coarse, fine = scan_factors(io, lens, Dk)
    close(y.reshape(want["y"].shape), want["y"], U[io] * np.abs(want["y"]) + coarse * mag["y"], "y")
    close(ST, want["ST"], fine * mag["ST"], "ST")
    for name in ("dx", "db", "dc"):
        close(g[name].reshape(want[name].shape), want[name],
              U[io] * np.abs(want[name]) + coarse * mag[name], name)
    close(g["dS0"], want["dS0"], fine * mag["dS0"], "dS0")
    close(g["ddt"].reshape(-1, H), want["ddt"],
          (np.abs(a["A"]) * mag["cancel"] + mag["ddt"]) * fine, "ddt")
    # norms: errors are random, so they stay far below the sums of their bounds
    for got, ref in ((ST, want["ST"]), (g["dS0"], want["dS0"])):
        assert np.linalg.norm(host(got) - ref) <= 1e-5 * np.linalg.norm(ref)
    assert np.linalg.norm(host(y).reshape(-1) - want["y"].reshape(-1)) <= 2.0 ** -8 * np.linalg.norm(want["y"])


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_scan_extreme_steps(osdn, io):
    """Steps of 0 (masked tokens: dt = -inf), steps so large that the state is forgotten, and
    A = 0 (a state that never decays): finite results, equal to the 64-bit ones."""
    lens, H, G, Dk, Dv = [300], 3, 1, 64, 64
    a, rng = scan_inputs(io, lens, H, G, Dk, Dv, True, True, True, True, seed=5)
    a["dt"][10:20] = -np.inf
    a["dt"][130:140] = 40.0
    a["A"][1] = 0.0
    dy = rounded(rng.standard_normal((300, H, Dv)), io)
    with np.errstate(invalid="ignore"):
        want = scan_ref(a, True, lens, dy=dy)
        mag = scan_ref(a, True, lens, dy=dy, absolute=True)
    t = scan_dev(a, io, lens, False)
    y, ST = scan_fwd(osdn, t)
    g = scan_bwd(osdn, t, dev(dy, io).reshape(t["x"].shape))
    finish(osdn)
    coarse, fine = scan_factors(io, lens, Dk)
    close(y.reshape(want["y"].shape), want["y"], U[io] * np.abs(want["y"]) + coarse * mag["y"], "y")
    close(ST, want["ST"], fine * mag["ST"], "ST")
    for name in ("dx", "db", "dc"):
        close(g[name].reshape(want[name].shape), want[name],
              U[io] * np.abs(want[name]) + coarse * mag[name], name)
    close(g["ddt"].reshape(300, H), want["ddt"],
          (np.abs(a["A"]) * mag["cancel"] + mag["ddt"]) * fine, "ddt")


def test_bad_offsets_are_reported(osdn):
    """Offsets out of order: the status word says so, and the sequences that are right are right."""
    C, W = 64, 4
    x = torch.randn(1, 100, C, device="cuda").bfloat16()
    w = torch.randn(C, W, device="cuda")
    good = offsets([30, 40, 30])
    bad = torch.tensor([0, 30, 20, 100], dtype=torch.int32, device="cuda")
    y0, _ = osdn.osdn_conv_fwd(x, w, cu_seqlens=good)
    y1, _ = osdn.osdn_conv_fwd(x, w, cu_seqlens=bad)
    torch.cuda.synchronize()
    assert osdn.osdn_get_device_status() == osdn.OSDN_ERR_DEVICE_BOUNDS
    assert osdn.osdn_get_device_status() == osdn.OSDN_OK
    assert torch.equal(y0[:, :20], y1[:, :20])
    a, _ = scan_inputs("bf16", [100], 2, 1, 64, 64, True, True, False, True)
    t = scan_dev(a, "bf16", [100], True)
    scan_fwd(osdn, dict(t, cu=bad))
    torch.cuda.synchronize()
    assert osdn.osdn_get_device_status() == osdn.OSDN_ERR_DEVICE_BOUNDS
    scan_bwd(osdn, dict(t, cu=bad), torch.randn_like(t["x"]))
    torch.cuda.synchronize()
    assert osdn.osdn_get_device_status() == osdn.OSDN_ERR_DEVICE_BOUNDS


# ====================================================================================== norm
NORMS = [  # io, R, D, gate, gate_first, act, post, res, next
    ("bf16", 1, 1, True, False, "silu", True, True, True),
    ("bf16", 37, 64, True, False, "silu", True, False, False),
    ("bf16", 130, 128, True, True, "silu", True, False, False),
    ("bf16", 9, 100, True, False, "sigmoid", True, True, True),
    ("bf16", 33, 256, False, False, "silu", False, True, True),
    ("bf16", 7, 513, True, True, "sigmoid", True, True, True),
    ("bf16", 20, 2048, True, False, "silu", True, True, True),
    ("bf16", 3, 8192, True, False, "silu", True, True, True),
    ("bf16", 4, 5001, False, False, "silu", True, True, False),
    ("f32", 11, 33, True, False, "silu", True, True, True),
    ("f32", 6, 1000, True, True, "silu", True, True, True),
    ("f32", 5, 4096, False, False, "silu", False, False, True),
    ("f32", 64, 128, True, False, "sigmoid", False, True, False),
    ("f32", 2, 8191, True, False, "silu", True, True, True),
]


def norm_inputs(io, Rr, D, gate, post, res, nxt, seed=0):
    rng = np.random.default_rng(seed)
    return dict(f=rounded(rng.standard_normal((Rr, D)), io),
                x=rounded(2 * rng.standard_normal((Rr, D)), io) if res else None,
                gate=rounded(rng.standard_normal((Rr, D)), io) if gate else None,
                w_post=rounded(1 + 0.1 * rng.standard_normal(D), "f32") if post else None,
                w_next=rounded(1 + 0.1 * rng.standard_normal(D), "f32") if nxt else None), rng


def norm_tol(want, io, D):
    return U[io] * np.abs(want) + (64 + D) * E * 16 * np.abs(want).max(-1, keepdims=True) + 1e-30


@pytest.mark.parametrize("io,Rr,D,gate,first,act,post,res,nxt", NORMS)
def test_norm(osdn, io, Rr, D, gate, first, act, post, res, nxt):
    a, rng = norm_inputs(io, Rr, D, gate, post, res, nxt)
    dxo = rounded(rng.standard_normal((Rr, D)), io)
    dh = rounded(rng.standard_normal((Rr, D)), io) if nxt else None
    scale, eps = 0.7, 1e-5
    want = R.norm(a["f"], a["x"], a["gate"], a["w_post"], a["w_next"], act, first, scale, eps, dxo, dh)
    d = {k: dev(v, "f32" if k.startswith("w") else io) for k, v in a.items()}
    kw = dict(gate_act=act, gate_first=first, scale=scale, eps=eps)
    xo, h = osdn.osdn_norm_fwd(d["f"], d["x"], d["gate"], d["w_post"], d["w_next"], **kw)
    g = osdn.osdn_norm_bwd(d["f"], dev(dxo, io), dev(dh, io), d["x"], d["gate"], d["w_post"],
                           d["w_next"], **kw)
    if nxt:
        none, h2 = osdn.osdn_norm_fwd(d["f"], d["x"], d["gate"], d["w_post"], d["w_next"],
                                      return_x_out=False, **kw)
        assert none is None and torch.equal(h, h2)
    finish(osdn)
    close(xo, want["x_out"], norm_tol(want["x_out"], io, D), "x_out")
    if nxt:
        close(h, want["h"], norm_tol(want["h"], io, D), "h")
    assert (h is None) == (not nxt)
    for name, on in (("df", True), ("dx", res), ("dgate", gate)):
        assert (g[name] is not None) == on
        if on:  # gradients: up to three products per term more than the forward pass
            close(g[name], want[name], 2 * norm_tol(want[name], io, D), name)
    for name, on in (("dw_post", post), ("dw_next", nxt)):
        assert (g[name] is not None) == on
        if on:
            mag = np.sqrt((want[name] ** 2).mean()) + np.abs(want[name])
            close(g[name], want[name], (64 + D + Rr) * E * 16 * (mag + Rr ** 0.5), name)


def test_norm_of_zero_rows_and_zero_tokens(osdn):
    """Rows of zeros give zeros (eps keeps the division finite), and no rows give zero gradients."""
    f = torch.zeros(4, 96, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(96, device="cuda")
    xo, h = osdn.osdn_norm_fwd(f, w_post=w, w_next=w)
    g = osdn.osdn_norm_bwd(f, f, f, w_post=w, w_next=w)
    assert not xo.any() and not h.any() and not g["df"].any() and not g["dw_post"].any()
    e = f[:0]
    g = osdn.osdn_norm_bwd(e, e, e, w_post=w, w_next=w)
    assert not g["dw_post"].any() and not g["dw_next"].any()
    x = torch.zeros(2, 0, 16, device="cuda")
    g = osdn.osdn_conv_bwd(x, torch.ones(16, 4, device="cuda"), x, torch.ones(16, device="cuda"))
    assert not g["dweight"].any() and not g["dbias"].any()
    z = torch.zeros(2, 0, 2, 64, device="cuda")
    A = -torch.ones(2, device="cuda")
    S0 = torch.randn(2, 2, 64, 64, device="cuda")
    y, ST = osdn.osdn_ssm_fwd(z, z[..., 0].contiguous(), A, z, z, S0=S0)
    assert torch.equal(ST, S0)
    g = osdn.osdn_ssm_bwd(z, z[..., 0].contiguous(), A, z, z, z, D=A, S0=S0, dST=S0)
    assert torch.equal(g["dS0"], S0) and not g["dA"].any() and not g["dD"].any()
    finish(osdn)


# ================================================================= streams, graphs, refusals
def test_binding_refuses(osdn):
    x = torch.randn(2, 8, 4, 64, device="cuda").bfloat16()
    w = torch.randn(256, 4, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        osdn.osdn_conv_fwd(x.transpose(1, 2), w)
    with pytest.raises(ValueError, match="shape"):
        osdn.osdn_conv_fwd(x, w[:-1].contiguous())
    with pytest.raises(TypeError):
        osdn.osdn_conv_fwd(x, w.bfloat16())
    with pytest.raises(TypeError):
        osdn.osdn_conv_fwd(x.half(), w)
    with pytest.raises(ValueError, match="activation"):
        osdn.osdn_conv_fwd(x, w, activation="gelu")
    with pytest.raises(TypeError):
        osdn.osdn_conv_bwd(x, w, x.half())
    with pytest.raises(osdn.OsdnError) as e:
        osdn.osdn_conv_fwd(x, torch.randn(256, 5, device="cuda"))
    assert e.value.status == osdn.OSDN_ERR_UNSUPPORTED
    with pytest.raises(osdn.OsdnError) as e:  # in place
        osdn.osdn_conv_fwd(x, w, y=x)
    assert e.value.status == osdn.OSDN_ERR_INVALID_ARG
    b = torch.randn(2, 8, 3, 64, device="cuda").bfloat16()
    dt, A = torch.randn(2, 8, 4, device="cuda"), -torch.ones(4, device="cuda")
    with pytest.raises(osdn.OsdnError) as e:  # 4 heads over 3 groups
        osdn.osdn_ssm_fwd(x, dt, A, b, b)
    assert e.value.status == osdn.OSDN_ERR_INVALID_ARG
    with pytest.raises(ValueError, match="shape"):
        osdn.osdn_ssm_fwd(x, dt, A[:2].contiguous(), x, x)
    with pytest.raises(ValueError, match="h needs"):
        osdn.osdn_norm_fwd(x, h=torch.empty_like(x))
    with pytest.raises(ValueError, match="dh"):
        osdn.osdn_norm_bwd(x, x, x)
    with pytest.raises(ValueError, match="cuda:0|cpu|CUDA"):
        osdn.osdn_norm_fwd(x, x=x.cpu())


def test_calls_by_keyword(osdn):
    t = layer_inputs("bf16", [20], 2, 1, 64, 64, 5)
    want = osdn.osdn_ssm_fwd(t["u"], t["dt"], t["A"], t["b"], t["c"])
    got = osdn.osdn_ssm_fwd(c=t["c"], b=t["b"], A=t["A"], dt=t["dt"], x=t["u"],
                            stream=torch.cuda.current_stream())
    same(got, want)
    with pytest.raises(TypeError, match="dt"):
        osdn.osdn_ssm_fwd(t["u"])


def layer(osdn, t, io, cu=None):
    """A run of the operators as a layer makes it: convolution, scan, gated norm over each head;
    and back.  Returns everything it computes."""
    y, cst = osdn.osdn_conv_fwd(t["u"], t["w"], t["wb"], t["cst"], cu_seqlens=cu)
    o, ST = osdn.osdn_ssm_fwd(y, t["dt"], t["A"], t["b"], t["c"], t["D"], t["dt_bias"], S0=t["S0"],
                              cu_seqlens=cu)
    out, _ = osdn.osdn_norm_fwd(o, gate=t["z"], w_post=t["wn"])
    gn = osdn.osdn_norm_bwd(o, t["dout"], gate=t["z"], w_post=t["wn"])
    gs = osdn.osdn_ssm_bwd(y, t["dt"], t["A"], t["b"], t["c"], gn["df"], t["D"], t["dt_bias"],
                           S0=t["S0"], cu_seqlens=cu)
    gc = osdn.osdn_conv_bwd(t["u"], t["w"], gs["dx"], t["wb"], t["cst"], cu_seqlens=cu)
    return [y, cst, o, ST, out, *gn.values(), *gs.values(), *gc.values()]


def layer_inputs(io, lens, H, G, Dk, Dv, seed):
    rng = np.random.default_rng(seed)
    n, N = sum(lens), len(lens)

    def r(*s, k=1.0, i="f32"):
        return dev(k * rng.standard_normal(s), i)

    return dict(u=r(1, n, H, Dv, i=io), w=r(H * Dv, 4, k=0.5), wb=r(H * Dv, k=0.2),
                cst=r(N, 3, H * Dv, i=io), dt=r(1, n, H, k=0.5) - 3, A=-torch.exp(r(H)),
                b=r(1, n, G, Dk, k=0.5, i=io), c=r(1, n, G, Dk, k=0.5, i=io), D=r(H),
                dt_bias=r(H, k=0.3), S0=r(N, H, Dv, Dk, k=0.3), z=r(1, n, H, Dv, i=io),
                wn=1 + r(Dv, k=0.1), dout=r(1, n, H, Dv, i=io))


def same(xs, ys):
    assert len(xs) == len(ys)
    for i, (x, y) in enumerate(zip(xs, ys)):
        assert (x is None) == (y is None) and (x is None or torch.equal(x, y)), i


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_layer_run_against_64_bits(osdn, io):
    """The operators one after another, each fed with what the one before stored."""
    lens, H, G, Dk, Dv = [130, 3, 0, 77], 4, 2, 128, 64
    t = layer_inputs(io, lens, H, G, Dk, Dv, 7)
    out = layer(osdn, t, io, offsets(lens))
    finish(osdn)
    y, cst, o, ST, res = out[:5]
    h = {k: host(v) for k, v in t.items()}
    n, C = sum(lens), H * Dv
    args = (h["u"].reshape(n, C), h["w"], h["wb"], h["cst"], True, lens)
    want, mag = R.conv(*args), R.conv(*args, absolute=True)
    close(y.reshape(n, C), want["y"], U[io] * np.abs(want["y"]) + 80 * E * mag["y"], "y")
    a = dict(x=host(y).reshape(n, H, Dv), dt=h["dt"][0], A=h["A"], b=h["b"][0], c=h["c"][0], D=h["D"],
             dt_bias=h["dt_bias"], S0=h["S0"])
    want, mag = scan_ref(a, True, lens), scan_ref(a, True, lens, absolute=True)
    coarse, fine = scan_factors(io, lens, Dk)
    close(o.reshape(n, H, Dv), want["y"], U[io] * np.abs(want["y"]) + coarse * mag["y"], "o")
    close(ST, want["ST"], fine * mag["ST"], "ST")
    want = R.norm(host(o).reshape(-1, Dv), None, h["z"].reshape(-1, Dv), h["wn"], None, "silu", False,
                  1.0, 1e-5)
    close(res.reshape(-1, Dv), want["x_out"], norm_tol(want["x_out"], io, Dv), "out")


def test_mixer_between_the_operators(osdn):
    """Short convolutions in front of the OSDN mixer's q, k, v and a gated norm behind its output,
    forward and backward: osdn_bwd's fp32 gradients feed osdn_conv_bwd as they are."""
    B, T, H, D = 2, 150, 2, 128
    g = torch.Generator().manual_seed(3)
    mk = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    raw = [mk(B, T, H, D).bfloat16() for _ in range(3)]
    ws = [0.5 * mk(H * D, 4) for _ in range(3)]
    beta = torch.sigmoid(mk(B, T, H))
    q, k, v = (osdn.osdn_conv_fwd(x, w)[0] for x, w in zip(raw, ws))
    q, k = (torch.nn.functional.normalize(t.float(), dim=-1).bfloat16() for t in (q, k))
    o, _, _ = osdn.osdn_fwd(q, k, v, beta, eta=0.05)
    out, _ = osdn.osdn_norm_fwd(o, gate=raw[0], w_post=torch.ones(D, device="cuda"))
    gn = osdn.osdn_norm_bwd(o, torch.ones_like(o), gate=raw[0], w_post=torch.ones(D, device="cuda"))
    gm = osdn.osdn_bwd(q, k, v, beta, gn["df"], eta=0.05)
    gv = osdn.osdn_conv_bwd(raw[2], ws[2], gm["dv"])
    finish(osdn)
    args = (host(raw[2]).reshape(B * T, -1), host(ws[2]), None, None, True, [T] * B,
            host(gm["dv"]).reshape(B * T, -1))
    want, mag = R.conv(*args), R.conv(*args, absolute=True)
    close(gv["dx"].reshape(B * T, -1), want["dx"],
          U["bf16"] * np.abs(want["dx"]) + 80 * E * mag["dx"], "dv")
    assert out.shape == o.shape and torch.isfinite(out.float()).all()


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_layer_on_another_stream_and_in_graphs(osdn, io):
    """The same bits on a side stream, twice, and from two captured graphs replayed in turn."""
    lens = [130, 3, 0, 300]
    cu = offsets(lens)
    t1, t2 = (layer_inputs(io, lens, 4, 2, 128, 64, s) for s in (8, 9))
    want1, want2 = layer(osdn, t1, io, cu), layer(osdn, t2, io, cu)
    same(layer(osdn, t1, io, cu), want1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = layer(osdn, t1, io, cu)
    side.synchronize()
    same(got, want1)
    y, _ = osdn.osdn_conv_fwd(t1["u"], t1["w"], t1["wb"], t1["cst"], cu_seqlens=cu, stream=side)
    side.synchronize()
    assert torch.equal(y, want1[0])
    graphs = []
    for t in (t1, t2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs = layer(osdn, t, io, cu)
        graphs.append((gr, outs))
    for _ in range(2):
        for (gr, outs), want in zip(graphs, (want1, want2)):
            for o in outs:
                if o is not None:
                    o.zero_()
            gr.replay()
            torch.cuda.synchronize()
            same(outs, want)
    finish(osdn)


def test_two_streams_at_once(osdn):
    lens = [257, 64]
    cu = offsets(lens)
    ts = [layer_inputs("bf16", lens, 4, 1, 64, 128, s) for s in (10, 11)]
    want = [layer(osdn, t, "bf16", cu) for t in ts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ts]
    got = [None, None]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = layer(osdn, ts[i], "bf16", cu)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        same(g, w)
    finish(osdn)


# ============================================================================ what calls may be
@pytest.mark.parametrize("io,lens", [("bf16", [150, 150]), ("bf16", [3200]), ("f32", [90, 90])])
@pytest.mark.parametrize("given", ["S0", "dST"])
def test_scan_bwd_with_one_of_the_states(osdn, io, lens, given):
    H, G, Dk, Dv = 2, 1, 64, 64
    a, rng = scan_inputs(io, lens, H, G, Dk, Dv, True, True, given == "S0", True, seed=9)
    dy = rounded(rng.standard_normal(a["x"].shape), io)
    dST = rounded(rng.standard_normal((len(lens), H, Dv, Dk)), "f32") if given == "dST" else None
    want = scan_ref(a, True, lens, dy=dy, dST=dST)
    mag = scan_ref(a, True, lens, dy=dy, dST=dST, absolute=True)
    t = scan_dev(a, io, lens, False)
    g = scan_bwd(osdn, t, dev(dy, io).reshape(t["x"].shape), dev(dST))
    finish(osdn)
    coarse, fine = scan_factors(io, lens, Dk)
    for name in ("dx", "db", "dc"):
        close(g[name].reshape(want[name].shape), want[name],
              U[io] * np.abs(want[name]) + coarse * mag[name], name)
    close(g["ddt"].reshape(-1, H), want["ddt"],
          (np.abs(a["A"]) * mag["cancel"] + mag["ddt"]) * fine, "ddt")
    assert (g["dS0"] is None) == (given == "dST")
    if given == "S0":
        close(g["dS0"], want["dS0"], fine * mag["dS0"], "dS0")


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_scan_of_growing_states(osdn, io):
    """A > 0, and steps below 0 (no softplus): states grow by up to e^4 over a sequence."""
    lens, H, G, Dk, Dv = [200, 200], 2, 2, 64, 64
    a, rng = scan_inputs(io, lens, H, G, Dk, Dv, True, False, True, False, seed=10)
    a["dt"] = rounded(rng.uniform(-0.1, 0.1, a["dt"].shape), "f32")
    a["dt"][:, 0] = rounded(np.abs(a["dt"][:, 0]), "f32")
    a["A"][:] = rounded([0.4, 0.6], "f32")
    dy = rounded(rng.standard_normal(a["x"].shape), io)
    want = scan_ref(a, False, lens, dy=dy)
    mag = scan_ref(a, False, lens, dy=dy, absolute=True)
    t = scan_dev(a, io, lens, False)
    y, ST = scan_fwd(osdn, t, False)
    g = scan_bwd(osdn, t, dev(dy, io).reshape(t["x"].shape), None, False)
    finish(osdn)
    coarse, fine = scan_factors(io, lens, Dk)
    close(y.reshape(want["y"].shape), want["y"], U[io] * np.abs(want["y"]) + coarse * mag["y"], "y")
    close(ST, want["ST"], fine * mag["ST"], "ST")
    for name in ("dx", "db", "dc"):
        close(g[name].reshape(want[name].shape), want[name],
              U[io] * np.abs(want[name]) + coarse * mag[name], name)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_thousands_of_tiny_sequences(osdn, io):
    """More sequences than the convolution has blocks for them, none of more than two tokens."""
    rng = np.random.default_rng(11)
    lens = [int(v) for v in rng.integers(0, 3, 5000)]
    n, C, W = sum(lens), 64, 4
    a, _ = conv_inputs(io, lens, C, W, True, True)
    args = (a["x"], a["weight"], a["bias"], a["state0"], True, lens)
    want, mag = R.conv(*args), R.conv(*args, absolute=True)
    y, st = osdn.osdn_conv_fwd(dev(a["x"], io).reshape(1, n, C), dev(a["weight"]), dev(a["bias"]),
                               dev(a["state0"], io), "silu", offsets(lens))
    close(y.reshape(-1, C), want["y"], U[io] * np.abs(want["y"]) + 80 * E * mag["y"], "y")
    np.testing.assert_array_equal(host(st), want["stateT"])
    s, _ = scan_inputs(io, lens, 1, 1, 64, 64, True, True, True, True)
    dy = rounded(rng.standard_normal(s["x"].shape), io)
    want, mag = scan_ref(s, True, lens, dy=dy), scan_ref(s, True, lens, dy=dy, absolute=True)
    t = scan_dev(s, io, lens, True)
    y, ST = scan_fwd(osdn, t)
    g = scan_bwd(osdn, t, dev(dy, io).reshape(t["x"].shape))
    finish(osdn)
    coarse, fine = scan_factors(io, lens, 64)
    close(y.reshape(want["y"].shape), want["y"], U[io] * np.abs(want["y"]) + coarse * mag["y"], "y")
    close(ST, want["ST"], fine * mag["ST"], "ST")
    for name in ("dx", "db", "dc"):
        close(g[name].reshape(want[name].shape), want[name],
              U[io] * np.abs(want[name]) + coarse * mag[name], name)


def test_offsets_past_32_bits(osdn):
    """Tensors of more than 2^31 values: the last head, channels and rows are those of a call on
    them alone (the scan's to bf16 rounding: its chains are cut elsewhere)."""
    T, H, Dv, Dk = 66000, 256, 128, 64
    g = torch.Generator(device="cuda").manual_seed(12)
    draw = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    x = draw(1, T, H, Dv)
    assert x.numel() > 2 ** 31
    w = torch.randn(H * Dv, 4, generator=g, device="cuda")
    last = lambda t: t[:, :, -1:].clone()  # noqa: E731
    y, st = osdn.osdn_conv_fwd(x, w)
    y1, st1 = osdn.osdn_conv_fwd(last(x), w[-Dv:].clone())
    assert torch.equal(last(y), y1) and torch.equal(st[..., -Dv:], st1)
    del y
    dy = draw(1, T, H, Dv)
    c = osdn.osdn_conv_bwd(x, w, dy)
    c1 = osdn.osdn_conv_bwd(last(x), w[-Dv:].clone(), last(dy))
    assert torch.equal(last(c["dx"]), c1["dx"])
    err = (c["dweight"][-Dv:] - c1["dweight"]).norm() / c1["dweight"].norm()
    assert err <= T * E
    del c
    u, _ = osdn.osdn_norm_fwd(x, gate=dy, w_post=torch.ones(Dv, device="cuda"))
    u1, _ = osdn.osdn_norm_fwd(last(x), gate=last(dy), w_post=torch.ones(Dv, device="cuda"))
    assert torch.equal(last(u), u1)
    del u
    b, cc = 0.2 * draw(1, T, 1, Dk), 0.2 * draw(1, T, 1, Dk)
    dt, A = torch.randn(1, T, H, generator=g, device="cuda") - 3, torch.full((H,), -4.0, device="cuda")
    o, ST = osdn.osdn_ssm_fwd(x, dt, A, b, cc)
    o1, ST1 = osdn.osdn_ssm_fwd(last(x), last(dt), A[-1:].clone(), b, cc)
    near = lambda p, q, tol: (p.float() - q.float()).norm() <= tol * q.float().norm()  # noqa: E731
    assert near(last(o), o1, 2 ** -7) and near(ST[:, -1:], ST1, 2.0 ** -15)
    del o
    s = osdn.osdn_ssm_bwd(x, dt, A, b, cc, dy)
    s1 = osdn.osdn_ssm_bwd(last(x), last(dt), A[-1:].clone(), b, cc, last(dy))
    finish(osdn)
    assert near(last(s["dx"]), s1["dx"], 2 ** -7) and near(last(s["ddt"]), s1["ddt"], 2.0 ** -13)
    assert near(s["dA"][-1:], s1["dA"], 2.0 ** -13)
