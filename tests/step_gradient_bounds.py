"""How far the scan's step gradients (ddt, dA, ddt_bias) may be off, as relative L2 norms, from the
64-bit statement's own signed terms (test helper, no tests).

The kernels form, per token and head,
    d(log a_t) = sum_{i >= t} c_i.dc_i - sum_{i >= t} b_i.db_i + <G, S>  (sums within a block or chunk)
    dstep_t    = x_t.dx_t / step_t + A d(log a_t)
from dot products of dc, db, dx shares whose elements are good to a relative d of their rms: a
rounding error of d |c| |dc| / sqrt(Dk) for c.dc, the elements' errors being independent, and alike
for the others.  Within a block the sums share their terms, so the errors of its tokens' d(log a)
are taken as one and the same (they add up in dA and ddt_bias), those of different blocks as
independent.  Every bound is 4 such standard deviations.
  d = 2^-20 for bf16 tokens: two exponentials of 2^-22 each a decay, fp32 accumulation, operands that
      enter products exactly or as three bf16 terms.
  d = 2^-22 sqrt(T) + 2^-21 for fp32 tokens: an exponential of two units in the last place and three
      roundings for every token that a state passes, independent from token to token.
"""
import numpy as np

from tests.layer_ref import scan, sigmoid, softplus


def relative_error(io, T):
    return 2.0 ** -20 if io == "bf16" else 2.0 ** -22 * T ** 0.5 + 2.0 ** -21


def heads_apart(a, G, H):
    return {**a, "b": np.repeat(a["b"], H // G, 1), "c": np.repeat(a["c"], H // G, 1)}


def bounds(a, io, use_softplus, lens, dy, dST, block=128):
    """dict(ddt, dA, ddt_bias): per head, the L2 norm (ddt: over the tokens) that the error may have."""
    rows, H, Dv = a["x"].shape
    G, Dk = a["b"].shape[1:]
    h = heads_apart(a, G, H)
    ref = scan(h["x"], h["dt"], h["A"], h["b"], h["c"], None, h["dt_bias"], use_softplus, h["S0"], lens,
               dy=dy, dST=dST)
    raw = a["dt"] + (0.0 if a["dt_bias"] is None else a["dt_bias"])
    step = softplus(raw) if use_softplus else raw
    act = sigmoid(raw) if use_softplus else np.ones_like(raw)
    norm = lambda t: np.sqrt((np.asarray(t, np.float64) ** 2).sum(-1))  # noqa: E731
    safe = np.where(step == 0, 1.0, step)
    pos = norm(h["c"]) * norm(ref["dc"]) / Dk ** 0.5                    # [rows, H]
    neg = norm(h["b"]) * norm(ref["db"]) / Dk ** 0.5
    own = norm(h["x"]) * norm(ref["dx"]) / np.abs(safe) / Dv ** 0.5
    sq = lambda t: 0.0 if t is None else np.square(t).sum((0, 2, 3))    # noqa: E731
    whole = np.sqrt(sq(a["S0"]) * sq(dST) / (Dk * Dv)) / max(len(lens), 1)  # <G, S> of what is given
    d = 4 * relative_error(io, max(lens))
    ddt, dA, db = (np.zeros(H) for _ in range(3))
    at = 0
    for T in lens:
        for t0 in range(0, T, block):
            s = slice(at + t0, at + min(t0 + block, T))
            la = np.sqrt((pos[s] ** 2 + neg[s] ** 2).sum(0)) + whole
            ddt += ((np.abs(a["A"]) * la * act[s]) ** 2 + (own[s] * act[s]) ** 2).sum(0)
            dA += ((np.abs(step[s]) * la).sum(0)) ** 2
            db += ((np.abs(a["A"]) * la * act[s]).sum(0)) ** 2 + ((own[s] * act[s]) ** 2).sum(0)
        at += T
    return dict(ddt=d * np.sqrt(ddt), dA=d * np.sqrt(dA), ddt_bias=d * np.sqrt(db))


def chunk_sums(a, use_softplus, lens, dy, dST, block=128):
    """(ddt, what it is without the <G, S> terms), both from the chunk form in 64 bits."""
    rows, H, _ = a["x"].shape
    h = heads_apart(a, a["b"].shape[1], H)
    ref = scan(h["x"], h["dt"], h["A"], h["b"], h["c"], None, h["dt_bias"], use_softplus, h["S0"], lens,
               dy=dy, dST=dST)
    raw = a["dt"] + (0.0 if a["dt_bias"] is None else a["dt_bias"])
    step = softplus(raw) if use_softplus else raw
    act = sigmoid(raw) if use_softplus else np.ones_like(raw)
    net = (h["c"] * ref["dc"]).sum(-1) - (h["b"] * ref["db"]).sum(-1)
    own = (h["x"] * ref["dx"]).sum(-1) / step
    inner = np.zeros_like(net)
    at = 0
    for T in lens:
        for t0 in range(0, T, block):
            s = slice(at + t0, at + min(t0 + block, T))
            inner[s] = net[s][::-1].cumsum(0)[::-1]
        at += T
    return ref["ddt"], (own + a["A"] * inner) * act
