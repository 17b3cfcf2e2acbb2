"""Plain 64-bit statements (numpy, one token at a time) of the layer operators around the mixer:
the short causal convolution, the selective scan, the block norm, each with its gradient written
out from the formulas.  Test infrastructure; shares nothing with the kernels.

Each also runs on magnitudes (``absolute=True``: every term enters with its absolute value, so
the outputs are the sums of the magnitudes of the terms that make up each output).  Rounding
errors of an fp32 evaluation are bounded by multiples of those sums, which is how the tests'
tolerances are derived.
"""
import numpy as np


def lens_of(B, T, cu):
    return [T] * B if cu is None else [int(b - a) for a, b in zip(cu[:-1], cu[1:])]


# ------------------------------------------------------------------------------- convolution
def sigmoid(z):
    return np.exp(-np.logaddexp(0.0, -z))


def conv(x, weight, bias, state0, silu, lens, dy=None, dstateT=None, absolute=False):
    """x [rows, C], weight [C, W], state0 [N, W - 1, C] or None.  Returns dict(y, stateT) and,
    with dy, dx, dweight, dbias, dstate0."""
    C, W = weight.shape
    N = len(lens)
    st = np.zeros((N, W - 1, C)) if state0 is None else state0.astype(np.float64)
    out = dict(y=np.zeros_like(x, np.float64), stateT=np.zeros((N, W - 1, C)))
    if dy is not None:
        out.update(dx=np.zeros(x.shape), dweight=np.zeros((C, W)), dbias=np.zeros(C),
                   dstate0=np.zeros((N, W - 1, C)))
    at = 0
    for n, T in enumerate(lens):
        seq = np.concatenate([st[n], x[at:at + T]]).astype(np.float64)
        z = np.zeros((T, C))
        za = np.zeros((T, C))
        for t in range(T):
            for w in range(W):
                z[t] += weight[:, w] * seq[t + w]
                za[t] += np.abs(weight[:, w] * seq[t + w])
        if bias is not None:
            z = z + bias
            za = za + np.abs(bias)
        s = sigmoid(z)
        # |silu'| <= 1.1 everywhere
        out["y"][at:at + T] = (1.1 * za if silu else za) if absolute else (z * s if silu else z)
        out["stateT"][n] = seq[T:]
        if dy is not None:
            act = s * (1 + z * (1 - s)) if silu else np.ones_like(z)
            if absolute:
                act = np.full_like(z, 1.1) + (0.5 * za if silu else 0.0)  # |silu''| <= 0.5
            dz = dy[at:at + T] * act
            if absolute:
                dz = np.abs(dz)
            sg = np.abs if absolute else (lambda v: v)
            dseq = np.zeros_like(seq)
            for t in range(T):
                for w in range(W):
                    dseq[t + w] += sg(weight[:, w]) * dz[t]
                    out["dweight"][:, w] += sg(seq[t + w]) * dz[t]
            out["dbias"] += dz.sum(0)
            if dstateT is not None:
                dseq[T:] += sg(dstateT[n])
            out["dx"][at:at + T] = dseq[W - 1:]
            out["dstate0"][n] = dseq[:W - 1]
        at += T
    return out


# --------------------------------------------------------------------------------------- scan
def softplus(x):
    return np.logaddexp(0.0, x)


def scan(x, dt, A, b, c, D, dt_bias, use_softplus, S0, lens, dy=None, dST=None, absolute=False):
    """x [rows, H, Dv], dt [rows, H], b, c [rows, G, Dk], S0 [N, H, Dv, Dk] or None.  Returns
    dict(y, ST) and, with dy, dx, ddt, dA, db, dc, dD, ddt_bias, dS0 (and cancel: per token the
    magnitude of what nearly cancels in ddt when it is summed over up to 128 tokens)."""
    rows, H, Dv = x.shape
    G, Dk = b.shape[1:]
    rep = H // G
    raw = dt.astype(np.float64) + (0.0 if dt_bias is None else dt_bias)
    step = softplus(raw) if use_softplus else raw
    dstep = sigmoid(raw) if use_softplus else np.ones_like(raw)
    decay = np.exp(step * A)
    sg = np.abs if absolute else (lambda v: v)
    x, b, c = (sg(t.astype(np.float64)) for t in (x, b, c))
    stp, Ag = sg(step), sg(A.astype(np.float64))
    skip = np.zeros(H) if D is None else sg(D.astype(np.float64))
    N = len(lens)
    S0 = np.zeros((N, H, Dv, Dk)) if S0 is None else sg(S0.astype(np.float64))
    out = dict(y=np.zeros_like(x), ST=np.zeros((N, H, Dv, Dk)))
    back = dy is not None
    if back:
        dy = sg(dy.astype(np.float64))
        dST = np.zeros((N, H, Dv, Dk)) if dST is None else sg(dST.astype(np.float64))
        out.update(dx=np.zeros_like(x), ddt=np.zeros((rows, H)), dA=np.zeros(H),
                   db=np.zeros_like(b), dc=np.zeros_like(c), dS0=np.zeros_like(S0),
                   dD=(dy * x).sum((0, 2)), cancel=np.zeros((rows, H)))
    at = 0
    for n, T in enumerate(lens):
        S = S0[n].copy()
        before = []
        for t in range(at, at + T):
            bt, ct = np.repeat(b[t], rep, 0), np.repeat(c[t], rep, 0)
            before.append(S)
            S = decay[t][:, None, None] * S + (stp[t][:, None] * x[t])[:, :, None] * bt[:, None, :]
            out["y"][t] = np.einsum("hvk,hk->hv", S, ct) + skip[:, None] * x[t]
        out["ST"][n] = S
        if not back:
            at += T
            continue
        dS = dST[n].copy()
        cancel = np.zeros((T, H))
        for t in range(at + T - 1, at - 1, -1):
            bt, ct = np.repeat(b[t], rep, 0), np.repeat(c[t], rep, 0)
            prev = before[t - at]
            now = decay[t][:, None, None] * prev + (stp[t][:, None] * x[t])[:, :, None] * bt[:, None, :]
            reach = (dS * now).sum((1, 2))
            dS = dS + dy[t][:, :, None] * ct[:, None, :]
            dch = np.einsum("hvk,hv->hk", now, dy[t])
            dbh = np.einsum("hvk,hv->hk", dS, x[t])
            out["dc"][t] = dch.reshape(G, rep, Dk).sum(1)
            out["db"][t] = (stp[t][:, None] * dbh).reshape(G, rep, Dk).sum(1)
            dsb = np.einsum("hvk,hk->hv", dS, bt)
            out["dx"][t] = stp[t][:, None] * dsb + skip[:, None] * dy[t]
            q = (x[t] * dsb).sum(1)
            dla = decay[t] * (dS * prev).sum((1, 2))
            out["dA"] += stp[t] * dla
            out["ddt"][t] = (q + Ag * dla) * dstep[t]
            cancel[t - at] = (ct * dch).sum(1) + stp[t] * q + reach / 128
            dS = decay[t][:, None, None] * dS
        out["dS0"][n] = dS
        for t in range(T):
            out["cancel"][at + t] = cancel[t:t + 128].sum(0) + 127 * cancel[t:t + 128].max(0) / 128
        at += T
    if back:
        out["ddt_bias"] = out["ddt"].sum(0)
        out["reach"] = (stp * out["cancel"]).sum(0)
    return out


# --------------------------------------------------------------------------------------- norm
def norm(f, x, gate, w_post, w_next, act, gate_first, scale, eps, dx_out=None, dh=None):
    """f, x, gate [R, D].  Returns dict(x_out, h) and, with gradients, df, dx, dgate, dw_post,
    dw_next."""
    def rms(v):
        return np.sqrt((v * v).mean(-1, keepdims=True) + eps)

    def back(v, w, d):  # gradients of v / rms(v) * w
        r = rms(v)
        nv = v / r
        dn = d * w
        return (dn - nv * (dn * nv).mean(-1, keepdims=True)) / r, (d * nv).sum(0)

    f = f.astype(np.float64)
    s = None if gate is None else sigmoid(gate.astype(np.float64))
    a = None if gate is None else (gate * s if act == "silu" else s)
    v = f * a if gate is not None and gate_first else f
    m = v if w_post is None else v / rms(v) * w_post
    u = m * a if gate is not None and not gate_first else m
    xo = scale * u + (0.0 if x is None else x)
    out = dict(x_out=xo, h=None if w_next is None else xo / rms(xo) * w_next)
    if dx_out is None and dh is None:
        return out
    d = np.zeros_like(f) if dx_out is None else dx_out.astype(np.float64)
    if w_next is not None:
        dv, out["dw_next"] = back(xo, w_next, dh.astype(np.float64))
        d = d + dv
    out["dx"] = d
    d = scale * d
    da = None if gate is None else (s * (1 + gate * (1 - s)) if act == "silu" else s * (1 - s))
    if gate is not None and not gate_first:
        out["dgate"] = d * m * da
        d = d * a
    if w_post is not None:
        d, out["dw_post"] = back(v, w_post, d)
    if gate is not None and gate_first:
        out["dgate"] = d * f * da
        d = d * a
    out["df"] = d
    return out
