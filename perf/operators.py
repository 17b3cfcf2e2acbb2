"""What is measured of the recurrent-layer operators: the short causal convolution, the selective
state-space scan and the block norm, each for prompts, for single tokens where a decoder calls it
so, and in its backward direction.

``run`` computes them with elementary torch operations in 32 bits (64 where long sums of log
decays need it); with ``own`` set, through the library's binding.  ``exact`` computes the same
values from the definitions in 64 bits, token by token.

The definitions (n a sequence, t its tokens):
  conv   z_t[c] = bias[c] + sum_w weight[c][w] x_{t-W+1+w}[c],  y_t = silu(z_t); tokens before the
         first come from the state (the W - 1 inputs before the sequence, oldest first)
  scan   D_t = softplus(dt_t + dt_bias),  S_t = exp(D_t A) S_{t-1} + D_t x_t b_t^T,
         y_t = S_t c_t + D x_t   (per head; H / G heads share a row of b and c)
  norm   u = f / rms(f) * w_post * silu(gate)  (or rms of f * silu(gate), the gate first),
         x' = x + scale u,  h = x' / rms(x') * w_next
"""
import math

import torch

own = False

CHUNK = 128  # tokens per chunk of the plain scan


# ------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # a prompt batch through the convolution in front of a 1.3B layer's mixer
        dict(name="conv prompt 1.3B", op="conv_fwd", io="bf16", B=4, T=4096, lens="", C=2048, W=4,
             bias=False, state=False),
        # packed requests of any length continuing from their states, a width that no vector
        # divides, in single precision
        dict(name="conv prompt packed", op="conv_fwd", io="f32", B=1, T=6028,
             lens="1,777,2,4095,130,0,1023", C=1001, W=3, bias=True, state=True),
        # the smallest call: one token for each of a few sequences being decoded
        dict(name="conv token 8", op="conv_step", io="bf16", N=8, C=2048, W=4, bias=True),
        # training a 340M layer
        dict(name="conv backward 340M", op="conv_bwd", io="bf16", B=8, T=2048, lens="", C=1024,
             W=4, bias=True, state=False),
        # a prompt batch at the 1.3B layer's heads, every head with its own b and c
        dict(name="scan prompt 1.3B", op="ssm_fwd", io="bf16", B=4, T=4096, lens="", H=16, G=16,
             Dk=128, Dv=128, D=True, state=False),
        # one long document continued from a state, all heads sharing b and c
        dict(name="scan prompt long", op="ssm_fwd", io="bf16", B=1, T=65536, lens="", H=16, G=1,
             Dk=128, Dv=64, D=True, state=True),
        # a few short packed requests in single precision
        dict(name="scan prompt packed f32", op="ssm_fwd", io="f32", B=1, T=1499,
             lens="5,1,300,0,64,129,1000", H=4, G=2, Dk=64, Dv=64, D=True, state=True),
        # a decoding batch: one token for each of 256 sequences
        dict(name="scan token 256", op="ssm_step", io="bf16", N=256, H=16, G=1, Dk=128, Dv=128,
             D=True),
        # training a 340M layer
        dict(name="scan backward 340M", op="ssm_bwd", io="bf16", B=8, T=2048, lens="", H=8, G=8,
             Dk=128, Dv=128, D=True, state=False),
        # training on packed documents, heads sharing b and c in groups, through the states too
        dict(name="scan backward packed", op="ssm_bwd", io="bf16", B=1, T=7112,
             lens="128,2047,1,63,4096,777", H=16, G=2, Dk=128, Dv=64, D=True, state=True),
        # the end of a 1.3B block and the start of the next, over a prompt batch
        dict(name="norm prompt 1.3B", op="norm_fwd", io="bf16", R=16384, D=2048, gate=True,
             first=False, post=True, res=True, next=True),
        # training the gated norm over each head of a 340M layer's mixer output
        dict(name="norm backward heads", op="norm_bwd", io="bf16", R=131072, D=128, gate=True,
             first=False, post=True, res=False, next=False),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_lens(rng, total):
    """Sequence lengths, zero and one among them, that add up to about `total`."""
    n = rng.randint(1, 12)
    cuts = [rng.random() ** 2 + 1e-3 for _ in range(n)]
    lens = [int(total * c / sum(cuts)) for c in cuts] + rng.choice([[], [0], [1], [0, 1]])
    if not sum(lens):
        lens[0] = 1
    rng.shuffle(lens)
    return lens


def _draw_tokens(rng, most):
    total = _logint(rng, 16, most)
    if rng.random() < 0.5:
        B = rng.choice([1, 1, 2, 3, 4, 7, 8])
        return dict(B=B, T=max(1, total // B), lens="")
    lens = _draw_lens(rng, total)
    return dict(B=1, T=sum(lens), lens=",".join(str(n) for n in lens))


def draw(rng):
    op = rng.choice(["conv_fwd", "conv_step", "conv_bwd", "ssm_fwd", "ssm_fwd", "ssm_step",
                     "ssm_bwd", "ssm_bwd", "norm_fwd", "norm_bwd"])
    c = dict(op=op, io=rng.choice(["bf16", "bf16", "bf16", "f32"]))
    f32 = c["io"] == "f32"
    flag = lambda: rng.random() < 0.5  # noqa: E731
    if op.startswith("conv"):
        C = rng.choice([_logint(rng, 65, 2500), 8 * _logint(rng, 8, 320), 512, 1024, 2048])
        if op == "conv_step":
            c.update(N=_logint(rng, 1, 1024))
        else:
            c.update(_draw_tokens(rng, 12000), state=flag())
        c.update(C=C, W=rng.choice([2, 3, 4, 4]), bias=flag())
    elif op.startswith("ssm"):
        H = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
        G = rng.choice([g for g in range(1, H + 1) if H % g == 0])
        if op == "ssm_step":
            c.update(N=_logint(rng, 1, 300))
        else:
            c.update(_draw_tokens(rng, 3000 if f32 else 12000), state=flag())
        c.update(H=H, G=G, Dk=rng.choice([64, 128]), Dv=rng.choice([64, 128]), D=flag())
    else:
        D = rng.choice([64, 128, 1024, 2048, 4096, _logint(rng, 33, 4200), 8 * _logint(rng, 5, 500)])
        post, gate = flag(), flag()
        c.update(R=max(1, _logint(rng, 1 << 14, 1 << 25) // D), D=D, gate=gate, post=post,
                 first=gate and post and flag(), res=flag(), next=flag())
    return c


# ------------------------------------------------------------------------------------ the inputs
def _io(case):
    return torch.bfloat16 if case["io"] == "bf16" else torch.float32


def _lens(case):
    if case.get("lens"):
        return [int(v) for v in case["lens"].split(",")]
    return [case["T"]] * case["B"]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 2654435761 % (1 << 62) + 17)
    io = _io(case)

    def rnd(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    def uni(lo, hi, *shape):
        return lo + (hi - lo) * torch.rand(*shape, generator=g, device="cuda")

    s = dict(case=dict(case))
    op = case["op"]
    if op.startswith("conv"):
        C, W = case["C"], case["W"]
        s["weight"] = rnd(C, W, scale=W ** -0.5)
        s["bias"] = rnd(C, scale=0.2) if case["bias"] else None
        if op == "conv_step":
            s["x"] = rnd(case["N"], C, dtype=io)
            s["state"] = rnd(case["N"], W - 1, C, dtype=io)
            return s
        lens = _lens(case)
        s["x"] = rnd(case["B"], case["T"], C, dtype=io)
        s["state0"] = rnd(len(lens), W - 1, C, dtype=io) if case["state"] else None
        if op == "conv_bwd":
            s["dy"] = rnd(case["B"], case["T"], C, dtype=io)
            s["dstateT"] = rnd(len(lens), W - 1, C) if case["state"] else None
    elif op.startswith("ssm"):
        H, G, Dk, Dv = case["H"], case["G"], case["Dk"], case["Dv"]
        lead = (case["N"],) if op == "ssm_step" else (case["B"], case["T"])
        n = case["N"] if op == "ssm_step" else len(_lens(case))
        s["x"] = rnd(*lead, H, Dv, dtype=io)
        s["b"] = rnd(*lead, G, Dk, dtype=io, scale=0.5)
        s["c"] = rnd(*lead, G, Dk, dtype=io, scale=0.5)
        s["dt"] = rnd(*lead, H, scale=0.5)
        s["A"] = -uni(1.0, 16.0, H)
        step = torch.exp(uni(math.log(1e-3), math.log(1e-1), H))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))  # softplus^-1 of the step
        s["D"] = 1.0 + rnd(H, scale=0.1) if case["D"] else None
        if op == "ssm_step":
            s["S"] = rnd(n, H, Dv, Dk, scale=0.5)
            return s
        s["S0"] = rnd(n, H, Dv, Dk, scale=0.5) if case["state"] else None
        if op == "ssm_bwd":
            s["dy"] = rnd(*lead, H, Dv, dtype=io)
            s["dST"] = rnd(n, H, Dv, Dk, scale=0.1) if case["state"] else None
    else:
        R, D = case["R"], case["D"]
        s["f"] = rnd(R, D, dtype=io)
        s["x"] = rnd(R, D, dtype=io, scale=2.0) if case["res"] else None
        s["gate"] = rnd(R, D, dtype=io) if case["gate"] else None
        s["w_post"] = 1.0 + rnd(D, scale=0.1) if case["post"] else None
        s["w_next"] = 1.0 + rnd(D, scale=0.1) if case["next"] else None
        s["scale"] = 0.5
        if op == "norm_bwd":
            s["dx_out"] = rnd(R, D, dtype=io)
            s["dh"] = rnd(R, D, dtype=io) if case["next"] else None
    if case.get("lens"):
        s["cu"] = torch.tensor([0] + _lens(case), device="cuda").cumsum(0).to(torch.int32)
    else:
        s["cu"] = None
    if own:
        from delta_rule_recurrent_osdn_b200 import osdn  # noqa: F401  (loads the library)
    return s


# ------------------------------------------------------------------------------------- one pass
def run(s):
    if own:
        return _run_own(s)
    with torch.no_grad():
        return PLAIN[s["case"]["op"]](s)


def _run_own(s):
    from delta_rule_recurrent_osdn_b200 import osdn
    op = s["case"]["op"]
    if op == "conv_fwd":
        y, st = osdn.osdn_conv_fwd(s["x"], s["weight"], s["bias"], s["state0"],
                                   cu_seqlens=s["cu"])
        return dict(y=y, stateT=st)
    if op == "conv_step":
        y = osdn.osdn_conv_step(s["x"], s["weight"], s["state"], s["bias"])
        return dict(y=y, state=s["state"])
    if op == "conv_bwd":
        return osdn.osdn_conv_bwd(s["x"], s["weight"], s["dy"], s["bias"], s["state0"],
                                  s["dstateT"], cu_seqlens=s["cu"])
    if op == "ssm_fwd":
        y, ST = osdn.osdn_ssm_fwd(s["x"], s["dt"], s["A"], s["b"], s["c"], s["D"], s["dt_bias"],
                                  S0=s["S0"], cu_seqlens=s["cu"])
        return dict(y=y, ST=ST)
    if op == "ssm_step":
        y = osdn.osdn_ssm_step(s["x"], s["dt"], s["A"], s["b"], s["c"], s["S"], s["D"],
                               s["dt_bias"])
        return dict(y=y, S=s["S"])
    if op == "ssm_bwd":
        return osdn.osdn_ssm_bwd(s["x"], s["dt"], s["A"], s["b"], s["c"], s["dy"], s["D"],
                                 s["dt_bias"], S0=s["S0"], dST=s["dST"], cu_seqlens=s["cu"])
    if op == "norm_fwd":
        xo, h = osdn.osdn_norm_fwd(s["f"], s["x"], s["gate"], s["w_post"], s["w_next"],
                                   gate_first=s["case"]["first"], scale=s["scale"])
        return dict(x_out=xo, h=h)
    return osdn.osdn_norm_bwd(s["f"], s["dx_out"], s["dh"], s["x"], s["gate"], s["w_post"],
                              s["w_next"], gate_first=s["case"]["first"], scale=s["scale"])


# ------------------------------------------------------------- plain form: the convolution
def _silu(z):
    return z / (1.0 + torch.exp(-z))


def _silu_grad(z):
    e = 1.0 / (1.0 + torch.exp(-z))
    return e * (1.0 + z * (1.0 - e))


def _taps(s):
    """[rows, W]: the rows of [states; x] that each output reads, and [N, W-1]: those of its
    sequence's final state."""
    case, W = s["case"], s["case"]["W"]
    dev = s["x"].device
    lens = torch.tensor(_lens(case), device=dev)
    ends = lens.cumsum(0)
    first = ends - lens
    row = torch.arange(case["B"] * case["T"], device=dev)
    n = torch.searchsorted(ends, row, right=True)
    nst = lens.numel() * (W - 1)

    def source(n, pos):  # position pos (negative: a state row) of sequence n
        return torch.where(pos >= 0, nst + first[n] + pos, n * (W - 1) + (W - 1) + pos)

    pos = (row - first[n])[:, None] - (W - 1) + torch.arange(W, device=dev)
    m = torch.arange(lens.numel(), device=dev)[:, None]
    last = lens[:, None] - (W - 1) + torch.arange(W - 1, device=dev)
    return source(n[:, None], pos), source(m, last)


def _with_state(s):
    C, W = s["case"]["C"], s["case"]["W"]
    n = len(_lens(s["case"]))
    st = s["state0"]
    st = st.float().reshape(-1, C) if st is not None else s["x"].new_zeros(n * (W - 1), C).float()
    return torch.cat([st, s["x"].float().reshape(-1, C)])


def _conv_z(s, ext, idx):
    z = (ext[idx] * s["weight"].t()).sum(1)
    return z if s["bias"] is None else z + s["bias"]


def _plain_conv_fwd(s):
    ext = _with_state(s)
    idx, last = _taps(s)
    y = _silu(_conv_z(s, ext, idx))
    return dict(y=y.to(s["x"].dtype).reshape(s["x"].shape), stateT=ext[last].to(s["x"].dtype))


def _plain_conv_step(s):
    win = torch.cat([s["state"].float(), s["x"].float()[:, None]], 1)
    z = (win * s["weight"].t()).sum(1)
    z = z if s["bias"] is None else z + s["bias"]
    s["state"].copy_(win[:, 1:])  # the state is a decoder's own buffer, updated in place
    return dict(y=_silu(z).to(s["x"].dtype), state=s["state"])


def _plain_conv_bwd(s):
    C, W = s["case"]["C"], s["case"]["W"]
    ext = _with_state(s)
    idx, last = _taps(s)
    dz = s["dy"].float().reshape(-1, C) * _silu_grad(_conv_z(s, ext, idx))
    dext = torch.zeros_like(ext)
    dext.index_add_(0, idx.reshape(-1), (dz[:, None] * s["weight"].t()).reshape(-1, C))
    if s["dstateT"] is not None:
        dext.index_add_(0, last.reshape(-1), s["dstateT"].reshape(-1, C))
    dw = (dz[:, None] * ext[idx]).sum(0, dtype=torch.float64).float().t().contiguous()
    db = None if s["bias"] is None else dz.sum(0, dtype=torch.float64).float()
    nst = last.numel()
    return dict(dx=dext[nst:].to(s["x"].dtype).reshape(s["x"].shape), dweight=dw, dbias=db,
                dstate0=None if s["state0"] is None else dext[:nst].reshape(-1, W - 1, C))


# --------------------------------------------------------------------- plain form: the scan
def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def _padded(case, dev):
    """[N, Tp] rows of the packed tokens (Tp whole chunks) and which of them are tokens."""
    lens = torch.tensor(_lens(case), device=dev)
    tp = max(CHUNK, -(-max(_lens(case)) // CHUNK) * CHUNK)
    t = torch.arange(tp, device=dev)
    mask = t < lens[:, None]
    row = (lens.cumsum(0) - lens)[:, None] + t
    return torch.where(mask, row, 0), mask


def _plain_scan(case, x, dt, A, b, c, D, dt_bias, S0):
    """The chunked form, in 32 bits; log decays are summed in 64."""
    H, G, Dk, Dv = case["H"], case["G"], case["Dk"], case["Dv"]
    rows = case["B"] * case["T"]
    idx, mask = _padded(case, x.device)
    N, Tp = idx.shape
    L, nc = CHUNK, Tp // CHUNK
    xs, bs, cs = (t.float().reshape(rows, n, d)[idx].reshape(N, nc, L, n, d).transpose(2, 3)
                  for t, n, d in ((x, H, Dv), (b, G, Dk), (c, G, Dk)))  # [N, nc, heads, L, d]
    step = _softplus(dt.double().reshape(rows, H) + dt_bias.double())[idx] * mask[..., None]
    step = step.reshape(N, nc, L, H).transpose(2, 3)                    # [N, nc, H, L]
    log = (step * A.double()[:, None]).cumsum(-1)
    tri = torch.ones(L, L, dtype=torch.bool, device=x.device).tril()
    decay = torch.exp((log[..., :, None] - log[..., None, :]).masked_fill(~tri, -math.inf)).float()
    stepf = step.float()
    heads = lambda t: t.repeat_interleave(H // G, 2)  # noqa: E731
    xd = xs * stepf[..., None]
    y = (heads(cs @ bs.transpose(-1, -2)) * decay) @ xd
    to_end = torch.exp(log[..., -1:] - log).float()
    add = (xd * to_end[..., None]).transpose(-1, -2) @ heads(bs)        # [N, nc, H, Dv, Dk]
    # the state in front of each chunk, and behind the last: a sum over the earlier chunks
    whole = torch.nn.functional.pad(log[..., -1].cumsum(1), (0, 0, 1, 0)).transpose(1, 2)
    low = torch.ones(nc + 1, nc + 1, dtype=torch.bool, device=x.device).tril()
    mix = torch.exp((whole[..., :, None] - whole[..., None, :]).masked_fill(~low, -math.inf))
    S0 = add.new_zeros(N, H, Dv, Dk) if S0 is None else S0
    parts = torch.cat([S0[:, None], add], 1).transpose(1, 2).reshape(N, H, nc + 1, Dv * Dk)
    states = (mix.float() @ parts).reshape(N, H, nc + 1, Dv, Dk)
    before = states[:, :, :-1].transpose(1, 2)
    y = y + (heads(cs) @ before.transpose(-1, -2)) * torch.exp(log).float()[..., None]
    if D is not None:
        y = y + D[:, None, None] * xs
    y = y.transpose(2, 3).reshape(N, Tp, H, Dv)[mask].reshape(x.shape)
    return y, states[:, :, -1].contiguous()


def _plain_ssm_fwd(s):
    y, ST = _plain_scan(s["case"], s["x"], s["dt"], s["A"], s["b"], s["c"], s["D"], s["dt_bias"],
                        s["S0"])
    return dict(y=y.to(s["x"].dtype), ST=ST)


def _plain_ssm_step(s):
    rep = s["case"]["H"] // s["case"]["G"]
    b, c = (t.float().repeat_interleave(rep, 1) for t in (s["b"], s["c"]))
    x = s["x"].float()
    step = _softplus(s["dt"] + s["dt_bias"])
    S = s["S"].mul_(torch.exp(step * s["A"])[..., None, None])  # in place, as above
    S.add_((step[..., None] * x)[..., None] * b[:, :, None, :])
    y = (S * c[:, :, None, :]).sum(-1)
    if s["D"] is not None:
        y = y + s["D"][:, None] * x
    return dict(y=y.to(s["x"].dtype), S=S)


def _plain_ssm_bwd(s):
    """The chunked form's gradients, by the chain rule through its operations."""
    names = [k for k in ("x", "dt", "A", "b", "c", "D", "dt_bias", "S0") if s[k] is not None]
    with torch.enable_grad():
        a = {k: s[k].detach().float().requires_grad_() for k in names}
        y, ST = _plain_scan(s["case"], *(a.get(k) for k in ("x", "dt", "A", "b", "c", "D",
                                                            "dt_bias", "S0")))
        outs, grads = [y], [s["dy"].float()]
        if s["dST"] is not None:
            outs.append(ST)
            grads.append(s["dST"])
        g = dict(zip(names, torch.autograd.grad(outs, [a[k] for k in names], grads)))
    io = s["x"].dtype
    out = {"d" + k: (g[k].to(io) if k in ("x", "b", "c") else g[k]) if k in g else None
           for k in ("x", "dt", "A", "b", "c", "D", "dt_bias")}
    if s["S0"] is not None:
        out["dS0"] = g["S0"]
    return out


# --------------------------------------------------------------------- plain form: the norm
EPS = 1e-5


def _rms(x):
    return torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)


def _branch(s):
    """(v, r, u0, a): the norm's input, its reciprocal rms, the branch and the gate's factor."""
    f = s["f"].float()
    a = None if s["gate"] is None else _silu(s["gate"].float())
    v = f * a if s["case"]["first"] else f
    r = None if s["w_post"] is None else _rms(v)
    u = v if r is None else v * r * s["w_post"]
    if a is not None and not s["case"]["first"]:
        u = u * a
    return v, r, u, a


def _plain_norm_fwd(s):
    xo = s["scale"] * _branch(s)[2]
    if s["x"] is not None:
        xo = s["x"].float() + xo
    io = s["f"].dtype
    h = None if s["w_next"] is None else (xo * _rms(xo) * s["w_next"]).to(io)
    return dict(x_out=xo.to(io), h=h)


def _norm_grad(v, r, w, dout):
    """Gradients of v * r(v) * w with respect to v and w."""
    n = v * r
    dn = dout * w
    return r * (dn - n * (dn * n).mean(-1, keepdim=True)), \
        (dout * n).sum(0, dtype=torch.float64).float()


def _plain_norm_bwd(s):
    v, r, u, a = _branch(s)
    io, first = s["f"].dtype, s["case"]["first"]
    d = s["dx_out"].float()
    out = dict(dw_post=None, dw_next=None, dgate=None, dx=None)
    if s["w_next"] is not None:
        xo = s["scale"] * u if s["x"] is None else s["x"].float() + s["scale"] * u
        dn, out["dw_next"] = _norm_grad(xo, _rms(xo), s["w_next"], s["dh"].float())
        d = d + dn
    if s["x"] is not None:
        out["dx"] = d.to(io)
    d = d * s["scale"]
    gate = None if a is None else _silu_grad(s["gate"].float())
    if a is not None and not first:
        out["dgate"] = (d * (v if r is None else v * r * s["w_post"]) * gate).to(io)
        d = d * a
    if r is not None:
        d, out["dw_post"] = _norm_grad(v, r, s["w_post"], d)
    if a is not None and first:
        out["dgate"] = (d * s["f"].float() * gate).to(io)
        d = d * a
    out["df"] = d.to(io)
    return out


PLAIN = dict(conv_fwd=_plain_conv_fwd, conv_step=_plain_conv_step, conv_bwd=_plain_conv_bwd,
             ssm_fwd=_plain_ssm_fwd, ssm_step=_plain_ssm_step, ssm_bwd=_plain_ssm_bwd,
             norm_fwd=_plain_norm_fwd, norm_bwd=_plain_norm_bwd)


# ----------------------------------------------------------------------------- what a pass needs
def work(case):
    es = 2 if case["io"] == "bf16" else 4
    op = case["op"]
    if op.startswith("conv"):
        C, W = case["C"], case["W"]
        par = C * W * 4 + (C * 4 if case["bias"] else 0)
        if op == "conv_step":
            n = case["N"]
            return dict(bytes=n * C * es * 2 * W + par, flops=n * C * (2 * W + 4))
        rows, n = case["B"] * case["T"], len(_lens(case))
        st = n * (W - 1) * C
        if op == "conv_fwd":
            return dict(bytes=rows * C * es * 2 + par + st * es * (2 if case["state"] else 1),
                        flops=rows * C * (2 * W + 4))
        return dict(bytes=rows * C * es * 3 + 2 * par +
                    (st * (es + 8) if case["state"] else 0), flops=rows * C * (6 * W + 8))
    if op.startswith("ssm"):
        H, G, Dk, Dv = case["H"], case["G"], case["Dk"], case["Dv"]
        n = case["N"] if op == "ssm_step" else len(_lens(case))
        rows = n if op == "ssm_step" else case["B"] * case["T"]
        par = 8 * H + (4 * H if case["D"] else 0)
        state = n * H * Dv * Dk * 4
        token = H * Dv * es * 2 + 2 * G * Dk * es + 4 * H
        if op == "ssm_step":
            return dict(bytes=rows * token + 2 * state + par, flops=rows * H * 5 * Dk * Dv)
        if op == "ssm_fwd":
            return dict(bytes=rows * token + state * (2 if case["state"] else 1) + par,
                        flops=rows * H * 4 * Dk * Dv)
        return dict(bytes=rows * (3 * H * Dv * es + 4 * G * Dk * es + 8 * H) + 2 * par +
                    (3 * state if case["state"] else 0), flops=rows * H * 12 * Dk * Dv)
    R, D = case["R"], case["D"]
    par = D * 4 * (int(case["post"]) + int(case["next"]))
    if op == "norm_fwd":
        return dict(bytes=R * D * es * (2 + case["gate"] + case["res"] + case["next"]) + par,
                    flops=R * D * (4 + 4 * case["gate"] + 3 * case["post"] + 4 * case["next"]))
    return dict(bytes=R * D * es * (3 + 2 * case["gate"] + 2 * case["res"] + case["next"]) + 2 * par,
                flops=R * D * (4 + 12 * case["gate"] + 10 * case["post"] + 12 * case["next"]))


# ---------------------------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    s = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v
         for k, v in s.items()}
    op = case["op"]
    with torch.no_grad():
        if op == "conv_step":
            return _exact_conv_step(s)
        if op.startswith("conv"):
            return _exact_conv(s)
        if op.startswith("ssm"):
            return _exact_scan(s)
        return _exact_norm(s)


def _exact_conv_step(s):
    W = s["case"]["W"]
    z = s["x"] * s["weight"][:, W - 1]
    for w in range(W - 1):
        z = z + s["state"][:, w] * s["weight"][:, w]
    if s["bias"] is not None:
        z = z + s["bias"]
    new = [s["state"][:, w] for w in range(1, W - 1)] + [s["x"]]
    return dict(y=z * torch.sigmoid(z), state=torch.stack(new, 1))


def _exact_conv(s):
    """Sequence by sequence, tap by tap."""
    case, W, C = s["case"], s["case"]["W"], s["case"]["C"]
    rows = s["x"].reshape(-1, C)
    back = case["op"] == "conv_bwd"
    ys, sts, dxs, dsts, at = [], [], [], [], 0
    dw, db = torch.zeros_like(s["weight"]), rows.new_zeros(C)
    for n, T in enumerate(_lens(case)):
        head = rows.new_zeros(W - 1, C) if s["state0"] is None else s["state0"][n]
        seq = torch.cat([head, rows[at:at + T]])
        z = rows.new_zeros(T, C)
        for w in range(W):
            z = z + s["weight"][:, w] * seq[w:w + T]
        if s["bias"] is not None:
            z = z + s["bias"]
        sig = torch.sigmoid(z)
        if back:
            dz = s["dy"].reshape(-1, C)[at:at + T] * (sig + z * sig * (1 - sig))
            dseq = torch.zeros_like(seq)
            for w in range(W):
                dseq[w:w + T] += s["weight"][:, w] * dz
                dw[:, w] += (dz * seq[w:w + T]).sum(0)
            db += dz.sum(0)
            if s["dstateT"] is not None:
                dseq[T:] += s["dstateT"][n]
            dxs.append(dseq[W - 1:])
            dsts.append(dseq[:W - 1])
        else:
            ys.append(z * sig)
            sts.append(seq[T:])
        at += T
    if back:
        return dict(dx=torch.cat(dxs).reshape(s["x"].shape), dweight=dw,
                    dbias=None if s["bias"] is None else db,
                    dstate0=None if s["state0"] is None else torch.stack(dsts))
    return dict(y=torch.cat(ys).reshape(s["x"].shape), stateT=torch.stack(sts))


def _exact_scan(s):
    """The recurrence, token by token over all sequences at once (a sequence that has ended
    keeps its state: its step is zero there)."""
    case, op = s["case"], s["case"]["op"]
    H, G, Dk, Dv = case["H"], case["G"], case["Dk"], case["Dv"]
    dev, rep = s["x"].device, case["H"] // case["G"]
    if op == "ssm_step":
        lens, rows = [1] * case["N"], case["N"]
    else:
        lens, rows = _lens(case), case["B"] * case["T"]
    N, T = len(lens), max(lens)
    ln = torch.tensor(lens, device=dev)
    first = ln.cumsum(0) - ln
    x, dt = s["x"].reshape(rows, H, Dv), s["dt"].reshape(rows, H)
    b, c = s["b"].reshape(rows, G, Dk), s["c"].reshape(rows, G, Dk)
    raw = dt + s["dt_bias"]
    step = torch.logaddexp(raw, torch.zeros_like(raw))
    A = s["A"]

    def at(t):  # rows of token t, and which sequences have one
        live = t < ln
        return torch.where(live, first + t, 0), live

    def token(t):
        r, live = at(t)
        st = step[r] * live[:, None]
        return r, live, st, torch.exp(st * A), x[r], b[r].repeat_interleave(rep, 1), \
            c[r].repeat_interleave(rep, 1)

    S = s["S"].clone() if op == "ssm_step" else \
        x.new_zeros(N, H, Dv, Dk) if s["S0"] is None else s["S0"].clone()
    back = op == "ssm_bwd"
    every, kept = 64, []
    y = torch.zeros_like(x)
    for t in range(T):
        if back and t % every == 0:
            kept.append(S)
        r, live, st, a, xt, bt, ct = token(t)
        S = a[..., None, None] * S + (st[..., None] * xt)[..., None] * bt[:, :, None, :]
        if not back:
            yt = torch.einsum("nhvk,nhk->nhv", S, ct)
            y.index_add_(0, r, yt * live[:, None, None])
    if not back:
        if s["D"] is not None:
            y = y + s["D"][:, None] * x
        y = y.reshape(s["x"].shape)
        return dict(y=y, S=S) if op == "ssm_step" else dict(y=y, ST=S)
    dy = s["dy"].reshape(rows, H, Dv)
    dx, ddt = torch.zeros_like(x), torch.zeros_like(dt)
    dbh, dch = x.new_zeros(rows, H, Dk), x.new_zeros(rows, H, Dk)
    dA = torch.zeros_like(A)
    dS = x.new_zeros(N, H, Dv, Dk) if s["dST"] is None else s["dST"].clone()
    for k in reversed(range(len(kept))):
        seg = [kept[k]]
        for t in range(k * every, min(T, (k + 1) * every)):
            r, live, st, a, xt, bt, ct = token(t)
            seg.append(a[..., None, None] * seg[-1] +
                       (st[..., None] * xt)[..., None] * bt[:, :, None, :])
        for t in reversed(range(k * every, min(T, (k + 1) * every))):
            r, live, st, a, xt, bt, ct = token(t)
            on = live[:, None, None].double()
            dyt = dy[r] * on
            dS = dS + dyt[..., None] * ct[:, :, None, :]
            dch.index_add_(0, r, torch.einsum("nhvk,nhv->nhk", seg[t - k * every + 1], dyt))
            dbh.index_add_(0, r, torch.einsum("nhvk,nhv->nhk", dS, st[..., None] * xt))
            dsb = torch.einsum("nhvk,nhk->nhv", dS, bt)
            dx.index_add_(0, r, st[..., None] * dsb)
            dla = a * (dS * seg[t - k * every]).sum((-1, -2))
            dA += (st * dla).sum(0)
            ddt.index_add_(0, r, ((xt * dsb).sum(-1) + A * dla) * on[..., 0])
            dS = a[..., None, None] * dS
    ddt = ddt * torch.sigmoid(raw)
    D = s["D"]
    if D is not None:
        dx = dx + D[:, None] * dy
    out = dict(dx=dx.reshape(s["x"].shape), ddt=ddt.reshape(s["dt"].shape), dA=dA,
               db=dbh.reshape(rows, G, rep, Dk).sum(2).reshape(s["b"].shape),
               dc=dch.reshape(rows, G, rep, Dk).sum(2).reshape(s["c"].shape),
               dD=None if D is None else (dy * x).sum((0, 2)), ddt_bias=ddt.sum(0))
    if s["S0"] is not None:
        out["dS0"] = dS
    return out


def _exact_norm(s):
    """From the definitions; the gradients by the quotient rule on u / sqrt(mean(u^2) + eps)."""
    case = s["case"]
    f, g, wp, wn, k = s["f"], s["gate"], s["w_post"], s["w_next"], s["scale"]
    sg = None if g is None else torch.sigmoid(g)
    before = f if g is None or not case["first"] else f * (g * sg)
    rp = None if wp is None else (before.pow(2).mean(-1, keepdim=True) + EPS).sqrt()
    mid = before if wp is None else before / rp * wp
    u = mid * (g * sg) if g is not None and not case["first"] else mid
    xo = k * u if s["x"] is None else s["x"] + k * u
    rn = None if wn is None else (xo.pow(2).mean(-1, keepdim=True) + EPS).sqrt()
    if case["op"] == "norm_fwd":
        return dict(x_out=xo, h=None if wn is None else xo / rn * wn)

    def through(v, root, w, d):  # d(v / root * w)
        dv = d * w / root - v * ((d * w * v).sum(-1, keepdim=True) / (v.shape[-1] * root.pow(3)))
        return dv, (d * v / root).sum(0)

    out = dict(dw_post=None, dw_next=None, dgate=None, dx=None)
    d = s["dx_out"]
    if wn is not None:
        dv, out["dw_next"] = through(xo, rn, wn, s["dh"])
        d = d + dv
    if s["x"] is not None:
        out["dx"] = d
    d = k * d
    act = None if g is None else sg * (1 + g * (1 - sg))
    if g is not None and not case["first"]:
        out["dgate"] = d * mid * act
        d = d * (g * sg)
    if wp is not None:
        d, out["dw_post"] = through(before, rp, wp, d)
    if g is not None and case["first"]:
        out["dgate"] = d * f * act
        d = d * (g * sg)
    out["df"] = d
    return out
