"""The layer operators' C ABI without a GPU: the binding's argument types are the header's, and
bad arguments are refused before anything reaches CUDA."""
import ctypes
import re

import pytest

osdn = pytest.importorskip("delta_rule_recurrent_osdn_b200.osdn")
L = osdn.LIB
INV, UNS, ALI, OK = (osdn.OSDN_ERR_INVALID_ARG, osdn.OSDN_ERR_UNSUPPORTED,
                     osdn.OSDN_ERR_ALIGNMENT, osdn.OSDN_OK)
BF, F32 = osdn.OSDN_BF16, osdn.OSDN_F32
SPACE = 0x10000000


def fake(i, off=0):
    return ctypes.c_void_p(0x100000000 + i * SPACE + off)


def test_argument_types_match_the_header():
    text = open(osdn.HEADER).read()
    for name in osdn.header_symbols():
        decl = re.search(r"OSDN_API\s+[\w\s\*]*?" + name + r"\s*\((.*?)\);", text, re.S).group(1)
        args = [a.strip() for a in re.sub(r"\s+", " ", decl).split(",")]
        kinds = []
        for a in [] if args == ["void"] else args:
            kinds.append(ctypes.c_void_p if "*" in a else ctypes.c_int32 if a.startswith("int32_t")
                         else ctypes.c_int64 if a.startswith("int64_t")
                         else ctypes.c_float if a.startswith("float")
                         else ctypes.c_size_t if a.startswith("size_t") else ctypes.c_int)
        types = getattr(L, name).argtypes
        if types is not None:
            assert list(types) == kinds, name


def call(fn, names, defaults, kw):
    args = dict(defaults)
    assert set(kw) <= set(args), kw
    args.update(kw)
    return getattr(L, fn)(*(args[n] for n in names.split()))


# ------------------------------------------------------------------------------- convolution
CONV = dict(x=fake(1), weight=fake(2), bias=fake(3), state0=fake(4), silu=1, y=fake(5),
            stateT=fake(6), cu=None, num_seqs=0, B=2, T=8, C=96, W=4, io=BF, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(C=0), INV), (dict(T=-1), INV), (dict(B=-1), INV), (dict(silu=2), INV), (dict(io=5), INV),
    (dict(W=1), UNS), (dict(W=5), UNS), (dict(C=(1 << 30) + 1), UNS),
    (dict(x=None), INV), (dict(y=None), INV), (dict(weight=None), INV),
    (dict(cu=fake(9), num_seqs=2), INV),                       # packed needs B == 1
    (dict(cu=fake(9), num_seqs=0, B=1), INV),                  # tokens of no sequence
    (dict(cu=fake(9), num_seqs=-1, B=1), INV),
    (dict(B=1 << 20, T=1 << 12), UNS),                         # B * T = 2^32 rows
    (dict(x=fake(1, 8)), ALI), (dict(bias=fake(3, 4)), ALI), (dict(stateT=fake(6, 2)), ALI),
    (dict(cu=fake(9, 4), num_seqs=1, B=1), ALI),
    (dict(y=fake(1)), INV), (dict(y=fake(1, 256)), INV), (dict(stateT=fake(4)), INV),
    (dict(stateT=fake(5, 1024)), INV), (dict(y=fake(2, 16)), INV),
    (dict(B=0, cu=None, stateT=None), OK), (dict(T=0, B=0, x=None, y=None), OK),
])
def test_conv_fwd_refuses(kw, status):
    assert call("osdn_conv_fwd", "x weight bias state0 silu y stateT cu num_seqs B T C W io stream",
                CONV, kw) == status


STEP = dict(x=fake(1), weight=fake(2), bias=None, state=fake(4), silu=1, y=fake(5), N=4, C=64, W=4,
            io=F32, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), INV), (dict(C=0), INV), (dict(W=9), UNS), (dict(state=None), INV),
    (dict(x=None), INV), (dict(y=fake(1)), INV), (dict(state=fake(1)), INV),
    (dict(y=fake(4, 64)), INV), (dict(state=fake(4, 8)), ALI), (dict(io=2), INV),
    (dict(N=0, x=None, state=None, y=None), OK),
])
def test_conv_step_refuses(kw, status):
    assert call("osdn_conv_step", "x weight bias state silu y N C W io stream", STEP, kw) == status


BWD = dict(x=fake(1), weight=fake(2), bias=fake(3), state0=fake(4), silu=1, dy=fake(5), dy_io=BF,
           dstateT=fake(6), dx=fake(7), dweight=fake(8), dbias=fake(9), dstate0=fake(10), cu=None,
           num_seqs=0, B=2, T=64, C=96, W=3, io=BF, ws=fake(11), ws_bytes=SPACE, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), INV), (dict(dx=None), INV), (dict(dweight=None), INV), (dict(dy_io=7), INV),
    (dict(io=F32, dy_io=BF), INV), (dict(W=6), UNS), (dict(ws=None), INV), (dict(ws_bytes=64), INV),
    (dict(ws=fake(11, 16)), ALI), (dict(dx=fake(1)), INV), (dict(dx=fake(5)), INV),
    (dict(dweight=fake(11, 256)), INV), (dict(dstate0=fake(6)), INV), (dict(dbias=fake(8, 16)), INV),
    (dict(dstateT=fake(6, 4)), ALI),
])
def test_conv_bwd_refuses(kw, status):
    assert call("osdn_conv_bwd", "x weight bias state0 silu dy dy_io dstateT dx dweight dbias "
                "dstate0 cu num_seqs B T C W io ws ws_bytes stream", BWD, kw) == status


# --------------------------------------------------------------------------------------- scan
SSM = dict(x=fake(1), dt=fake(2), A=fake(3), b=fake(4), c=fake(5), D=fake(6), dt_bias=fake(7),
           softplus=1, S0=fake(8), y=fake(9), ST=fake(10), cu=None, num_seqs=0, B=2, T=8, H=4, G=2,
           Dk=128, Dv=64, io=BF, ws=fake(11), ws_bytes=SPACE, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(H=0), INV), (dict(G=0), INV), (dict(G=3), INV), (dict(H=2, G=4), INV),
    (dict(Dk=96), UNS), (dict(Dv=32), UNS), (dict(softplus=3), INV), (dict(io=9), INV),
    (dict(x=None), INV), (dict(dt=None), INV), (dict(A=None), INV), (dict(b=None), INV),
    (dict(c=None), INV), (dict(y=None), INV), (dict(T=-2), INV),
    (dict(cu=fake(12), num_seqs=2), INV), (dict(cu=fake(12), num_seqs=0, B=1), INV),
    (dict(B=1 << 16, T=1 << 15), UNS),
    (dict(dt=fake(2, 4)), ALI), (dict(S0=fake(8, 8)), ALI),
    (dict(y=fake(1)), INV), (dict(ST=fake(8)), INV), (dict(ST=fake(9, 256)), INV),
    (dict(y=fake(4, 512)), INV),
])
def test_ssm_fwd_refuses(kw, status):
    assert call("osdn_ssm_fwd", "x dt A b c D dt_bias softplus S0 y ST cu num_seqs B T H G Dk Dv io "
                "ws ws_bytes stream", SSM, kw) == status


SSTEP = dict(x=fake(1), dt=fake(2), A=fake(3), b=fake(4), c=fake(5), D=fake(6), dt_bias=fake(7),
             softplus=1, S=fake(8), y=fake(9), N=3, H=4, G=2, Dk=128, Dv=64, io=BF, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), INV), (dict(G=3), INV), (dict(Dk=32), UNS), (dict(S=None), INV),
    (dict(y=fake(1)), INV), (dict(S=fake(9)), INV), (dict(S=fake(8, 4)), ALI),
    (dict(N=0, x=None, S=None, y=None), OK), (dict(N=1 << 30, H=4, G=1), UNS),
])
def test_ssm_step_refuses(kw, status):
    assert call("osdn_ssm_step", "x dt A b c D dt_bias softplus S y N H G Dk Dv io stream", SSTEP,
                kw) == status


SBWD = dict(x=fake(1), dt=fake(2), A=fake(3), b=fake(4), c=fake(5), D=fake(6), dt_bias=fake(7),
            softplus=1, S0=fake(8), dy=fake(9), dST=fake(10), dx=fake(11), ddt=fake(12),
            dA=fake(13), db=fake(14), dc=fake(15), dD=fake(16), ddt_bias=fake(17), dS0=fake(18),
            cu=None, num_seqs=0, B=2, T=8, H=4, G=2, Dk=128, Dv=64, io=BF, ws=fake(19),
            ws_bytes=SPACE, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), INV), (dict(dx=None), INV), (dict(ddt=None), INV), (dict(dA=None), INV),
    (dict(db=None), INV), (dict(dc=None), INV), (dict(G=3), INV), (dict(Dv=100), UNS),
    (dict(ws=None), INV), (dict(ws_bytes=1000), INV), (dict(ws=fake(19, 64)), ALI),
    (dict(dx=fake(9)), INV), (dict(db=fake(14), dc=fake(14, 256)), INV), (dict(dS0=fake(10)), INV),
    (dict(ddt=fake(2)), INV), (dict(dD=fake(13)), INV), (dict(dx=fake(19, 4096)), INV),
    (dict(dST=fake(10, 4)), ALI),
])
def test_ssm_bwd_refuses(kw, status):
    assert call("osdn_ssm_bwd", "x dt A b c D dt_bias softplus S0 dy dST dx ddt dA db dc dD ddt_bias "
                "dS0 cu num_seqs B T H G Dk Dv io ws ws_bytes stream", SBWD, kw) == status


# --------------------------------------------------------------------------------------- norm
NORM = dict(f=fake(1), x=fake(2), gate=fake(3), w_post=fake(4), w_next=fake(5), act=0, first=0,
            scale=1.0, eps=1e-5, x_out=fake(6), h=fake(7), R=4, D=64, io=BF, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(R=-1), INV), (dict(D=0), INV), (dict(D=8200), UNS), (dict(act=2), INV),
    (dict(first=2), INV), (dict(io=3), INV), (dict(f=None), INV), (dict(h=None), INV),
    (dict(w_next=None), INV),                                   # h without w_next
    (dict(w_next=None, h=None, x_out=None), INV),               # nothing to write
    (dict(x_out=fake(2)), INV), (dict(h=fake(6, 64)), INV), (dict(gate=fake(3, 2)), ALI),
    (dict(x_out=fake(4)), INV), (dict(R=0, f=None, x_out=None, h=None), OK),
])
def test_norm_fwd_refuses(kw, status):
    assert call("osdn_norm_fwd", "f x gate w_post w_next act first scale eps x_out h R D io stream",
                NORM, kw) == status


NBWD = dict(f=fake(1), x=fake(2), gate=fake(3), w_post=fake(4), w_next=fake(5), act=0, first=0,
            scale=1.0, eps=1e-5, dx_out=fake(6), dh=fake(7), df=fake(8), dx=fake(9),
            dgate=fake(10), dw_post=fake(11), dw_next=fake(12), R=4, D=64, io=BF, ws=fake(13),
            ws_bytes=SPACE, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(df=None), INV), (dict(dgate=None), INV), (dict(gate=None), INV), (dict(dh=None), INV),
    (dict(w_next=None), INV), (dict(dw_next=None), INV), (dict(dw_post=None), INV),
    (dict(w_post=None), INV), (dict(x=None), INV), (dict(ws=None), INV), (dict(ws_bytes=8), INV),
    (dict(ws=fake(13, 128)), ALI), (dict(df=fake(1)), INV), (dict(dx=fake(6)), INV),
    (dict(dw_post=fake(12)), INV), (dict(D=9000), UNS), (dict(dh=fake(7, 4)), ALI),
    (dict(w_next=None, dw_next=None, dh=None, dx_out=None), INV),
])
def test_norm_bwd_refuses(kw, status):
    assert call("osdn_norm_bwd", "f x gate w_post w_next act first scale eps dx_out dh df dx dgate "
                "dw_post dw_next R D io ws ws_bytes stream", NBWD, kw) == status


def test_workspace_sizes():
    assert L.osdn_conv_bwd_workspace_bytes(2, 64, 96, 3) > 0
    assert L.osdn_conv_bwd_workspace_bytes(2, 64, 96, 9) == 0
    assert L.osdn_ssm_bwd_workspace_bytes(0, 2, 64, 4, 128, 64, BF) > 0
    assert L.osdn_ssm_bwd_workspace_bytes(0, 2, 64, 4, 96, 64, BF) == 0
    assert L.osdn_ssm_fwd_workspace_bytes(0, 2, 64, 4, 128, 64, F32) == 0
    assert L.osdn_norm_bwd_workspace_bytes(16, 64) >= 2 * 64 * 4
    assert L.osdn_norm_bwd_workspace_bytes(16, 9000) == 0


# ------------------------------------------------------------------- the binding's own refusals
def test_binding_refuses_host_tensors():
    import torch
    x, w = torch.zeros(1, 2, 8), torch.zeros(8, 4)
    with pytest.raises(ValueError, match="CUDA"):
        osdn.osdn_conv_fwd(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        osdn.osdn_norm_fwd(x)
