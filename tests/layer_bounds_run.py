"""Runs the operators around the mixer with whichever library build OSDN_LIBRARY selects on fixed
seeded inputs and writes each output tensor's SHA-256 and the status word per call, as JSON; what
tests/debug_bounds_run.py does for the mixer's entry points.

Usage: ``python -m tests.layer_bounds_run OUT.json``
"""
import json
import sys

import numpy as np
import torch

from delta_rule_recurrent_osdn_b200 import osdn
from tests.debug_bounds_run import digest

LENS = [1, 33, 0, 128, 100, 300, 0, 7]


def draw(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *s, dtype=torch.float32: torch.randn(*s, generator=g).to("cuda", dtype)


def offsets(lens):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).cuda()


def conv_case(dtype, C, W, seed):
    mk, n, N = draw(seed), sum(LENS), len(LENS)
    x, w, bias = mk(1, n, C, dtype=dtype), mk(C, W), mk(C)
    s0, cu = mk(N, W - 1, C, dtype=dtype), offsets(LENS)
    y, sT = osdn.osdn_conv_fwd(x, w, bias, s0, cu_seqlens=cu)
    out = dict(y=y, sT=sT)
    out.update(osdn.osdn_conv_bwd(x, w, mk(1, n, C, dtype=dtype), bias, s0, mk(N, W - 1, C),
                                  cu_seqlens=cu))
    out["step"] = osdn.osdn_conv_step(mk(N, C, dtype=dtype), w, sT, bias)
    return out


def ssm_case(dtype, lens, H, G, Dk, Dv, seed):
    mk, n, N = draw(seed), sum(lens), len(lens)
    x, dy = mk(1, n, H, Dv, dtype=dtype), mk(1, n, H, Dv, dtype=dtype)
    b, c = mk(1, n, G, Dk, dtype=dtype), mk(1, n, G, Dk, dtype=dtype)
    dt, A, D, bias = mk(1, n, H) - 2, -mk(H).abs(), mk(H), 0.1 * mk(H)
    S0, dST, cu = mk(N, H, Dv, Dk), mk(N, H, Dv, Dk), offsets(lens)
    y, ST = osdn.osdn_ssm_fwd(x, dt, A, b, c, D, bias, True, S0, cu)
    out = dict(y=y, ST=ST.clone())
    out.update(osdn.osdn_ssm_bwd(x, dt, A, b, c, dy, D, bias, True, S0, dST, cu))
    first = lambda t: t[0, :N].clone()  # noqa: E731
    out["step"] = osdn.osdn_ssm_step(first(x), first(dt), A, first(b), first(c), ST, D, bias)
    return out


def norm_case(dtype, R, D, seed):
    mk = draw(seed)
    f, x, z = (mk(R, D, dtype=dtype) for _ in range(3))
    w = dict(x=x, gate=z, w_post=mk(D), w_next=mk(D))
    x_out, h = osdn.osdn_norm_fwd(f, **w)
    out = dict(x_out=x_out, h=h)
    out.update(osdn.osdn_norm_bwd(f, mk(R, D, dtype=dtype), mk(R, D, dtype=dtype), **w))
    return out


B16, F32 = torch.bfloat16, torch.float32
CASES = {
    "conv_bf16": lambda: conv_case(B16, 264, 4, 1),
    "conv_bf16_odd": lambda: conv_case(B16, 77, 3, 2),
    "conv_f32": lambda: conv_case(F32, 132, 2, 3),
    "ssm_bf16": lambda: ssm_case(B16, LENS, 4, 4, 128, 128, 4),
    "ssm_bf16_groups": lambda: ssm_case(B16, LENS, 6, 2, 64, 128, 5),
    "ssm_bf16_segments": lambda: ssm_case(B16, [4000, 90], 2, 1, 128, 64, 6),
    "ssm_f32": lambda: ssm_case(F32, LENS, 4, 2, 64, 64, 7),
    "ssm_f32_segments": lambda: ssm_case(F32, [3000, 5], 2, 1, 128, 128, 8),
    "norm_bf16": lambda: norm_case(B16, 1001, 128, 9),
    "norm_f32_odd": lambda: norm_case(F32, 37, 1001, 10),
    "norm_bf16_wide": lambda: norm_case(B16, 5, 8192, 11),
}


def main(path):
    torch.cuda.set_device(0)
    res = {"library": osdn.LIB_PATH}
    for name, fn in CASES.items():
        out = fn()
        torch.cuda.synchronize()
        res[name] = {"status": osdn.osdn_get_device_status(),
                     "outputs": {k: digest(v) for k, v in out.items()}}
    with open(path, "w") as f:
        json.dump(res, f, indent=1)


if __name__ == "__main__":
    main(sys.argv[1])
