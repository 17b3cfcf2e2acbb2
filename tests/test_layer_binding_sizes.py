"""Sizes past 32 bits at the layer operators' binding, without a GPU: the C entry points take int32,
and a size cut to its lower half would pass as another, smaller one."""
import pytest
import torch

osdn = pytest.importorskip("delta_rule_recurrent_osdn_b200.osdn")
BIG = 2 ** 32


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


def f32(*shape):
    return meta(*shape, dtype=torch.float32)


def i32(n):
    return meta(n, dtype=torch.int32)


CALLS = {
    "conv_fwd channels": (osdn.osdn_conv_fwd, (meta(1, 1, BIG + 4), f32(BIG + 4, 4)), {}),
    "conv_fwd tokens": (osdn.osdn_conv_fwd, (meta(1, BIG + 5, 1), f32(1, 2)), {}),
    "conv_fwd batch": (osdn.osdn_conv_fwd, (meta(BIG + 2, 1, 1), f32(1, 2)), {}),
    "conv_fwd taps": (osdn.osdn_conv_fwd, (meta(1, 4, 1), f32(1, BIG + 4)), dict(return_state=False)),
    "conv_fwd sequences": (osdn.osdn_conv_fwd, (meta(1, 4, 1), f32(1, 2)),
                           dict(cu_seqlens=i32(BIG + 2), return_state=False)),
    "conv_fwd heads": (osdn.osdn_conv_fwd, (meta(1, 1, BIG // 64 + 1, 64), f32(BIG + 64, 4)), {}),
    "conv_step batch": (osdn.osdn_conv_step, (meta(BIG + 1, 1), f32(1, 2), meta(BIG + 1, 1, 1)), {}),
    "conv_step channels": (osdn.osdn_conv_step, (meta(1, BIG + 1), f32(BIG + 1, 2), meta(1, 1, BIG + 1)), {}),
    "conv_bwd tokens": (osdn.osdn_conv_bwd, (meta(1, BIG + 5, 1), f32(1, 2), meta(1, BIG + 5, 1)), {}),
    "conv_bwd channels": (osdn.osdn_conv_bwd, (meta(1, 1, BIG + 4), f32(BIG + 4, 4), meta(1, 1, BIG + 4)), {}),
    "ssm_fwd tokens": (osdn.osdn_ssm_fwd, (meta(1, BIG + 8, 1, 64), f32(1, BIG + 8, 1), f32(1),
                                           meta(1, BIG + 8, 1, 64), meta(1, BIG + 8, 1, 64)), {}),
    "ssm_fwd sequences": (osdn.osdn_ssm_fwd, (meta(1, 8, 1, 64), f32(1, 8, 1), f32(1), meta(1, 8, 1, 64),
                                              meta(1, 8, 1, 64)),
                          dict(cu_seqlens=i32(BIG + 2), return_ST=False)),
    "ssm_step batch": (osdn.osdn_ssm_step, (meta(BIG + 1, 1, 64), f32(BIG + 1, 1), f32(1), meta(BIG + 1, 1, 64),
                                            meta(BIG + 1, 1, 64), f32(BIG + 1, 1, 64, 64)), {}),
    "ssm_bwd tokens": (osdn.osdn_ssm_bwd, (meta(1, BIG + 8, 1, 64), f32(1, BIG + 8, 1), f32(1),
                                           meta(1, BIG + 8, 1, 64), meta(1, BIG + 8, 1, 64),
                                           meta(1, BIG + 8, 1, 64)), {}),
    "ssm_bwd sequences": (osdn.osdn_ssm_bwd, (meta(1, 8, 1, 64), f32(1, 8, 1), f32(1), meta(1, 8, 1, 64),
                                              meta(1, 8, 1, 64), meta(1, 8, 1, 64)),
                          dict(cu_seqlens=i32(BIG + 2))),
    "norm_fwd width": (osdn.osdn_norm_fwd, (meta(1, BIG + 8),), {}),
    "norm_bwd width": (osdn.osdn_norm_bwd, (meta(1, BIG + 8), meta(1, BIG + 8)), {}),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_sizes_past_32_bits_are_refused(monkeypatch, name):
    fn, args, kw = CALLS[name]
    monkeypatch.setattr(osdn, "_raw_stream", lambda index: 0)
    with pytest.raises(osdn.OsdnError) as e:
        fn.__wrapped__(*args, **kw)
    assert e.value.status == osdn.OSDN_ERR_UNSUPPORTED


def test_workspace_sizes_past_32_bits_are_refused():
    with pytest.raises(osdn.OsdnError):
        osdn.osdn_ssm_fwd_workspace_bytes(1, BIG + 8, 1, 64, 64)


@pytest.mark.parametrize("T", [1100, 7112, 65536])
def test_one_sequence_with_offsets_is_cut_like_one_without(T):
    """The forward workspace holds the segments' states, so its size tells how a call is cut."""
    for H in (1, 2, 16):
        assert (osdn.osdn_ssm_fwd_workspace_bytes(1, T, H, 128, 64, num_seqs=1) ==
                osdn.osdn_ssm_fwd_workspace_bytes(1, T, H, 128, 64))
