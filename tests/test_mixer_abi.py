"""Refusals of the short convolution, the Mamba-2 mixer and RMS norm: bad
arguments are turned away on the host before any device work (CPU)."""
import ctypes

import pytest
import torch

import selective_state_space_25_amd as ss

FAKE = 4096   # a non-null pointer value; never dereferenced because validation fails first
BAD, NO = ss.ERR_INVALID_ARG, ss.ERR_UNSUPPORTED


def conv(**kw):
    base = dict(batch=2, seqlen=8, dim=12, width=4, x_row=12, x_batch=96, split=(8, 2, 2), in_dtype=ss.BF16, out_dtype=ss.F32)
    base.update(kw)
    return ss.ShortConvShape(*(base[k] for k in ("batch", "seqlen", "dim", "width", "x_row", "x_batch")),
                             (ctypes.c_int64 * 3)(*base["split"]), base["in_dtype"], base["out_dtype"], None, 0)


def conv_fwd(s, x=FAKE, w=FAKE, silu=1, state=None, y=(FAKE,) * 3, last=None):
    return ss.lib().selscan_short_conv_fwd(None if s is None else ctypes.byref(s), x, w, None, silu, None, state, *y, last, None)


def conv_bwd(s, x=FAKE, w=FAKE, silu=1, dy=(FAKE,) * 3, dx=FAKE):
    return ss.lib().selscan_short_conv_bwd(None if s is None else ctypes.byref(s), x, w, None, silu, None, None, *dy, None, dx,
                                           FAKE, None, None, None)


def conv_step(s, state=FAKE, x=FAKE, w=FAKE, silu=1, y=FAKE):
    return ss.lib().selscan_short_conv_step(None if s is None else ctypes.byref(s), state, x, w, None, silu, y, None)


SHARED = [("batch", 0, BAD), ("dim", 0, BAD), ("width", 0, BAD), ("width", 1, NO), ("width", 5, NO), ("in_dtype", 2, NO),
          ("out_dtype", 2, NO), ("x_batch", -1, BAD), ("x_batch", 1 << 62, BAD), ("dim", 1 << 62, BAD)]


@pytest.mark.parametrize("field,value,status", SHARED + [
    ("seqlen", 0, BAD), ("x_row", -1, BAD), ("x_row", 1 << 61, BAD), ("split", (0, 6, 6), BAD), ("split", (8, 2, 3), BAD),
    ("split", (12, -1, 1), BAD), ("split", (1 << 62, 1 << 62, 12), BAD)])
def test_conv_bad_shape(field, value, status):
    s = conv(**{field: value})
    assert conv_fwd(s) == status and ss.last_error()
    assert conv_bwd(s) == status and ss.last_error()
    assert ss.lib().selscan_short_conv_bwd_workspace_bytes(ctypes.byref(s)) == 0


@pytest.mark.parametrize("field,value,status", SHARED)
def test_conv_step_bad_shape(field, value, status):
    assert conv_step(conv(**{field: value})) == status and ss.last_error()


def test_conv_null_and_alias():
    s = conv()
    assert conv_fwd(None) == conv_bwd(None) == conv_step(None) == BAD
    assert conv_fwd(s, x=None) == conv_fwd(s, w=None) == conv_fwd(s, silu=2) == BAD
    for i in range(3):
        y = tuple(None if j == i else FAKE for j in range(3))
        assert conv_fwd(s, y=y) == conv_bwd(s, dy=y) == BAD
    assert conv_fwd(s, state=FAKE, last=FAKE) == BAD and "alias" in ss.last_error()
    assert conv_bwd(s, x=None) == conv_bwd(s, w=None) == conv_bwd(s, dx=None) == conv_bwd(s, silu=-1) == BAD
    assert conv_step(s, state=None) == conv_step(s, x=None) == conv_step(s, w=None) == conv_step(s, y=None) == BAD


def test_conv_too_many_elements_for_a_launch():
    assert conv_fwd(conv(seqlen=1 << 57, x_row=0, x_batch=0)) in (BAD, NO)
    assert conv_fwd(conv(batch=1 << 40, x_batch=0)) in (BAD, NO)
    assert conv_step(conv(batch=1 << 40, x_batch=0)) in (BAD, NO)


def test_conv_gradients_past_the_sums_launch():
    """(width + 1) dim columns, and partial rows, that one launch adds up."""
    size = lambda s: ss.lib().selscan_short_conv_bwd_workspace_bytes(ctypes.byref(s))
    for kw in [dict(dim=(1 << 24) + 4, split=((1 << 24), 2, 2)), dict(batch=1 << 27, x_batch=0, dim=1, split=(1, 0, 0)),
               dict(seqlen=1 << 40, x_batch=0, x_row=0, dim=1, split=(1, 0, 0))]:
        s = conv(**kw)
        assert conv_bwd(s) == NO and size(s) == 0
    assert size(conv(dim=1 << 24, split=((1 << 24) - 4, 2, 2))) > 0


def mixer(**kw):
    base = dict(batch=2, seqlen=8, nheads=4, headdim=8, ngroups=2, dstate=16, width=4, xbc_row=96, xbc_batch=768, dt_row=4,
                dt_batch=32, in_dtype=ss.BF16, out_dtype=ss.F32)
    base.update(kw)
    return ss.M2ConvShape(*(base[k] for k in ("batch", "seqlen", "nheads", "headdim", "ngroups", "dstate", "width", "xbc_row",
                                              "xbc_batch", "dt_row", "dt_batch", "in_dtype", "out_dtype")), None, 0)


def mixer_fwd(s, ptrs=(FAKE,) * 5, h0=None, cs=None, last=None, last_cs=None):
    xbc, dt, w, A, y = ptrs
    return ss.lib().selscan_mamba2_conv_fwd(None if s is None else ctypes.byref(s), xbc, dt, w, None, A, None, None, None, h0, cs,
                                            y, last, last_cs, None)


def mixer_step(s, ptrs=(FAKE,) * 7):
    state, cs, xbc, dt, w, A, y = ptrs
    return ss.lib().selscan_mamba2_conv_step(None if s is None else ctypes.byref(s), state, cs, xbc, dt, w, None, A, None, None, y,
                                             None)


MIXER = [("batch", 0, BAD), ("nheads", 0, BAD), ("headdim", -1, BAD), ("ngroups", 3, BAD), ("dstate", 17, NO), ("dstate", 256, NO),
         ("width", 0, BAD), ("width", 5, NO), ("in_dtype", 2, NO), ("out_dtype", -1, NO), ("xbc_batch", -1, BAD),
         ("dt_batch", -2, BAD), ("headdim", 1 << 61, BAD), ("nheads", 1 << 62, BAD), ("headdim", 1 << 21, NO)]


@pytest.mark.parametrize("field,value,status", MIXER + [("seqlen", 0, BAD), ("xbc_row", -1, BAD), ("dt_row", 1 << 62, BAD)])
def test_mixer_bad_shape(field, value, status):
    s = mixer(**{field: value})
    assert mixer_fwd(s) == status and ss.last_error()
    assert ss.lib().selscan_mamba2_conv_workspace_bytes(ctypes.byref(s)) == 0


@pytest.mark.parametrize("field,value,status", MIXER)
def test_mixer_step_bad_shape(field, value, status):
    assert mixer_step(mixer(**{field: value})) == status and ss.last_error()


def test_mixer_past_a_launch():
    """Chunks, segments' states and their bytes that no launch holds."""
    for kw in [dict(seqlen=1 << 43, xbc_row=0, dt_row=0, xbc_batch=0, dt_batch=0),
               dict(seqlen=1 << 51, xbc_row=0, dt_row=0, xbc_batch=0, dt_batch=0),
               dict(batch=1 << 31, seqlen=4096, xbc_batch=0, dt_batch=0, ngroups=4)]:
        s = mixer(**kw)
        assert mixer_fwd(s) in (BAD, NO) and ss.lib().selscan_mamba2_conv_workspace_bytes(ctypes.byref(s)) == 0
    s = mixer(batch=1 << 20, seqlen=4096)
    assert ss.lib().selscan_mamba2_conv_workspace_bytes(ctypes.byref(s)) > 0


def test_mixer_null_alias_and_alignment():
    s = mixer()
    assert mixer_fwd(None) == mixer_step(None) == BAD
    for i in range(5):
        assert mixer_fwd(s, tuple(None if j == i else FAKE for j in range(5))) == BAD
    for i in range(7):
        assert mixer_step(s, tuple(None if j == i else FAKE for j in range(7))) == BAD
    assert mixer_fwd(s, h0=FAKE, last=FAKE) == BAD and "alias" in ss.last_error()
    assert mixer_fwd(s, cs=FAKE, last_cs=FAKE) == BAD and "alias" in ss.last_error()
    assert mixer_step(s, (FAKE + 4,) + (FAKE,) * 6) == BAD and "aligned" in ss.last_error()


def rms(**kw):
    base = dict(rows=4, dim=24, groups=1, gate_row=24, scale_block=0, in_dtype=ss.BF16, res_dtype=ss.F32, out_dtype=ss.BF16,
                eps=1e-5)
    base.update(kw)
    return ss.RmsShape(*(base[k] for k in ("rows", "dim", "groups", "gate_row", "scale_block", "in_dtype", "res_dtype",
                                           "out_dtype", "eps")), None, 0)


def rms_fwd(s, x=FAKE, res=None, gate=None, y=FAKE, res_out=None, scale=None):
    return ss.lib().selscan_rms_norm_fwd(None if s is None else ctypes.byref(s), x, res, gate, None, y, res_out, None, scale, None)


def rms_bwd(s, dy=FAKE, x=FAKE, gate=None, rstd=FAKE, dr=None, dx=FAKE, dres=None, dgate=None):
    return ss.lib().selscan_rms_norm_bwd(None if s is None else ctypes.byref(s), dy, x, gate, None, rstd, dr, dx, dres, dgate, None,
                                         None)


@pytest.mark.parametrize("field,value,status", [
    ("rows", 0, BAD), ("dim", 0, BAD), ("groups", 0, BAD), ("groups", 5, BAD), ("gate_row", -1, BAD), ("scale_block", 16, NO),
    ("scale_block", 96, NO), ("scale_block", 1024, NO), ("scale_block", -32, NO), ("in_dtype", 2, NO), ("res_dtype", 2, NO),
    ("out_dtype", 3, NO), ("eps", -1.0, BAD), ("eps", float("nan"), BAD), ("rows", 1 << 31, NO), ("rows", 1 << 62, BAD),
    ("dim", 1 << 27, NO)])
def test_rms_bad_shape(field, value, status):
    s = rms(**{field: value})
    assert rms_fwd(s) == status and ss.last_error()
    assert rms_bwd(s) == status and ss.last_error()
    assert ss.lib().selscan_rms_norm_bwd_workspace_bytes(ctypes.byref(s)) == 0


def test_rms_combinations():
    s = rms()
    assert rms_fwd(None) == rms_bwd(None) == BAD
    assert rms_fwd(s, x=None) == rms_fwd(s, y=None) == BAD
    assert rms_fwd(s, gate=FAKE, res=FAKE) == rms_fwd(s, gate=FAKE, res_out=FAKE) == NO
    assert rms_fwd(rms(out_dtype=ss.E4M3)) == BAD and "scale" in ss.last_error()
    assert rms_bwd(rms(out_dtype=ss.E4M3)) == NO
    assert rms_bwd(s, dy=None) == rms_bwd(s, x=None) == rms_bwd(s, rstd=None) == rms_bwd(s, dx=None) == BAD
    assert rms_bwd(s, gate=FAKE) == NO            # s is x: its type is in_dtype
    b = rms(res_dtype=ss.BF16)
    assert rms_bwd(b, gate=FAKE, dr=FAKE) == rms_bwd(b, gate=FAKE, dres=FAKE) == NO
    assert rms_bwd(b, dgate=FAKE) == BAD


def test_tensors_off_the_gpu():
    x, w = torch.zeros(1, 4, 8), torch.zeros(8, 4)
    for call in (lambda: ss.short_conv_fwd(x, w), lambda: ss.short_conv_bwd(x, w, None, x), lambda: ss.rms_norm_fwd(x),
                 lambda: ss.short_conv_step(torch.zeros(1, 3, 8), x[:, 0], w), lambda: ss.rms_norm_bwd(x, x, None, x[..., :1]),
                 lambda: ss.mamba2_conv_fwd(x, x[..., :1], w, None, w[0], ngroups=1, dstate=2)):
        with pytest.raises(ValueError, match="GPU"):
            call()


@pytest.mark.parametrize("rows,dim,groups", [(1, 3, 1), (70, 8192, 1), (1 << 20, 2560, 1), (1 << 22, 64, 1), (300, 20000, 1),
                                             (1 << 30, 8, 2), (5, 16384, 4)])
def test_rms_workspace_holds_a_row_for_each_workgroup(rows, dim, groups):
    """At least one partial row and no more than one for each row, with the room for their sums."""
    n = ss.lib().selscan_rms_norm_bwd_workspace_bytes(ctypes.byref(rms(rows=rows, dim=dim, groups=groups)))
    assert 4 * dim <= n <= 4 * dim * (rows + rows // 512 + 2) + 256


def test_outputs_over_inputs():
    """The convolution reads tokens that other threads' outputs would be written over."""
    s = conv()
    for i in range(3):
        y = tuple(FAKE if j == i else 2 * FAKE for j in range(3))
        assert conv_fwd(s, y=y) == BAD and "alias" in ss.last_error()
        assert conv_bwd(s, dy=y, x=3 * FAKE) == BAD and "alias" in ss.last_error()
    assert conv_bwd(s, dy=(2 * FAKE,) * 3) == BAD and "alias" in ss.last_error()
    m = mixer()
    assert mixer_fwd(m, (FAKE, 2 * FAKE, FAKE, FAKE, FAKE)) == BAD and "alias" in ss.last_error()
    assert mixer_fwd(m, (2 * FAKE, FAKE, FAKE, FAKE, FAKE)) == BAD and "alias" in ss.last_error()
