"""Convolution, its gradients and the mixer over sequences: outputs that overlap
inputs or each other anywhere, not at their first element alone, are turned away
on the host (CPU)."""
import ctypes

import pytest

import selective_state_space_25_amd as ss

BAD = ss.ERR_INVALID_ARG
AT = 1 << 20   # addresses far apart; never dereferenced: validation fails first


def conv(x_row=12, x_batch=96, out_dtype=ss.F32):
    """2 x 8 x 12 bf16, width 4, outputs of 8 and 4 channels."""
    return ss.ShortConvShape(2, 8, 12, 4, x_row, x_batch, (ctypes.c_int64 * 3)(8, 4), ss.BF16, out_dtype, None, 0)


def conv_fwd(s, **at):
    p = dict(x=AT, state=2 * AT, w=3 * AT, y0=4 * AT, y1=5 * AT, y2=None, last=6 * AT)
    p.update(at)
    return ss.lib().selscan_short_conv_fwd(ctypes.byref(s), p["x"], p["w"], None, 1, None, p["state"], p["y0"], p["y1"], p["y2"],
                                           p["last"], None)


X, ST, Y0, Y1 = 2 * 8 * 12 * 2, 2 * 3 * 12 * 2, 2 * 8 * 8 * 4, 2 * 8 * 4 * 4   # bytes


@pytest.mark.parametrize("at", [
    dict(y0=AT), dict(y0=AT + X - 4), dict(y0=AT - Y0 + 4), dict(y1=AT + 8), dict(y0=2 * AT + ST - 2), dict(y1=4 * AT + Y0 - 4),
    dict(last=AT + X - 2), dict(last=2 * AT), dict(last=2 * AT + 8), dict(last=5 * AT + Y1 - 2), dict(last=4 * AT - ST + 2)])
def test_conv(at):
    assert conv_fwd(conv(), **at) == BAD and "alias" in ss.last_error()


@pytest.mark.parametrize("x_row,x_batch", [(1000, 8000), (2000, 1000), (0, 40), (40, 0), (3, 5)])
def test_conv_strided_rows(x_row, x_batch):
    """Each row of x, batch elements outside, inside or over each other."""
    s = conv(x_row, x_batch)
    for b in range(2):
        for t in range(8):
            row = AT + 2 * (b * x_batch + t * x_row)
            for y in (row - Y1 + 4, row, row + 20):
                assert conv_fwd(s, y1=y) == BAD and "alias" in ss.last_error()


def conv_bwd(s, **at):
    p = dict(x=AT, state=2 * AT, w=3 * AT, d0=4 * AT, d1=5 * AT, dlast=6 * AT, dx=7 * AT, dw=8 * AT, db=9 * AT, ds=10 * AT)
    p.update(at)
    return ss.lib().selscan_short_conv_bwd(ctypes.byref(s), p["x"], p["w"], None, 1, None, p["state"], p["d0"], p["d1"], None,
                                           p["dlast"], p["dx"], p["dw"], p["db"], p["ds"], None)


@pytest.mark.parametrize("at", [
    dict(dx=AT + 2), dict(dx=4 * AT + Y0 - 2), dict(dx=5 * AT - X + 2), dict(dx=2 * AT), dict(dx=6 * AT + ST - 2), dict(ds=2 * AT),
    dict(ds=6 * AT + 2), dict(ds=AT + X - 2), dict(ds=7 * AT), dict(dw=4 * AT), dict(dw=7 * AT), dict(db=8 * AT + 188), dict(db=AT)])
def test_conv_gradients(at):
    assert conv_bwd(conv(), **at) == BAD and "alias" in ss.last_error()


def mixer_fwd(**at):
    """2 x 8, 4 heads of 8 x 16 in two groups (96 channels), bf16, y fp32."""
    p = dict(xbc=AT, dt=2 * AT, w=3 * AT, A=4 * AT, h0=5 * AT, cs=6 * AT, y=7 * AT, last=8 * AT, last_cs=9 * AT)
    p.update(at)
    s = ss.M2ConvShape(2, 8, 4, 8, 2, 16, 4, 100, 800, 100, 800, ss.BF16, ss.F32, None, 0)
    return ss.lib().selscan_mamba2_conv_fwd(ctypes.byref(s), p["xbc"], p["dt"], p["w"], None, p["A"], None, None, None, p["h0"],
                                            p["cs"], p["y"], p["last"], p["last_cs"], None)


YB, SB, CB, XB = 2 * 8 * 32 * 4, 2 * 32 * 16 * 4, 2 * 3 * 96 * 2, 15 * 200 + 192


@pytest.mark.parametrize("at", [
    dict(y=AT), dict(y=AT + XB - 4), dict(y=AT - YB + 4), dict(y=2 * AT + 4), dict(y=2 * AT + 15 * 200 + 4), dict(y=5 * AT + SB - 4),
    dict(y=6 * AT + CB - 4), dict(last=5 * AT), dict(last=5 * AT + 16), dict(last=7 * AT + YB - 4), dict(last=AT + XB - 4),
    dict(last_cs=6 * AT), dict(last_cs=6 * AT + 2), dict(last_cs=AT + 200), dict(last_cs=8 * AT + SB - 2), dict(last_cs=2 * AT)])
def test_mixer(at):
    assert mixer_fwd(**at) == BAD and "alias" in ss.last_error()
