"""RMS norm: outputs over inputs other than element by element are turned away
on the host (CPU)."""
import ctypes

import pytest

import selective_state_space_25_amd as ss

BAD, F32, BF16, E4M3 = ss.ERR_INVALID_ARG, ss.F32, ss.BF16, ss.E4M3
AT = 1 << 22   # addresses far apart; never dereferenced: validation fails first


def shape(in_dtype=BF16, res_dtype=BF16, out_dtype=BF16, rows=4, dim=24, gate_row=40):
    return ss.RmsShape(rows, dim, 1, gate_row, 0, in_dtype, res_dtype, out_dtype, 1e-5, None, 0)


def fwd(s, x=AT, res=None, gate=None, y=2 * AT, res_out=None):
    return ss.lib().selscan_rms_norm_fwd(ctypes.byref(s), x, res, gate, None, y, res_out, None, 9 * AT, None)


def bwd(s, dy=AT, x=2 * AT, gate=None, dr=None, dx=None, dres=None, dgate=None, dw=None):
    return ss.lib().selscan_rms_norm_bwd(ctypes.byref(s), dy, x, gate, None, 3 * AT, dr, dx, dres, dgate, dw, None)


# 4 rows of 24: 192 bytes in bf16, 384 in fp32, 96 in e4m3
@pytest.mark.parametrize("types,at", [
    (dict(out_dtype=F32), dict(y=AT)), (dict(out_dtype=E4M3), dict(y=AT)), (dict(in_dtype=F32, out_dtype=E4M3), dict(y=AT)),
    ({}, dict(y=AT + 2)), ({}, dict(y=AT + 190)), (dict(out_dtype=F32), dict(y=AT - 380)),
    (dict(res_dtype=F32), dict(res=3 * AT, res_out=AT)), (dict(res_dtype=F32), dict(res=3 * AT, y=3 * AT)),
    ({}, dict(res=3 * AT, res_out=2 * AT)), ({}, dict(res=3 * AT, res_out=3 * AT + 48)), ({}, dict(gate=2 * AT)),
    ({}, dict(gate=2 * AT - 40)), (dict(out_dtype=E4M3), dict(gate=2 * AT - 280))])
def test_forward(types, at):
    assert fwd(shape(**types), **at) == BAD and "alias" in ss.last_error()


@pytest.mark.parametrize("types,at", [
    (dict(out_dtype=F32), dict(dx=AT)), (dict(res_dtype=F32), dict(dx=2 * AT)), ({}, dict(dx=AT + 2)), ({}, dict(dx=2 * AT + 190)),
    ({}, dict(dx=4 * AT, dres=4 * AT)), (dict(res_dtype=F32), dict(dr=5 * AT, dx=5 * AT)), ({}, dict(dr=5 * AT, dres=5 * AT + 2)),
    ({}, dict(gate=6 * AT, dgate=6 * AT)), ({}, dict(gate=6 * AT, dx=7 * AT, dgate=7 * AT))])
def test_gradients(types, at):
    assert bwd(shape(**types), **at) == BAD and "alias" in ss.last_error()


@pytest.mark.parametrize("at", [dict(dx=AT), dict(dx=2 * AT), dict(gate=6 * AT, dgate=6 * AT), dict(dres=2 * AT)])
def test_long_groups_read_twice(at):
    """dweight of a group past 8192 is made after the other gradients, from the same inputs."""
    assert bwd(shape(dim=8200, gate_row=8200), dw=8 * AT, **at) == BAD and "alias" in ss.last_error()
