"""One token of the mixer: outputs that would be written over what other
workgroups still read are turned away on the host, wherever they lie (CPU)."""
import ctypes

import pytest

import selective_state_space_25_amd as ss

BAD = ss.ERR_INVALID_ARG
AT = 1 << 20   # addresses far apart; never dereferenced: validation fails first


def mixer(batch=3, in_dtype=ss.BF16, out_dtype=ss.F32, xbc_batch=96, dt_batch=4):
    """4 heads of 8 x 16 in two groups: xbc 96 channels, dt 4, y 32, conv_state 3 x 96."""
    return ss.M2ConvShape(batch, 1, 4, 8, 2, 16, 4, 0, xbc_batch, 0, dt_batch, in_dtype, out_dtype, None, 0)


def mixer_step(s, **at):
    p = dict(state=1 * AT, cs=2 * AT, xbc=3 * AT, dt=4 * AT, w=5 * AT, A=6 * AT, y=7 * AT)
    p.update(at)
    return ss.lib().selscan_mamba2_conv_step(ctypes.byref(s), p["state"], p["cs"], p["xbc"], p["dt"], p["w"], None, p["A"], None,
                                             None, p["y"], None)


XBC, DT, CS, STATE, Y = 3 * 96 * 2, 3 * 4 * 2, 3 * 3 * 96 * 2, 3 * 32 * 16 * 4, 3 * 32 * 4   # bytes


@pytest.mark.parametrize("at", [
    dict(y=3 * AT), dict(y=3 * AT + XBC - 2), dict(y=3 * AT - Y + 2), dict(y=4 * AT), dict(y=4 * AT + DT - 2), dict(y=4 * AT - Y + 4),
    dict(y=1 * AT), dict(y=AT + STATE - 4), dict(y=2 * AT + CS - 2), dict(y=2 * AT - Y + 2), dict(cs=3 * AT), dict(cs=3 * AT - CS + 2),
    dict(cs=AT + STATE - 2), dict(state=2 * AT), dict(state=3 * AT - STATE + 16), dict(dt=AT + 64), dict(dt=2 * AT + CS - 2)])
def test_mixer_step(at):
    assert mixer_step(mixer(), **at) == BAD and "alias" in ss.last_error()


def test_mixer_step_between_strided_rows():
    """Rows of xbc 1000 elements apart: y in a gap is no overlap, y over a row is."""
    s = mixer(xbc_batch=1000)
    for row in range(3):
        for y in (3 * AT + 2000 * row - Y + 2, 3 * AT + 2000 * row, 3 * AT + 2000 * row + 190):
            assert mixer_step(s, y=y) == BAD and "alias" in ss.last_error()
    s = mixer(xbc_batch=0)
    assert mixer_step(s, y=3 * AT + 190) == BAD and "alias" in ss.last_error()
