"""One token of the short convolution: y or the state over what other threads
still read is turned away on the host (CPU)."""
import ctypes

import pytest

import selective_state_space_25_amd as ss

BAD = ss.ERR_INVALID_ARG
AT = 1 << 20   # addresses far apart; never dereferenced: validation fails first


def conv_step(batch=3, x_batch=12, in_dtype=ss.BF16, out_dtype=ss.F32, **at):
    """12 channels, width 4."""
    p = dict(state=AT, x=2 * AT, w=3 * AT, y=4 * AT)
    p.update(at)
    s = ss.ShortConvShape(batch, 1, 12, 4, 0, x_batch, (ctypes.c_int64 * 3)(12), in_dtype, out_dtype, None, 0)
    return ss.lib().selscan_short_conv_step(ctypes.byref(s), p["state"], p["x"], p["w"], None, 1, p["y"], None)


@pytest.mark.parametrize("kw", [
    dict(y=2 * AT), dict(batch=1, y=2 * AT), dict(in_dtype=ss.F32, out_dtype=ss.BF16, y=2 * AT),       # another type
    dict(out_dtype=ss.BF16, y=2 * AT, x_batch=16), dict(out_dtype=ss.BF16, y=2 * AT, x_batch=0),       # rows elsewhere
    dict(out_dtype=ss.BF16, y=2 * AT + 2), dict(out_dtype=ss.BF16, y=2 * AT - 2), dict(y=2 * AT + 70), dict(y=2 * AT - 142),
    dict(y=AT), dict(y=AT + 214), dict(y=AT - 142), dict(state=2 * AT), dict(x=AT + 214), dict(x=AT - 70)])
def test_conv_step(kw):
    assert conv_step(**kw) == BAD and "alias" in ss.last_error()
