"""The gated delta rule's gradients turn away what their launches cannot hold
(fewer than 2^32 threads in a launch: 512 to a chunk, 512 to 16 padded rows of
a head's state), on the host and before any device work."""
import ctypes

import pytest

import selective_state_space_25_amd as ss

FAKE = 4096   # a non-null pointer value; never dereferenced because validation fails first


def shape(batch, seqlen, nheads, headdim, dstate=8):
    return ss.M2Shape(batch, seqlen, nheads, headdim, 1, dstate, ss.BF16, ss.BF16, None, 0)


@pytest.mark.parametrize("sizes", [(1 << 10, 64 * 128, 64, 16),      # 2^23 chunks
                                   (1 << 12, 1, 1 << 10, 16),        # 2^22 heads, 16 rows padded to 32
                                   (1 << 12, 1, 1 << 9, 33)])        # 2^21 heads, 33 rows padded to 64
def test_gradients_refuse_more_than_a_launch(sizes):
    s = shape(*sizes)
    assert ss.lib().selscan_delta_bwd_workspace_bytes(ctypes.byref(s)) == 0
    r = ss.lib().selscan_delta_bwd(ctypes.byref(s), FAKE, FAKE, FAKE, FAKE, FAKE, 1.0, None, None, FAKE, None, FAKE,
                                   FAKE, FAKE, FAKE, FAKE, None, None)
    assert r == ss.ERR_UNSUPPORTED and "launch" in ss.last_error()


@pytest.mark.parametrize("sizes", [(1 << 10, 64 * 128 - 64, 64, 16), (1 << 12, 1, (1 << 10) - 2, 16),
                                   (1 << 12, 1, (1 << 9) - 2, 33)])
def test_gradients_take_what_a_launch_holds(sizes):
    assert ss.lib().selscan_delta_bwd_workspace_bytes(ctypes.byref(shape(*sizes))) > 0


@pytest.mark.parametrize("sizes", [(1 << 10, 64 * 128, 64, 16), (1 << 12, 20, 1 << 10, 16)])
def test_forward_keeps_its_own_limits(sizes):
    assert ss.lib().selscan_delta_workspace_bytes(ctypes.byref(shape(*sizes))) > 0
