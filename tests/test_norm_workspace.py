"""Workspace of the layer norm gradients: two fp32 partial rows for every
workgroup that has rows to work on, on the CPU."""
import ctypes

import pytest

import selective_state_space_25_amd as ss


@pytest.mark.parametrize("rows,dim,blocks", [
    (1, 768, 1), (5, 2560, 2), (4096, 2560, 512),     # a wave to a row, four rows a workgroup
    (1, 2568, 1), (256, 8192, 256), (300, 4096, 300), (4096, 8192, 512),   # a workgroup to a row
    (32768, 2568, 512), (65536, 2568, 1024),          # 64 rows a workgroup at most
    (1 << 20, 64, 4096 + 4)])                         # and the sums of 1024 partial rows each
def test_partial_rows(rows, dim, blocks):
    s = ss.NormShape(rows, dim, ss.BF16, ss.BF16, ss.BF16, 1e-5, 0.0, 0, 0, None, 0)
    assert ss.lib().selscan_layer_norm_bwd_workspace_bytes(ctypes.byref(s)) == (blocks * 2 * dim * 4 + 255) // 256 * 256
