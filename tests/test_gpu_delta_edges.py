"""The gated delta rule on the GPU where it can go wrong between its plain
cases: the rounding of bf16 outputs, values that are not finite, what calls
hold on to."""
import numpy as np
import pytest
import torch

import selective_state_space_25_amd as ss
from oracle import block_ops as ref
from parity import check_close, host
from test_gpu_delta import BF16, DEV, F32, douts, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(1, 200, 2, 2, 128, 128), (2, 129, 4, 2, 48, 40), (1, 77, 6, 3, 7, 3),
                                   (2, 150, 70, 70, 64, 128), (3, 70, 60, 4, 80, 40), (2, 9, 4, 2, 33, 27)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_bf16_y_is_the_fp32_y_rounded(gpu, shape, dtype):
    """The type that y is written in does not lower the precision of its sums:
    one and two column blocks a workgroup, and token by token."""
    i = inputs(*shape, dtype, seed=300 + sum(shape), h0=True)
    y, last = ss.delta_fwd(**i)
    yb, lastb = ss.delta_fwd(**i, out_dtype=BF16)
    torch.cuda.synchronize()
    assert torch.equal(yb, y.bfloat16())
    assert torch.equal(lastb, last)


@pytest.mark.parametrize("shape", [(1, 200, 2, 2, 128, 128), (2, 129, 4, 2, 48, 40), (1, 77, 6, 3, 7, 3),
                                   (2, 70, 64, 64, 64, 128)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_bf16_gradients_are_the_fp32_ones_rounded(gpu, shape, dtype):
    """bf16 inputs are one plane of the three that fp32 inputs take, the
    others zero: the same products in the same order, rounded at the end.
    dtype: dout's."""
    B, L, H, G, P, N = shape
    i = inputs(*shape, BF16, seed=320 + sum(shape), h0=True)
    dout, dlast = douts(B, L, H, P, N, dtype, 320)
    got = ss.delta_bwd(**i, dout=dout, dlast_state=dlast)
    want = ss.delta_bwd(**{n: x.float() for n, x in i.items()}, dout=dout, dlast_state=dlast)
    torch.cuda.synchronize()
    for n in want:
        assert torch.equal(got[n], want[n].to(got[n].dtype)), n
