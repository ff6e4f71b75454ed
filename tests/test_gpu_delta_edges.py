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


BAD = [("v", float("nan")), ("k", float("inf")), ("q", float("nan")), ("beta", float("inf")), ("g", float("nan")),
       ("h0", float("inf"))]


def spoilt(L, lengths, t, name, value, dtype, seed):
    """Inputs of len(lengths) sequences with one value of sequence 0, head 0,
    token t that is not finite (h0: the state that it starts from)."""
    i = inputs(len(lengths), L, 2, 2, 40, 48, dtype, seed=seed, h0=True)
    x = i[name]
    x[(0, 0, 3, 5) if name == "h0" else (0, t, 0, 7)[:x.dim()]] = value
    return i


# (length, token): the end of the sequence inside the last chunk, inside the first, in the token-by-token form
ENDS = [(150, 140, 130), (150, 40, 3), (14, 9, 2)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("L,n,t", ENDS)
@pytest.mark.parametrize("name,value", BAD)
def test_fwd_not_finite(gpu, dtype, L, n, t, name, value):
    """A value that is not finite reaches its chunk and head and what follows:
    not the chunks before, not other heads or sequences, and no token past
    the end, whose y is zero."""
    lengths = [n, L]
    i = spoilt(L, lengths, t, name, value, dtype, 340)
    for out in (F32, BF16):
        y, last = ss.delta_fwd(**i, lengths=torch.tensor(lengths, dtype=torch.int32, device=DEV), out_dtype=out)
        torch.cuda.synchronize()
        assert not host(y[0, n:]).any()
        with np.errstate(all="ignore"):
            yr, lr = ref.delta(**i, lengths=lengths)
        half = 2.0 ** -8 if out == BF16 else 0.0
        tol = (5e-5 * float(np.sqrt(np.mean(np.square(yr[1])))), 5e-5 + half)
        before = 0 if name == "h0" else t // 64 * 64
        for part in ((slice(0, 1), slice(0, before), slice(0, 1)), (slice(0, 1), slice(0, n), slice(1, 2)),
                     (slice(1, 2), slice(0, L), slice(0, 2))):
            check_close(host(y[part]).double().numpy(), yr[part], tol, "y that it does not reach")
        # what the definition leaves without a value has none here
        assert not np.isfinite(host(y).double().numpy()[~np.isfinite(yr)]).any()
        assert not np.isfinite(host(last).double().numpy()[~np.isfinite(lr)]).any()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("L,n,t", ENDS)
@pytest.mark.parametrize("name,value", BAD + [("dout", float("nan")), ("dlast", float("-inf"))])
def test_bwd_not_finite(gpu, dtype, L, n, t, name, value):
    """Gradients past the end are zero whatever a live token holds, and those
    of other heads and sequences are what they were."""
    lengths = [n, L]
    dout, dlast = douts(2, L, 2, 40, 48, dtype, 341)
    if name in ("dout", "dlast"):
        i = inputs(2, L, 2, 2, 40, 48, dtype, seed=341, h0=True)
        if name == "dout":
            dout[0, t, 0, 7] = value
        else:
            dlast[0, 0, 3, 5] = value
    else:
        i = spoilt(L, lengths, t, name, value, dtype, 341)
    got = ss.delta_bwd(**i, dout=dout, dlast_state=dlast, lengths=torch.tensor(lengths, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    with np.errstate(all="ignore"):
        want = ref.delta_bwd(**i, dout=dout, dlast=dlast, lengths=lengths)
    for name, x in got.items():
        x, w = host(x).double().numpy(), want[name]
        half = 2.0 ** -8 if got[name].dtype == BF16 else 0.0
        tol = (5e-5 * float(np.sqrt(np.mean(np.square(w[1])))), 5e-5 + half)
        check_close(x[1], w[1], tol, name + " of another sequence")
        if name == "dh0":
            check_close(x[0, 1], w[0, 1], tol, "dh0 of another head")
            continue
        assert not x[0, n:].any(), name
        check_close(x[0, :, 1], w[0, :, 1], tol, name + " of another head")
