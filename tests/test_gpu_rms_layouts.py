"""RMS norm at the widths where a group goes over from one wave to the four of a
workgroup: 1024, 1280 or 1536 elements by the bytes that an element moves, 2560
for the gradients.  Bounds as for other widths: 48 and 128 roundings."""
import ctypes

import pytest
import torch

import selective_state_space_25_amd as ss
from mixer_close import close
from oracle import mixer_ops as ops

pytestmark = pytest.mark.gpu

F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
DEV = "cuda:0"
WIDTHS = [1017, 1024, 1025, 1273, 1280, 1281, 1529, 1536, 1537, 1545]


def rnd(gen, *shape, dtype=F32):
    return torch.randn(shape, generator=gen).to(dtype).to(DEV)


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("kind,dtype,other,out", [
    ("", BF16, None, BF16), ("", F32, None, BF16), ("", F32, None, F32), ("", BF16, None, F32), ("res", BF16, BF16, BF16),
    ("res", BF16, F32, BF16), ("gate", BF16, BF16, BF16), ("gate", BF16, BF16, F32), ("gate", F32, F32, F32),
    ("gate", BF16, BF16, E4M3), ("", F32, None, E4M3)])
def test_forward(gpu, width, kind, dtype, other, out):
    gen = torch.Generator().manual_seed(width)
    x, w, o = rnd(gen, 5, width, dtype=dtype), 1 + 0.1 * rnd(gen, width), rnd(gen, 5, width, dtype=other or F32)
    res, gate = o if kind == "res" else None, o if kind == "gate" else None
    y, s, rstd, scale = ss.rms_norm_fwd(x, w, res, gate=gate, out_dtype=out, scale_block=128 if out is E4M3 else 0)
    torch.cuda.synchronize()
    ry, rs, rr, mag = ops.rms(x, w, res, gate)
    close(rstd, rr, rr, 48, "rstd")
    if out is E4M3:
        by = scale.cpu().double().repeat_interleave(128, 1)[:, :width]
        bound = torch.maximum(2.0 ** -4 * ry.abs(), 2.0 ** -10 * by) + 56 * 2.0 ** -24 * mag
        assert ((y.cpu().double() * by - ry).abs() <= bound).all()
    else:
        close(y, ry, mag, 48, "y")
    if kind == "res":
        close(s, rs, rs.abs(), 1, "s")


@pytest.mark.parametrize("width", [2553, 2560, 2561, 4104])
@pytest.mark.parametrize("gated", [False, True])
def test_gradients(gpu, width, gated):
    gen = torch.Generator().manual_seed(width)
    s, dy, w, z = rnd(gen, 9, width), rnd(gen, 9, width, dtype=BF16), 1 + 0.1 * rnd(gen, width), rnd(gen, 9, width) if gated else None
    rstd = ops.rms(s, None, None, z)[2].float().to(DEV)
    g = ss.rms_norm_bwd(dy, s, w, rstd, gate=z)
    torch.cuda.synchronize()
    ref, mag = ops.rms_bwd(dy, s, w, rstd, z)
    for k in g:
        close(g[k], ref[k], mag[k], 128, k)


@pytest.mark.parametrize("width", [1032, 1200, 1280, 1400, 2560])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_the_same_bits_with_and_without_s(gpu, width, dtype):
    """Whether s is asked for does not change y: over x (s in memory of its own) and without it."""
    gen = torch.Generator().manual_seed(width)
    x, r, w = rnd(gen, 40, width, dtype=dtype), rnd(gen, 40, width, dtype=dtype), rnd(gen, width)
    xx = x.clone()
    y = ss.rms_norm_fwd(x, w)[0]
    assert torch.equal(ss.rms_norm_fwd(xx, w, out=xx)[0], y)
    want, got = ss.rms_norm_fwd(x, w, r)[0], torch.empty_like(x)
    code = ss.F32 if dtype is F32 else ss.BF16
    sh = ss.RmsShape(40, width, 1, 0, 0, code, code, code, 1e-5, None, 0)
    assert ss.lib().selscan_rms_norm_fwd(ctypes.byref(sh), x.data_ptr(), r.data_ptr(), None, w.data_ptr(), got.data_ptr(), None, None,
                                         None, torch.cuda.current_stream().cuda_stream) == ss.OK
    torch.cuda.synchronize()
    assert torch.equal(got, want)
