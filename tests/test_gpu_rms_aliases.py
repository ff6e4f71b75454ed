"""RMS norm written over its inputs, element by element: the same bits."""
import ctypes

import pytest
import torch

import selective_state_space_25_amd as ss

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
DEV = "cuda:0"


@pytest.mark.parametrize("width", [40, 1000, 2557, 8000, 9001])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_in_place(gpu, width, dtype):
    gen = torch.Generator().manual_seed(width)
    r = lambda *s: torch.randn(s, generator=gen).to(DEV, dtype)
    x, res, z, dy = r(7, width), r(7, width), r(7, width), r(7, width)
    y, s, rstd, _ = ss.rms_norm_fwd(x, None, res)
    rr = res.clone()
    assert torch.equal(ss.rms_norm_fwd(x, None, rr, out=rr)[0], y)
    zz = z.clone()
    want = ss.rms_norm_fwd(x, gate=z)
    assert torch.equal(ss.rms_norm_fwd(x, gate=zz, out=zz)[0], want[0])
    g = ss.rms_norm_bwd(dy, x, None, want[2], gate=z)
    code = ss.F32 if dtype is F32 else ss.BF16
    sh = ss.RmsShape(7, width, 1, width, 0, code, code, code, 1e-5, None, 0)
    gx, gz = dy.clone(), z.clone()                        # dx over dy, dgate over gate
    st = ss.lib().selscan_rms_norm_bwd(ctypes.byref(sh), gx.data_ptr(), x.data_ptr(), gz.data_ptr(), None, want[2].data_ptr(), None,
                                       gx.data_ptr(), None, gz.data_ptr(), None, torch.cuda.current_stream().cuda_stream)
    assert st == ss.OK
    torch.cuda.synchronize()
    assert torch.equal(gx, g["dx"]) and torch.equal(gz, g["dgate"])


def test_other_overlaps(gpu):
    x = torch.randn(4, 64, device=DEV)
    keep = x.clone()
    for out in (x.view(-1).view(BF16)[:256].view(4, 64), x.view(-1).view(torch.float8_e4m3fn)[:256].view(4, 64)):
        with pytest.raises(ss.SelscanError, match="alias"):
            ss.rms_norm_fwd(x, out=out)
    room = torch.randn(300, device=DEV)
    with pytest.raises(ss.SelscanError, match="alias"):
        ss.rms_norm_fwd(room[:256].view(4, 64), out=room[4:260].view(4, 64))
    torch.cuda.synchronize()
    assert torch.equal(x, keep)
