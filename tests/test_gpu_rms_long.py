"""RMS norm of very long groups: the sums keep their precision at any length.

Terms that are alike are where a running fp32 sum loses most (each addition is
off the same way: 2^22 equal elements over 256 lanes come out by up to 2^-13).
Bounds as for short groups, without a part that grows with the width: 48
roundings for the forward, 128 for the gradients.
"""
import pytest
import torch

import selective_state_space_25_amd as ss
from mixer_close import close
from oracle import mixer_ops as ops

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
DEV = "cuda:0"
VALUES = [0.5123, 0.6123, 0.7123, 1.0123]


@pytest.mark.parametrize("width", [70001, (1 << 22) + 3])
@pytest.mark.parametrize("gated", [False, True])
def test_forward(gpu, width, gated):
    x = torch.tensor(VALUES, device=DEV)[:, None].expand(4, width).contiguous()
    z = torch.full_like(x, 1.5) if gated else None
    y, _, rstd, _ = ss.rms_norm_fwd(x, gate=z)
    torch.cuda.synchronize()
    ry, _, rr, mag = ops.rms(x, None, None, z)
    close(rstd, rr, rr, 48, "rstd")
    close(y, ry, mag, 48, "y")


@pytest.mark.parametrize("width", [70001, (1 << 22) + 3])
@pytest.mark.parametrize("gated", [False, True])
def test_gradients(gpu, width, gated):
    s = torch.tensor(VALUES, device=DEV)[:, None].expand(4, width).contiguous()
    dy = torch.tensor([0.9123, 0.3123, 1.1123, 0.7123], device=DEV)[:, None].expand(4, width).contiguous()
    z = torch.full_like(s, 1.5) if gated else None
    rstd = ops.rms(s, None, None, z)[2].float().to(DEV)
    g = ss.rms_norm_bwd(dy, s, None, rstd, gate=z)
    torch.cuda.synchronize()
    ref, mag = ops.rms_bwd(dy, s, None, rstd, z)
    for k in g:
        close(g[k], ref[k], mag[k], 128, k)
