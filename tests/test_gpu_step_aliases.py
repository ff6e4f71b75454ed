"""One token of the mixer through torch tensors: y over the inputs is refused
and leaves the states as they were; y beside them in one buffer is not."""
import pytest
import torch

import selective_state_space_25_amd as ss

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
DEV = "cuda:0"


def mixer_inputs(B, dtype):
    gen = torch.Generator().manual_seed(B)
    r = lambda *s: torch.randn(s, generator=gen).to(DEV)
    xbc, dt = r(B, 96).to(dtype), r(B, 4).to(dtype)
    return r(B, 4, 8, 16), r(B, 3, 96).to(dtype), xbc, dt, r(96, 4), r(96), -torch.rand(4, generator=gen).to(DEV)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_mixer_step(gpu, dtype):
    S, cs, xbc, dt, w, b, A = mixer_inputs(1, dtype)
    keep = S.clone(), cs.clone(), xbc.clone()
    for out in (xbc[:, :32].view(1, 4, 8), xbc[:, 60:92].view(1, 4, 8), cs[:, 0, :32].view(1, 4, 8)):
        with pytest.raises(ss.SelscanError, match="alias"):
            ss.mamba2_conv_step(S, cs, xbc, dt, w, b, A, out=out)
        with pytest.raises(ss.SelscanError, match="alias"):
            call, _ = ss.bind_mamba2_conv_step(S, cs, xbc, dt, w, b, A, out=out)
            call()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(keep, (S, cs, xbc)))


def test_mixer_step_beside_its_inputs(gpu):
    """y, states and inputs in one buffer, one after the other and between xbc's rows."""
    S, cs, xbc, dt, w, b, A = mixer_inputs(2, F32)
    want = ss.mamba2_conv_step(S.clone(), cs.clone(), xbc, dt, w, b, A)
    room = torch.zeros(2048 + 576 + 64 + 400, device=DEV)
    S2, cs2, y = room[:1024].view(2, 4, 8, 16), room[1024:1600].view(2, 3, 96), room[1700:1764].view(2, 4, 8)
    x2 = room[1600:1600 + 2 * 200].view(2, 200)[:, :96]      # y lies between its two rows
    for t, v in ((S2, S), (cs2, cs), (x2, xbc)):
        t.copy_(v)
    got = ss.mamba2_conv_step(S2, cs2, x2, dt, w, b, A, out=y)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(x2, xbc)
