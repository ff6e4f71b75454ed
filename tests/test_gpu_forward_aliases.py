"""Convolution and mixer over sequences, outputs beside and between their
inputs' rows in one buffer: taken, and the same bits as elsewhere; over them:
refused."""
import pytest
import torch

import selective_state_space_25_amd as ss

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
DEV = "cuda:0"


def r(gen, *shape):
    return torch.randn(shape, generator=gen).to(DEV)


@pytest.mark.parametrize("token_first", [False, True])
def test_conv_between_rows(gpu, token_first):
    """x: 2 x 5 rows of 12 in a buffer of wider ones, batch elements or tokens first; y stands between two of its rows."""
    gen = torch.Generator().manual_seed(1)
    x, w, state = r(gen, 2, 5, 12), r(gen, 12, 4), r(gen, 2, 3, 12)
    y, last = ss.short_conv_fwd(x, w, state=state)
    room = torch.zeros(10, 200, device=DEV)
    x2 = room.view(5, 2, 200)[..., 10:22].transpose(0, 1) if token_first else room.view(2, 5, 200)[..., 10:22]
    x2.copy_(x)
    out = room.view(-1)[3 * 200 + 30:3 * 200 + 150].view(2, 5, 12)
    y2, last2 = ss.short_conv_fwd(x2, w, state=state, out=out)
    torch.cuda.synchronize()
    assert torch.equal(y2, y) and torch.equal(last2, last) and torch.equal(x2, x)
    dout = r(gen, 2, 5, 12)
    g, g2 = ss.short_conv_bwd(x, w, None, dout, state=state), ss.short_conv_bwd(x2, w, None, dout, state=state)
    torch.cuda.synchronize()
    assert all(torch.equal(g[k], g2[k]) for k in g)
    with pytest.raises(ss.SelscanError, match="alias"):
        ss.short_conv_fwd(x2, w, state=state, out=room.view(-1)[3 * 200 + 100:3 * 200 + 220].view(2, 5, 12))


@pytest.mark.parametrize("L", [1, 5, 100])
def test_mixer(gpu, L):
    gen = torch.Generator().manual_seed(L)
    w, b, A = r(gen, 96, 4), r(gen, 96), -torch.rand(4, generator=gen).to(DEV)
    proj = r(gen, 1, L, 32 + 96 + 4)                       # z, xbc, dt
    xbc, dt = proj[..., 32:128], proj[..., 128:]
    call = lambda **kw: ss.mamba2_conv_fwd(xbc, dt, w, b, A, ngroups=2, dstate=16, **kw)
    want = call()
    if L == 1:      # y over z of the one row: beside xbc
        got = call(out=proj[..., :32].view(1, 1, 4, 8))
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        for at in (1, 33, 96, 100):
            with pytest.raises(ss.SelscanError, match="alias"):
                call(out=proj[0, 0, at:at + 32].view(1, 1, 4, 8))
    else:           # one buffer for all that is written
        room = torch.empty(L * 32 + 4 * 8 * 16 + 3 * 96, device=DEV)
        y, S, cs = room[:L * 32].view(1, L, 4, 8), room[L * 32:L * 32 + 512].view(1, 4, 8, 16), room[L * 32 + 512:].view(1, 3, 96)
        got = call(out=y, last_state=S, last_conv_state=cs)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        with pytest.raises(ss.SelscanError, match="alias"):
            call(out=y, last_state=room[L * 32 - 4:L * 32 + 508].view(1, 4, 8, 16))
