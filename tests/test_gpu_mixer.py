"""The Mamba-2 mixer on the GPU: prompts and single tokens against the fp64
oracle.

Bound, in roundings (2^-24) of the oracle's magnitudes (products of the
convolution's terms' absolute values, decayed): 16 for each of x, B, C, a few
for the step and its decay, and what sums over a sequence of L tokens add, at
most 4 a token: 96 + 4 L.  Where y is bf16 its products take two bf16 planes a
side: a side's third plane is at most 2^-16 of it, and so is the product of the
second ones of the sides', 3 x 2^-16 = 768 roundings a term in all.  A decay's exponent is off by roundings of itself,
whose weight falls as fast as it grows.
"""
import pytest
import torch

import selective_state_space_25_amd as ss
from mixer_close import close
from oracle import mixer_ops as ops

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
DEV = "cuda:0"


def rnd(gen, *shape, dtype=F32, scale=1.0):
    return (scale * torch.randn(shape, generator=gen)).to(dtype).to(DEV)


def planes(y):
    return 768 if y.dtype is BF16 else 0


class Inputs:
    def __init__(self, B, L, H, G, P, N, K, dtype, seed=1, states=True, bias=True):
        gen = self.gen = torch.Generator().manual_seed(seed)
        C, self.G, self.N = H * P + 2 * G * N, G, N
        rows = rnd(gen, B, L, 3 + C + H, dtype=dtype)       # one projection's result
        self.xbc, self.dt = rows[..., 3:3 + C], rows[..., 3 + C:]
        self.w, self.b = rnd(gen, C, K, scale=K ** -0.5), rnd(gen, C, scale=0.3) if bias else None
        self.A = -torch.exp(rnd(gen, H))
        self.D = rnd(gen, H) if bias else None
        self.dtb = rnd(gen, H) - 2 if bias else None
        self.h0 = rnd(gen, B, H, P, N, scale=0.3) if states else None
        self.cs = rnd(gen, B, K - 1, C, dtype=dtype) if states else None

    def fwd(self, out=F32, lengths=None, into=None, **kw):
        return ss.mamba2_conv_fwd(self.xbc, self.dt, self.w, self.b, self.A, self.D, self.dtb, ngroups=self.G, dstate=self.N,
                                  lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV),
                                  h0=self.h0, conv_state=self.cs, out=into, out_dtype=out, **kw)

    def ref(self, lengths=None):
        return ops.mixer(self.xbc, self.dt, self.w, self.b, self.A, self.D, self.dtb, self.G, self.N, lengths, self.h0, self.cs)


SHAPES = [  # B, L, H, G, P, N, K
    (1, 1, 2, 1, 64, 128, 4), (2, 15, 4, 2, 16, 16, 4), (1, 64, 2, 1, 64, 64, 4), (2, 65, 3, 1, 48, 128, 3), (1, 130, 4, 4, 80, 32, 2),
    (3, 200, 2, 1, 64, 128, 4), (1, 333, 8, 2, 33, 64, 3), (2, 129, 2, 2, 128, 16, 4), (1, 100, 1, 1, 1, 128, 4)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("ragged", [False, True])
def test_prompt(gpu, shape, dtype, out, ragged):
    B, L = shape[:2]
    i = Inputs(*shape, dtype, states=ragged, bias=shape[3] == 1)
    lengths = ([L, 1, 0] if B > 2 else [L // 2, L + 7] if B > 1 else [L - 1])[:B] if ragged else None
    y, S, cs = i.fwd(out, lengths)
    torch.cuda.synchronize()
    (ry, rS, rcs), (my, mS) = i.ref(lengths)
    close(y, ry, my, 96 + 4 * L + planes(y), "y")
    close(S, rS, mS, 96 + 4 * L, "state")
    assert torch.equal(cs.cpu().double(), rcs)


@pytest.mark.parametrize("shape", [(1, 4, 32, 1, 64, 128, 4), (3, 4, 4, 2, 48, 64, 3), (65, 4, 8, 1, 64, 128, 4), (2, 4, 3, 3, 20, 16, 2),
                                   (1, 4, 2, 1, 1, 32, 4), (9, 4, 16, 1, 100, 128, 4)])
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
def test_tokens_continue_a_prompt(gpu, shape, dtype, out):
    i = Inputs(*shape, dtype, bias=shape[3] != 3)
    (ry, rS, rcs), (my, mS) = i.ref()
    xbc, dt = i.xbc, i.dt
    i.xbc, i.dt = xbc[:, :2], dt[:, :2]
    _, S, cs = i.fwd()
    for t in (2, 3):
        y = ss.mamba2_conv_step(S, cs, xbc[:, t], dt[:, t], i.w, i.b, i.A, i.D, i.dtb, out_dtype=out)
        torch.cuda.synchronize()
        close(y, ry[:, t], my[:, t], 112, f"token {t}")
    close(S, rS, mS, 112, "state")
    assert torch.equal(cs.cpu().double(), rcs)
    S2, cs2 = S.clone(), cs.clone()
    call, y2 = ss.bind_mamba2_conv_step(S2, cs2, xbc[:, 0], dt[:, 0], i.w, i.b, i.A, i.D, i.dtb, out_dtype=out)
    call()
    y = ss.mamba2_conv_step(S, cs, xbc[:, 0], dt[:, 0], i.w, i.b, i.A, i.D, i.dtb, out_dtype=out)
    assert torch.equal(y, y2) and torch.equal(S, S2) and torch.equal(cs, cs2)


def test_prompt_in_two_parts(gpu):
    shape = (2, 150, 2, 1, 64, 128, 4)
    i = Inputs(*shape, BF16)
    (ry, rS, rcs), (my, mS) = i.ref()
    xbc, dt = i.xbc, i.dt
    i.xbc, i.dt = xbc[:, :70], dt[:, :70]
    y0, S, cs = i.fwd()
    i.xbc, i.dt, i.h0, i.cs = xbc[:, 70:], dt[:, 70:], S, cs
    y1, S, cs = i.fwd()
    torch.cuda.synchronize()
    close(torch.cat([y0, y1], 1), ry, my, 96 + 600, "y")
    close(S, rS, mS, 96 + 600, "state")
    assert torch.equal(cs.cpu().double(), rcs)


@pytest.mark.parametrize("L,n", [(40, [13, 0]), (200, [70, 0])])
def test_tokens_past_the_end_are_not_read(gpu, L, n):
    i = Inputs(2, L, 2, 1, 64, 128, 4, BF16)
    i.h0[1, 0, 0, 0] = float("inf")     # a state that is not finite, and no token: y is still zero
    clean = i.fwd(F32, n)
    for b in range(2):
        i.xbc[b, n[b]:] = float("nan")
        i.dt[b, n[b]:] = float("nan")
    again = i.fwd(F32, n)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(clean, again))
    assert not again[0][0, n[0]:].any() and not again[0][1].any() and torch.equal(again[1][1], i.h0[1])


def test_nan_reaches_its_head_and_nothing_before_its_chunk(gpu):
    i = Inputs(1, 300, 3, 1, 64, 128, 4, F32)
    clean = i.fwd()[0]
    i.xbc[0, 200, 70] = float("nan")      # head 1
    y, S, _ = i.fwd()
    torch.cuda.synchronize()
    assert torch.equal(y[:, :192], clean[:, :192]) and torch.equal(y[:, :, [0, 2]], clean[:, :, [0, 2]])
    assert y[0, 200, 1, 6].isnan() and S[0, 1, 6].isnan().all() and S[0, 0].isfinite().all()


def test_extreme_steps(gpu):
    """Decays of nearly one and of zero; steps of zero."""
    i = Inputs(1, 150, 4, 1, 64, 64, 4, F32)
    i.A = torch.tensor([-1e-8, -1e4, -1.0, 0.0], device=DEV)
    i.dt = i.dt.clone()
    i.dt[0, 40:60, 2] = -200.0             # softplus is zero
    i.dt[0, 80:85, 2] = 60.0
    y, S, _ = i.fwd()
    torch.cuda.synchronize()
    (ry, rS, _), (my, mS) = i.ref()
    close(y, ry, my, 96 + 600 + planes(y), "y")
    close(S, rS, mS, 96 + 600, "state")


def test_same_bits_every_time_and_on_another_stream(gpu):
    i = Inputs(2, 400, 4, 2, 64, 128, 4, BF16)
    a = i.fwd()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = i.fwd()
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("L", [10, 300])
def test_graph_replays(gpu, L):
    i = Inputs(2, L, 4, 1, 64, 128, 4, BF16)
    S, cs = i.h0.clone(), i.cs.clone()
    token = i.xbc[:, 0].clone(), i.dt[:, 0].clone()
    step = lambda s, c: ss.mamba2_conv_step(s, c, *token, i.w, i.b, i.A, i.D, i.dtb)
    i.fwd(), step(S.clone(), cs.clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = i.fwd()
        yt = step(S, cs)
    S2, cs2 = S.clone(), cs.clone()
    for _ in range(3):
        i.xbc.copy_(rnd(i.gen, *i.xbc.shape, dtype=BF16))
        token[0].copy_(i.xbc[:, 1])
        graph.replay()
        want, yw = i.fwd(), step(S2, cs2)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        assert torch.equal(yt, yw) and torch.equal(S, S2) and torch.equal(cs, cs2)


def test_workspace_of_the_caller(gpu):
    i = Inputs(1, 200, 2, 1, 64, 128, 4, BF16)
    need = ss.mamba2_conv_workspace_bytes(1, 200, 2, 64, 1, 128)
    want = i.fwd()
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device=DEV)
    got = i.fwd(workspace=ws[:need])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and (ws[need:] == 255).all()
    if need:
        with pytest.raises(ss.SelscanError):
            i.fwd(workspace=ws[:need - 256])
    with pytest.raises(ValueError):
        i.fwd(workspace=torch.empty(need, dtype=torch.uint8))


def test_refusals(gpu):
    i = Inputs(1, 8, 2, 1, 64, 128, 4, BF16)
    with pytest.raises(ValueError, match="channels"):
        ss.mamba2_conv_fwd(i.xbc, i.dt, i.w, i.b, i.A, ngroups=1, dstate=200)
    with pytest.raises(TypeError):
        ss.mamba2_conv_fwd(i.xbc, i.dt.float(), i.w, i.b, i.A, ngroups=1, dstate=128)
    with pytest.raises(ValueError, match="channels"):
        ss.mamba2_conv_step(i.h0[:, :, :1], i.cs, i.xbc[:, 0], i.dt[:, 0], i.w, i.b, i.A[:1])
    with pytest.raises(ss.SelscanError, match="alias"):
        i.fwd(last_state=i.h0)


@pytest.mark.parametrize("P", [64, 33])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strong_decays_beside_weak_ones(gpu, P, dtype):
    """Heads whose decays within 32 tokens span more than fp32's powers of two,
    heads on the border of it and others, in one workgroup, over segments."""
    i = Inputs(2, 400, 8, 1, P, 128, 4, dtype)
    i.A = torch.tensor([-0.01, -1e5, -30.0, -25.0, -20.0, -500.0, -1.0, -60.0], device=DEV)
    i.dtb = torch.full((8,), -2.0, device=DEV)
    i.dt = (0.1 * i.dt).to(dtype)
    (ry, rS, rcs), (my, mS) = i.ref()
    y, S, cs = i.fwd()
    torch.cuda.synchronize()
    close(y, ry, my, 96 + 1600 + planes(y), "y")
    close(S, rS, mS, 96 + 1600, "state")


@pytest.mark.parametrize("L", [60, 300])
def test_growing_states(gpu, L):
    """A positive A: the state grows by up to e^0.25 a token."""
    i = Inputs(1, L, 4, 1, 64, 64, 4, F32)
    i.A = torch.tensor([0.5, 1.0, 2.0, -1.0], device=DEV)
    i.dtb = torch.full((4,), -2.0, device=DEV)
    i.dt = 0.1 * i.dt
    (ry, rS, _), (my, mS) = i.ref()
    y, S, _ = i.fwd()
    torch.cuda.synchronize()
    close(y, ry, my, 96 + 4 * L + planes(y), "y")
    close(S, rS, mS, 96 + 4 * L, "state")


def test_many_groups_and_heads(gpu):
    """A group to each head, more units than a workgroup's waves, and unaligned states."""
    for shape in [(1, 140, 6, 6, 48, 32, 3), (1, 140, 20, 2, 64, 16, 4), (2, 140, 9, 1, 80, 64, 2)]:
        i = Inputs(*shape, BF16)
        room = torch.empty(i.h0.numel() + 1, device=DEV)
        h0 = room[1:].view(i.h0.shape)          # 4 bytes off a 16-byte boundary
        h0.copy_(i.h0)
        i.h0 = h0
        (ry, rS, rcs), (my, mS) = i.ref()
        y, S, cs = i.fwd(BF16)
        torch.cuda.synchronize()
        close(y, ry, my, 96 + 560 + planes(y), "y")
        close(S, rS, mS, 96 + 560, "state")
        assert torch.equal(cs.cpu().double(), rcs)


def test_two_streams_at_once(gpu):
    """Two prompts on two streams, each with workspaces of its own."""
    a, b = Inputs(1, 500, 4, 1, 64, 128, 4, BF16, seed=1), Inputs(1, 500, 4, 1, 64, 128, 4, BF16, seed=2)
    want = a.fwd(), b.fwd()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        with torch.cuda.stream(sa):
            x = a.fwd()
        with torch.cuda.stream(sb):
            y = b.fwd()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(x, want[0])) and all(torch.equal(p, q) for p, q in zip(y, want[1]))


def test_rows_too_far_apart_for_a_chunk(gpu):
    """Rows of xbc 2^23 elements apart: walked token by token."""
    i = Inputs(1, 70, 1, 1, 16, 16, 2, BF16)
    C = i.xbc.shape[2]
    big = torch.empty(70 << 23, dtype=BF16, device=DEV)
    far = big.as_strided((1, 70, C), (0, 1 << 23, 1))
    far.copy_(i.xbc)
    i.xbc = far
    (ry, rS, rcs), (my, mS) = i.ref()
    y, S, cs = i.fwd()
    torch.cuda.synchronize()
    close(y, ry, my, 96 + 280 + planes(y), "y")
    close(S, rS, mS, 96 + 280, "state")


@pytest.mark.parametrize("L", [20, 130])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_that_overlap(gpu, L, dtype):
    """One row for every token (an expanded tensor), and rows one element
    apart: what lies before the first token is still zero, not the buffer's."""
    i = Inputs(2, L, 4, 1, 64, 64, 4, dtype)
    i.cs = None
    C, room = i.xbc.shape[2], i.xbc.reshape(-1)
    for xbc in (room[:C].expand(2, L, C), room.as_strided((2, L, C), (7, 1, 1))):
        i.xbc = xbc
        (ry, rS, rcs), (my, mS) = i.ref()
        y, S, cs = i.fwd()
        torch.cuda.synchronize()
        close(y, ry, my, 96 + 4 * L + planes(y), "y")
        close(S, rS, mS, 96 + 4 * L, "state")
        assert torch.equal(cs.cpu().double(), rcs)


@pytest.mark.parametrize("lengths", [[0, 700, 1, 130, 64, 699, 65, 0, 128], [700] * 9, [0] * 9, [1, 0, 0, 0, 0, 0, 0, 0, 700]])
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (F32, F32)])
def test_segments_of_ragged_prompts(gpu, lengths, dtype, out):
    """Sequences cut into segments by their lengths, empty ones between."""
    i = Inputs(9, 700, 12, 6, 24, 32, 4, dtype)
    (ry, rS, rcs), (my, mS) = i.ref(lengths)
    room = torch.full((9, 700, 12, 24), float("nan"), dtype=out, device=DEV)
    y, S, cs = i.fwd(out, lengths, room)
    torch.cuda.synchronize()
    close(y, ry, my, 96 + 2800 + planes(y), "y")
    close(S, rS, mS, 96 + 2800, "state")
    assert torch.equal(cs.cpu().double(), rcs)
    for b, n in enumerate(lengths):
        assert not y[b, n:].any()


@pytest.mark.parametrize("batch", [64, 65, 70])
@pytest.mark.parametrize("odd", [False, True])
def test_many_ragged_prompts(gpu, batch, odd):
    """As many sequences as lanes, and more; y's rows off 16 bytes."""
    i = Inputs(batch, 200, 4, 4, 15 if odd else 16, 16, 3, BF16)
    lengths = [(37 * b) % 203 for b in range(batch)]
    (ry, rS, rcs), (my, mS) = i.ref(lengths)
    y, S, cs = i.fwd(BF16, lengths, torch.full((batch, 200, 4, 15 if odd else 16), float("nan"), dtype=BF16, device=DEV))
    torch.cuda.synchronize()
    close(y, ry, my, 96 + 800 + planes(y), "y")
    close(S, rS, mS, 96 + 800, "state")
    assert torch.equal(cs.cpu().double(), rcs)


def test_graph_of_changing_lengths(gpu):
    """A captured padded batch follows the lengths that stand on the device at
    each replay; eager calls between the replays share no workspace with it."""
    i = Inputs(9, 700, 12, 6, 24, 32, 4, BF16)
    lengths = torch.tensor([700] * 9, dtype=torch.int32, device=DEV)
    call = lambda n: ss.mamba2_conv_fwd(i.xbc, i.dt, i.w, i.b, i.A, i.D, i.dtb, ngroups=6, dstate=32, lengths=n, h0=i.h0,
                                        conv_state=i.cs)
    call(lengths)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call(lengths)
    for new in ([0] * 9, [700, 3, 0, 64, 65, 128, 699, 1, 400], [700] * 9, [5] * 9):
        lengths.copy_(torch.tensor(new, dtype=torch.int32))
        graph.replay()
        want = call(torch.tensor(new, dtype=torch.int32, device=DEV))
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(held, want)), new
