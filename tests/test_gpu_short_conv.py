"""Short convolution on the GPU: forward, gradients and one token against the
fp64 oracle.

Bounds, in roundings (2^-24) of the oracle's magnitudes.  Forward: K products
and sums, the activation (exp2 of a rounded product and a reciprocal, 2 ulp
each; its relative error grows with |pre|, where its weight falls as fast): 16.
dx: g's slope from a pre that is off by K + 1 roundings of its terms, then K
sums: 32.  dweight, dbias: the same, and 64 + 32 additions in fp32 of a
workgroup's tokens: 128.
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


def inputs(B, L, D, K, dtype, seed=1, pad=0, bias=True):
    """x as columns pad .. of wider rows."""
    gen = torch.Generator().manual_seed(seed)
    x = rnd(gen, B, L, D + 2 * pad, dtype=dtype)[..., pad:pad + D]
    return gen, x, rnd(gen, D, K, scale=K ** -0.5), rnd(gen, D, scale=0.5) if bias else None


CASES = [  # B, L, D, K, pad, split
    (1, 1, 8, 4, 0, None), (2, 5, 64, 4, 0, None), (3, 33, 40, 3, 5, None), (1, 300, 24, 2, 1, [8, 8, 8]),
    (2, 70, 203, 4, 3, [101, 51, 51]), (2, 17, 1, 3, 0, None), (1, 9, 520, 4, 8, [512, 8]), (4, 64, 288, 4, 0, [256, 16, 16]),
    (2, 1100, 16, 4, 2, None), (5, 3, 12, 4, 0, [4, 8])]


@pytest.mark.parametrize("B,L,D,K,pad,split", CASES)
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("ragged", [False, True])
def test_forward(gpu, B, L, D, K, pad, split, dtype, out, ragged):
    gen, x, w, b = inputs(B, L, D, K, dtype, pad=pad, bias=L % 2 == 1)
    state = rnd(gen, B, K - 1, D, dtype=dtype) if ragged else None
    lengths = torch.tensor(([L, 1, 0, L // 2, L + 5] * B)[:B], dtype=torch.int32) if ragged else None
    silu = D % 3 != 1
    y, last = ss.short_conv_fwd(x, w, b, silu, split, None if lengths is None else lengths.to(DEV), state, out_dtype=out)
    torch.cuda.synchronize()
    ref, rlast, mag = ops.conv(x, w, b, silu, lengths, state)
    got = y if split is None else torch.cat(y, -1)
    assert got.dtype is out and (split is None or [p.shape[-1] for p in y] == split)
    close(got, ref, mag, 16, "y")
    assert torch.equal(last.cpu().double(), rlast)
    if ragged:
        for i, n in enumerate(lengths.tolist()):
            assert not got[i, n:].any()


@pytest.mark.parametrize("B,L,D,K,pad,split", CASES)
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("ragged", [False, True])
def test_gradients(gpu, B, L, D, K, pad, split, dtype, out, ragged):
    gen, x, w, b = inputs(B, L, D, K, dtype, pad=pad, bias=L % 2 == 1)
    state = rnd(gen, B, K - 1, D, dtype=dtype) if ragged else None
    dlast = rnd(gen, B, K - 1, D, dtype=dtype) if ragged else None
    lengths = torch.tensor(([L, 1, 0, L // 2, L + 5] * B)[:B], dtype=torch.int32) if ragged else None
    silu = D % 3 != 1
    dout = [rnd(gen, B, L, n, dtype=out) for n in (split or [D])]
    g = ss.short_conv_bwd(x, w, b, dout if split else dout[0], silu, None if lengths is None else lengths.to(DEV), state, dlast,
                          want_dstate=True)
    torch.cuda.synchronize()
    ref, mag = ops.conv_bwd(x, w, b, torch.cat(dout, -1), silu, lengths, state, dlast)
    assert ("dbias" in g) == (b is not None) and g["dx"].dtype is dtype and g["dstate"].dtype is dtype
    for k in g:
        close(g[k], ref[k], mag[k], 128 if k in ("dweight", "dbias") else 32, k)


@pytest.mark.parametrize("B,D,K,pad", [(1, 8, 4, 0), (3, 203, 3, 2), (65, 40, 2, 7), (2, 1, 4, 0), (7, 2304, 4, 32)])
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
def test_steps_continue_a_prompt(gpu, B, D, K, pad, dtype, out):
    gen, x, w, b = inputs(B, 7, D, K, dtype, pad=pad)
    y, state = ss.short_conv_fwd(x[:, :4], w, b)
    for t in range(4, 7):
        got = ss.short_conv_step(state, x[:, t], w, b, out_dtype=out)
        ref, last, mag = ops.conv(x[:, :t + 1], w, b)
        torch.cuda.synchronize()
        close(got, ref[:, t], mag[:, t], 16, f"token {t}")
        assert torch.equal(state.cpu().double(), last)
    call, bound = ss.bind_short_conv_step(state.clone(), x[:, 6], w, b, out_dtype=out)
    call()
    assert torch.equal(bound, ss.short_conv_step(state, x[:, 6], w, b, out_dtype=out))


def test_gradients_are_differences(gpu):
    """A directional difference of the kernels' own forward, without the
    activation in one term only: linear in x, so exact but for roundings; with
    it, off by h^2 times a third derivative."""
    gen, x, w, b = inputs(2, 40, 24, 4, F32)
    dy, d = rnd(gen, 2, 40, 24), rnd(gen, 2, 40, 24)
    for silu in (False, True):
        g = ss.short_conv_bwd(x, w, b, dy, silu)["dx"]
        want = (g.double() * d.double()).sum().item()
        h = 2.0 ** -7
        up, down = (ss.short_conv_fwd(x + s * h * d, w, b, silu)[0].double() for s in (1, -1))
        got = ((up - down) * dy.double()).sum().item() / (2 * h)
        # roundings: x + h d and the forward's, 2^-24 of the terms each, over h
        mag = ops.conv(x, w, b, False)[2].to(DEV)
        size = (dy.double().abs() * mag).sum().item()
        # third derivative of silu: below 0.6; d's part of pre to the third
        pd = ops.conv(d, w, None, False)[0].to(DEV).abs()
        third = 0.6 / 6 * h * h * (dy.double().abs() * pd ** 3).sum().item() if silu else 0.0
        assert abs(got - want) <= 32 * 2.0 ** -24 * size / h + third


def test_tokens_past_the_end_are_not_read(gpu):
    gen, x, w, b = inputs(2, 50, 16, 4, BF16)
    n = [20, 0]
    lengths = torch.tensor(n, dtype=torch.int32, device=DEV)
    dy = rnd(gen, 2, 50, 16)
    clean = ss.short_conv_fwd(x, w, b, lengths=lengths), ss.short_conv_bwd(x, w, b, dy, lengths=lengths)
    for i in range(2):
        x[i, n[i]:] = float("nan")
        dy[i, n[i]:] = float("inf")
    again = ss.short_conv_fwd(x, w, b, lengths=lengths), ss.short_conv_bwd(x, w, b, dy, lengths=lengths)
    assert torch.equal(clean[0][0], again[0][0]) and torch.equal(clean[0][1], again[0][1])
    assert all(torch.equal(clean[1][k], again[1][k]) for k in clean[1])


def test_nan_and_infinity_stay_in_their_window(gpu):
    gen, x, w, b = inputs(1, 60, 16, 4, F32)
    clean, _ = ss.short_conv_fwd(x, w, b)
    x[0, 30, 3], x[0, 40, 5] = float("nan"), float("inf")
    y, _ = ss.short_conv_fwd(x, w, b)
    same = torch.ones(60, 16, dtype=torch.bool, device=DEV)
    same[30:34, 3] = same[40:44, 5] = False
    assert torch.equal(y[0][same], clean[0][same])
    assert y[0, 30:34, 3].isnan().all() and not y[0, 40:44, 5].isfinite().all()


def test_strided_batch_and_repeated_rows(gpu):
    gen = torch.Generator().manual_seed(3)
    x = rnd(gen, 40, 3, 16).transpose(0, 1)             # batch inside the tokens
    row = rnd(gen, 1, 1, 16).expand(2, 30, 16)          # the same row again and again
    w = rnd(gen, 16, 4)
    for t in (x, row):
        y, last = ss.short_conv_fwd(t, w)
        want, wlast = ss.short_conv_fwd(t.contiguous(), w)
        assert torch.equal(y, want) and torch.equal(last, wlast)
    with pytest.raises(ValueError, match="contiguous"):
        ss.short_conv_fwd(rnd(gen, 2, 8, 16).transpose(1, 2), rnd(gen, 8, 4))
    with pytest.raises(ValueError, match="split"):
        ss.short_conv_fwd(x, w, split=[8, 9])
    with pytest.raises(ss.SelscanError):
        ss.short_conv_fwd(x, rnd(gen, 16, 5))


def test_offsets_past_32_bits(gpu):
    """Rows that lie 2^32 elements apart in one allocation."""
    big = torch.empty(5 * (1 << 31), dtype=BF16, device=DEV)   # 20 GB
    gen = torch.Generator().manual_seed(4)
    small = rnd(gen, 1, 3, 16, dtype=BF16)
    x = big.as_strided((1, 3, 16), (0, 1 << 32, 1))
    x.copy_(small)
    w = rnd(gen, 16, 4)
    dy = rnd(gen, 1, 3, 16)
    assert torch.equal(ss.short_conv_fwd(x, w)[0], ss.short_conv_fwd(small, w)[0])
    assert torch.equal(ss.short_conv_bwd(x, w, None, dy)["dweight"], ss.short_conv_bwd(small, w, None, dy)["dweight"])


def test_long_sums_of_weight_gradients(gpu):
    """More workgroups than one pass of the column sums takes (1024), terms of one sign."""
    B, L, D = 4, 1 << 17, 8
    x = torch.ones(B, L, D, device=DEV)
    dy = torch.full((B, L, D), 1.0 / 3.0, device=DEV)
    g = ss.short_conv_bwd(x, torch.zeros(D, 4, device=DEV), None, dy, silu=False)
    third = torch.tensor(1.0 / 3.0).double()
    want = third * torch.tensor([B * (L - 3), B * (L - 2), B * (L - 1), B * L]).double()
    # a workgroup's 256 and less in fp32 (96 additions in a row at most), the rest in fp64
    assert ((g["dweight"].cpu().double() - want).abs() <= 97 * 2.0 ** -24 * want).all()


def test_graph_replays(gpu):
    gen, x, w, b = inputs(2, 130, 48, 4, BF16)
    dy = rnd(gen, 2, 130, 48)
    ss.short_conv_bwd(x, w, b, dy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, last = ss.short_conv_fwd(x, w, b)
        g = ss.short_conv_bwd(x, w, b, dy)
    for i in range(3):
        x.copy_(rnd(gen, 2, 130, 48, dtype=BF16))
        graph.replay()
        want, wlast = ss.short_conv_fwd(x, w, b)
        wg = ss.short_conv_bwd(x, w, b, dy)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(last, wlast) and all(torch.equal(g[k], wg[k]) for k in g)
