"""The fp64 oracle of the short convolution, the mixer and RMS norm against
other implementations and against differences (CPU)."""
import math

import pytest
import torch

import oracle
from oracle import mixer_ops as ops

F64 = torch.float64


def rnd(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=F64)


@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("silu", [True, False])
def test_conv_is_a_causal_convolution(K, silu):
    x, w, b, s = rnd(1, 2, 9, 5), rnd(2, 5, K), rnd(3, 5), rnd(4, 2, K - 1, 5)
    y, last, mag = ops.conv(x, w, b, silu, None, s)
    full = torch.cat([s, x], 1).transpose(1, 2)
    ref = torch.nn.functional.conv1d(full, w[:, None], b, groups=5).transpose(1, 2)
    ref = torch.nn.functional.silu(ref) if silu else ref
    assert torch.allclose(y, ref, atol=1e-14, rtol=1e-13)
    assert torch.equal(last, torch.cat([s, x], 1)[:, -(K - 1):])
    assert (mag >= y.abs() - 1e-12).all()


def test_conv_lengths_and_split_sequences():
    x, w, b = rnd(1, 3, 8, 4), rnd(2, 4, 4), rnd(3, 4)
    y, last, _ = ops.conv(x, w, b, True, [8, 1, 0])
    for i, n in enumerate([8, 1, 0]):
        yi, li, _ = ops.conv(x[i:i + 1, :n], w, b) if n else (x[i:i + 1, :0], torch.zeros(1, 3, 4, dtype=F64), None)
        assert torch.equal(y[i:i + 1, :n], yi) and torch.equal(last[i:i + 1], li) and not y[i, n:].any()
    a, mid, _ = ops.conv(x[:, :3], w, b)
    c, end, _ = ops.conv(x[:, 3:], w, b, True, None, mid)
    whole, last, _ = ops.conv(x, w, b)
    assert torch.allclose(torch.cat([a, c], 1), whole, atol=1e-15) and torch.equal(end, last)


def by_differences(f, args, names, grads, rtol=2e-6):
    """Gradients of sum of f against central differences at some elements."""
    h = 1e-5
    for name in names:
        t, g = args[name], grads[name]
        flat = t.reshape(-1)
        for e in torch.randperm(flat.numel(), generator=torch.Generator().manual_seed(7))[:6].tolist():
            was = flat[e].item()
            flat[e] = was + h
            up = f(**args)
            flat[e] = was - h
            down = f(**args)
            flat[e] = was
            d = (up - down) / (2 * h)
            assert abs(d - g.reshape(-1)[e].item()) <= rtol * (1 + abs(d)), (name, e)


@pytest.mark.parametrize("lengths", [None, [6, 1, 0]])
def test_conv_gradients_are_differences(lengths):
    x, w, b, s = rnd(1, 3, 6, 4), rnd(2, 4, 4), rnd(3, 4), rnd(4, 3, 3, 4)
    dy, dl = rnd(5, 3, 6, 4), rnd(6, 3, 3, 4)
    g, _ = ops.conv_bwd(x, w, b, dy, True, lengths, s, dl)

    def loss(x, w, b, s):
        y, last, _ = ops.conv(x, w, b, True, lengths, s)
        return (y * dy).sum().item() + (last * dl).sum().item()

    by_differences(loss, dict(x=x, w=w, b=b, s=s), ["x", "w", "b", "s"],
                   dict(x=g["dx"], w=g["dweight"], b=g["dbias"], s=g["dstate"]))


def test_mixer_is_the_scan_of_the_convolution():
    B, L, H, P, G, N = 2, 11, 4, 3, 2, 16
    C = H * P + 2 * G * N
    xbc, dt, w, b = rnd(1, B, L, C), rnd(2, B, L, H), rnd(3, C, 4) * 0.5, rnd(4, C)
    A, D, dtb, h0 = -torch.exp(rnd(5, H)), rnd(6, H), rnd(7, H), rnd(8, B, H, P, N)
    (y, S, _), (ym, Sm) = ops.mixer(xbc, dt, w, b, A, D, dtb, G, N, None, h0)
    v = ops.conv(xbc, w, b)[0]
    x, bb, cc = v.split([H * P, G * N, G * N], -1)
    f = lambda t: t.float()
    yr, Sr = oracle.m2(f(x).reshape(B, L, H, P), f(dt), f(A), f(bb).reshape(B, L, G, N), f(cc).reshape(B, L, G, N), f(D), None,
                       f(dtb), h0=f(h0))
    assert (y - torch.as_tensor(yr)).abs().max() <= 1e-5 * ym.max()
    assert (S - torch.as_tensor(Sr)).abs().max() <= 1e-5 * Sm.max()


@pytest.mark.parametrize("gate,groups", [(False, 1), (True, 1), (True, 2)])
def test_rms_gradients_are_differences(gate, groups):
    x, w, z, r = rnd(1, 3, 8), rnd(2, 8), rnd(3, 3, 8), rnd(4, 3, 8)
    dy, dr = rnd(5, 3, 8), rnd(6, 3, 8)
    args = dict(x=x, w=w, z=z) if gate else dict(x=x, w=w, r=r)

    def loss(x, w, z=None, r=None):
        y, s, _, _ = ops.rms(x, w, r, z, groups)
        return (y * dy).sum().item() + (0 if gate else (s * dr).sum().item())

    _, s, rstd, _ = ops.rms(x, w, None if gate else r, z if gate else None, groups)
    g, m = ops.rms_bwd(dy, x if gate else s, w, rstd, z if gate else None, groups, None if gate else dr)
    names = dict(x=g["dx"], w=g["dweight"], **({"z": g["dgate"]} if gate else {"r": g["dresidual"]}))
    by_differences(loss, args, list(names), names)
    assert all((m[k] >= g[k].abs() - 1e-12).all() for k in g)


def test_rms_value():
    x = torch.tensor([[3.0, 4.0]], dtype=F64)
    y, _, rstd, _ = ops.rms(x, None, eps=0.0)
    assert math.isclose(rstd.item(), math.sqrt(2) / 5) and torch.allclose(y, x * math.sqrt(2) / 5)
