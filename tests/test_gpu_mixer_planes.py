"""The mixer's products keep fp32's precision whatever y's type is: prompts with
a bf16 y under the bounds that an fp32 y has, and sums whose terms cancel.

Cancelling sums: terms come in pairs +c v1, -c v2 that nearly cancel, where v1
and v2 leave remainders of opposite sign when only their first 16 bits are
taken, so what is lost adds up over all pairs: 2^-17 of the terms' size (128
roundings of 2^-24; 0.75 of it for x), where three planes of 8 bits lose 2^-25.
Both terms of a pair have the same c, so c's own roundings act on the small
result alone.  Bound: one rounding for each addition of the n terms to a partial
sum of at most half their size, n / 2, and 8 for the planes' smaller products.
"""
import pytest
import torch

import selective_state_space_25_amd as ss
from mixer_close import close
from test_gpu_mixer import SHAPES, Inputs

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
F64 = torch.float64
DEV = "cuda:0"


def silu(x):
    return x * torch.sigmoid(x)


def silu_inverse(y):
    """The root beyond the minimum at -1.278, by bisection."""
    lo, hi = torch.full_like(y, -1.2784645), torch.full_like(y, 4.0)
    for _ in range(80):
        mid = (lo + hi) / 2
        low = silu(mid) < y
        lo, hi = torch.where(low, mid, lo), torch.where(low, hi, mid)
    return (lo + hi) / 2


def run(x, b, c, dt, A, h0, dtype, out):
    """x [1, L, H P], b, c [1, L, N]: inputs in front of the activation (taps 0, 1)."""
    L, H, N = x.shape[1], dt.shape[2], b.shape[2]
    xbc = torch.cat([x, b, c], -1).to(dtype)
    w = torch.zeros(xbc.shape[2], 2)
    w[:, 1] = 1.0
    y, _, _ = ss.mamba2_conv_fwd(xbc.to(DEV), dt.to(dtype).to(DEV), w.to(DEV), None, A.to(DEV), ngroups=1, dstate=N,
                                 h0=None if h0 is None else h0.to(DEV), out_dtype=out)
    torch.cuda.synchronize()
    return y, [silu(t.double()) for t in xbc.split([x.shape[2], N, N], -1)]


@pytest.mark.parametrize("N", [16, 64, 128])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("out", [BF16, F32])
def test_states_that_cancel(gpu, N, dtype, out):
    """y = S C from a state alone: steps of zero leave it as it is."""
    gen = torch.Generator().manual_seed(N)
    H, P, L = 8, 32, 70
    v = 1 + 2.0 ** -9 + 2.0 ** -10 + 2.0 ** -17
    h0 = torch.empty(1, H, P, N)
    h0[..., 0::2], h0[..., 1::2] = v - 2.0 ** -20, -(v + 2.0 ** -20)
    h0 *= torch.exp2(torch.randint(-2, 3, (1, H, P, N // 2), generator=gen).float()).repeat_interleave(2, -1)
    c = (1 + 3 * torch.rand(1, L, N // 2, generator=gen)).repeat_interleave(2, -1)
    x, b = torch.randn(1, L, H * P, generator=gen), torch.randn(1, L, N, generator=gen)
    y, (_, _, c64) = run(x, b, c, torch.full((1, L, H), -200.0), torch.full((H,), -1.0), h0, dtype, out)
    terms = c64[:, :, None, None] * h0[:, None].double()
    close(y, terms.sum(-1), terms.abs().sum(-1), N / 2 + 8, "y")


@pytest.mark.parametrize("N", [16, 64, 128])
@pytest.mark.parametrize("out", [BF16, F32])
def test_tokens_that_cancel(gpu, N, out):
    """y = G X inside a chunk, without decay: B is every token's, x comes in pairs (its roundings: 16)."""
    gen = torch.Generator().manual_seed(N)
    H, P, L = 8, 32, 64
    v = 1 + 2.0 ** -9 + 2.0 ** -10 + 2.0 ** -17
    x = torch.empty(1, L, H * P, dtype=F64)
    x[:, 0::2], x[:, 1::2] = 0.25 * (v - 2.0 ** -19), -0.25 * (v + 2.0 ** -19)
    b = (1 + 3 * torch.rand(1, 1, N, generator=gen)).expand(1, L, N)
    c = 1 + 3 * torch.rand(1, L, N, generator=gen)
    y, (x64, b64, c64) = run(silu_inverse(x).float(), b, c, torch.full((1, L, H), 32.0), torch.zeros(H), None, F32, out)
    step = 32.0 + torch.log1p(torch.exp(torch.tensor(-32.0, dtype=F64)))
    g = step * torch.tril(c64[0] @ b64[0].t())
    ref, size = ((m @ t[0]).reshape(1, L, H, P) for m, t in ((g, x64), (g, x64.abs())))
    close(y, ref, size, 16 + L / 2 + 8, "y")


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_bf16_y_has_the_bounds_of_an_fp32_y(gpu, shape, dtype):
    i = Inputs(*shape, dtype, states=True, bias=shape[3] == 1)
    y, _, _ = i.fwd(BF16)
    torch.cuda.synchronize()
    (ry, _, _), (my, _) = i.ref()
    close(y, ry, my, 96 + 4 * shape[1], "y")


def test_a_bf16_y_is_the_fp32_y_rounded(gpu):
    """One and the same computation, whatever the type that y is written in."""
    for shape in [(1, 333, 8, 1, 64, 128, 4), (2, 129, 6, 2, 33, 64, 3), (1, 20, 2, 1, 64, 128, 4)]:
        for dtype in (BF16, F32):
            i = Inputs(*shape, dtype)
            assert torch.equal(i.fwd(BF16)[0], i.fwd(F32)[0].to(BF16))
