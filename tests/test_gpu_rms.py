"""RMS norm on the GPU: forward, 8-bit output, gradients against the fp64 oracle.

Bounds, in roundings (2^-24) of the oracle's magnitudes.  Forward: s one sum
(or a gate: 6), a sum of squares with up to 40 additions in a row and 9 across
lanes, halved by the root, root, division and two products: 48; longer groups
add a row of 8 for each 2048 elements.  Gradients: a sum over the group of the
same length, and the same steps twice: 128; dweight: 64 rows and 32 partial
sums in fp32: 128.
"""
import pytest
import torch

import selective_state_space_25_amd as ss
from mixer_close import close
from oracle import mixer_ops as ops

pytestmark = pytest.mark.gpu

F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
DEV = "cuda:0"


def rnd(gen, *shape, dtype=F32, scale=1.0):
    return (scale * torch.randn(shape, generator=gen)).to(dtype).to(DEV)


WIDTHS = [1, 3, 7, 8, 9, 31, 64, 65, 120, 200, 257, 512, 520, 1000, 1537, 2048, 2560, 2561, 4096, 5119, 8192, 8193, 20001]
TYPES = [(BF16, BF16, BF16), (BF16, F32, BF16), (BF16, F32, F32), (F32, F32, F32), (F32, BF16, BF16)]


def roundings(width):
    return 48 + width // 256


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("dtype,res,out", TYPES)
def test_forward_with_residual(gpu, width, dtype, res, out):
    gen = torch.Generator().manual_seed(width)
    rows = 1 + 40 // (1 + width // 64)
    x, r, w = rnd(gen, rows, width, dtype=dtype), rnd(gen, rows, width, dtype=res, scale=2.0), 1 + rnd(gen, width, scale=0.1)
    y, s, rstd, scale = ss.rms_norm_fwd(x, w, r, out_dtype=out)
    torch.cuda.synchronize()
    ry, rs, rr, mag = ops.rms(x, w, r)
    assert scale is None and s.dtype is res and y.dtype is out and rstd.shape == (rows, 1)
    close(s, rs, rs.abs(), 1, "s")
    close(y, ry, mag, roundings(width), "y")
    close(rstd, rr, rr, roundings(width), "rstd")


@pytest.mark.parametrize("width,groups", [(64, 1), (33, 3), (512, 4), (640, 2), (2560, 1), (1280, 2), (5120, 1), (9000, 2)])
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("pad", [0, 3])
def test_forward_with_gate(gpu, width, groups, dtype, out, pad):
    gen = torch.Generator().manual_seed(width + pad)
    D = width * groups
    x, z, w = rnd(gen, 2, 5, D, dtype=dtype), rnd(gen, 2, 5, D + 2 * pad, dtype=dtype)[..., pad:pad + D], 1 + rnd(gen, D, scale=0.1)
    y, s, rstd, _ = ss.rms_norm_fwd(x, w, gate=z, groups=groups, out_dtype=out)
    torch.cuda.synchronize()
    ry, _, rr, mag = ops.rms(x.reshape(10, D), w, None, z.reshape(10, D), groups)
    assert s is None and rstd.shape == (2, 5, groups)
    close(y.reshape(10, D), ry, mag, roundings(width), "y")
    close(rstd.reshape(10, groups), rr, rr, roundings(width), "rstd")


@pytest.mark.parametrize("width,groups", [(3, 1), (32, 1), (100, 2), (128, 4), (513, 1), (2560, 1), (5120, 1), (8191, 1), (10000, 1)])
@pytest.mark.parametrize("block", [0, 32, 64, 128, 256, 512])
@pytest.mark.parametrize("dtype,gated", [(BF16, True), (F32, False)])
def test_eight_bits(gpu, width, groups, block, dtype, gated):
    gen = torch.Generator().manual_seed(width + block)
    D, rows = width * groups, 9
    x, w = rnd(gen, rows, D, dtype=dtype), 1 + rnd(gen, D, scale=0.1)
    x[4] = 0
    z = rnd(gen, rows, D, dtype=dtype) if gated else None
    y, _, rstd, scale = ss.rms_norm_fwd(x, w, gate=z, groups=groups, out_dtype=E4M3, scale_block=block)
    torch.cuda.synchronize()
    ry, _, _, mag = ops.rms(x, w, None, z, groups)
    per = -(-width // block) if block else 1
    assert y.dtype is E4M3 and scale.shape == (rows, groups * per)
    span = block or width
    index = (torch.arange(width) // span)[None] + per * torch.arange(groups)[:, None]
    index = index.reshape(-1)
    top = torch.zeros(rows, groups * per, dtype=torch.float64).scatter_reduce_(1, index.expand(rows, -1), ry.abs(), "amax")
    want = (top / 448).clamp(min=2.0 ** -126)
    tops = torch.zeros_like(top).scatter_reduce_(1, index.expand(rows, -1), mag, "amax")
    close(scale, want, tops / 448 + want, roundings(width) + 2, "scale")
    by = scale.cpu().double()[:, index]
    values = y.cpu().to(torch.float64) * by
    # half a step (2^-4 of a normal value, 2^-10 of the scale below 2^-6), and the fp32 roundings
    bound = torch.maximum(2.0 ** -4 * ry.abs(), 2.0 ** -10 * by) + (roundings(width) + 4) * 2.0 ** -24 * mag * 1.1
    assert ((values - ry).abs() <= bound).all()
    assert (y.cpu().float().abs() <= 448).all() and not y[4].float().any()
    # the largest of a block is 448 to a rounding of the scale
    got = torch.zeros(rows, groups * per).scatter_reduce_(1, index.expand(rows, -1), y.cpu().float().abs(), "amax")
    assert ((got == 448) | (top < 2.0 ** -100)).all()


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("dtype,res,out", TYPES)
@pytest.mark.parametrize("more", [False, True])
def test_gradients(gpu, width, dtype, res, out, more):
    gen = torch.Generator().manual_seed(width)
    rows = 1 + 90 // (1 + width // 64)
    s, dy, w = rnd(gen, rows, width, dtype=res, scale=2.0), rnd(gen, rows, width, dtype=out), 1 + rnd(gen, width, scale=0.1)
    dr = rnd(gen, rows, width, dtype=res) if more else None
    rstd = ops.rms(s)[2].float().to(DEV)
    g = ss.rms_norm_bwd(dy, s, w if more else None, rstd, dresidual=dr, x_dtype=dtype)
    torch.cuda.synchronize()
    ref, mag = ops.rms_bwd(dy, s, w if more else None, rstd, None, 1, dr)
    assert g["dx"].dtype is dtype and g["dresidual"].dtype is res and "dgate" not in g
    assert (g["dx"] is g["dresidual"]) == (dtype == res)
    for k in g:
        close(g[k], ref[k], mag[k], 128 + width // 256, k)


@pytest.mark.parametrize("width,groups", [(5, 1), (64, 2), (33, 3), (512, 4), (1280, 2), (2560, 1), (4099, 1), (8192, 1), (9000, 2)])
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (BF16, F32), (F32, F32)])
def test_gradients_with_gate(gpu, width, groups, dtype, out):
    gen = torch.Generator().manual_seed(width)
    D, rows = width * groups, 70
    x, z = rnd(gen, rows, D, dtype=dtype), rnd(gen, rows, D + 3, dtype=dtype)[:, 3:]
    dy, w = rnd(gen, rows, D, dtype=out), 1 + rnd(gen, D, scale=0.1)
    rstd = ops.rms(x, None, None, z, groups)[2].float().to(DEV)
    g = ss.rms_norm_bwd(dy, x, w, rstd, gate=z, groups=groups)
    torch.cuda.synchronize()
    ref, mag = ops.rms_bwd(dy, x, w, rstd, z, groups)
    assert sorted(g) == ["dgate", "dweight", "dx"]
    for k in g:
        close(g[k], ref[k], mag[k], 128 + width // 256, k)


def test_gradients_are_differences(gpu):
    """Directional differences of the kernels' own forward: off by its
    roundings over h, and by h^2 / 6 of a third derivative, which for unit
    rows and directions stays under 30."""
    gen = torch.Generator().manual_seed(2)
    x, z, w, dy = (rnd(gen, 6, 96), rnd(gen, 6, 96), 1 + rnd(gen, 96, scale=0.1), rnd(gen, 6, 96))
    _, _, rstd, _ = ss.rms_norm_fwd(x, w, gate=z)
    g = ss.rms_norm_bwd(dy, x, w, rstd, gate=z)
    h = 2.0 ** -8
    args = {"x": x, "z": z, "w": w}
    for name, key in (("x", "dx"), ("z", "dgate"), ("w", "dweight")):
        d = rnd(gen, *args[name].shape)
        d = d / d.double().square().mean().sqrt().float()
        want = (g[key].double() * d.double()).sum().item()
        f = lambda s: ss.rms_norm_fwd(*[(args[n] + s * h * d if n == name else args[n]) for n in ("x", "w")],
                                      gate=args["z"] + s * h * d if name == "z" else args["z"])[0].double()
        got = ((f(1) - f(-1)) * dy.double()).sum().item() / (2 * h)
        mag = ops.rms(x, w, None, z)[3].to(DEV)
        size = (dy.double().abs() * (mag + 1)).sum().item()
        assert abs(got - want) <= 64 * 2.0 ** -24 * size / h + 30 * h * h / 6 * dy.double().abs().sum().item()


def test_written_over_its_inputs(gpu):
    """y over x, s over residual through the C ABI, dresidual over its input: a row is read before it is written."""
    import ctypes
    gen = torch.Generator().manual_seed(6)
    for width in (100, 2557, 8000, 9001):
        x, r = rnd(gen, 7, width), rnd(gen, 7, width)
        want = ss.rms_norm_fwd(x, None, r)
        xx, rr = x.clone(), r.clone()
        sh = ss.RmsShape(7, width, 1, 0, 0, ss.F32, ss.F32, ss.F32, 1e-5, None, 0)
        st = ss.lib().selscan_rms_norm_fwd(ctypes.byref(sh), xx.data_ptr(), rr.data_ptr(), None, None, xx.data_ptr(), rr.data_ptr(),
                                           None, None, torch.cuda.current_stream().cuda_stream)
        assert st == ss.OK
        torch.cuda.synchronize()
        assert torch.equal(xx, want[0]) and torch.equal(rr, want[1])
        y, s, _, _ = ss.rms_norm_fwd(xx, out=xx)
        assert y is xx and s is not xx
        dy, dr = rnd(gen, 7, width), rnd(gen, 7, width)
        g = ss.rms_norm_bwd(dy, r, None, want[2], dresidual=dr)
        st = ss.lib().selscan_rms_norm_bwd(ctypes.byref(sh), dy.data_ptr(), r.data_ptr(), None, None, want[2].data_ptr(),
                                           dr.data_ptr(), None, dr.data_ptr(), None, None, torch.cuda.current_stream().cuda_stream)
        assert st == ss.OK
        torch.cuda.synchronize()
        assert torch.equal(dr, g["dresidual"])


def test_rows_do_not_touch_each_other(gpu):
    gen = torch.Generator().manual_seed(8)
    for width in (9, 100, 2557, 9001):
        x = rnd(gen, 5, width, dtype=BF16)
        want = ss.rms_norm_fwd(x)[0]
        for bad in (float("nan"), float("inf")):
            z = x.clone()
            z[2, width // 2] = bad
            y, _, rstd, _ = ss.rms_norm_fwd(z)
            keep = [0, 1, 3, 4]
            assert torch.equal(y[keep], want[keep]) and y[2, width // 2].isnan()
            q, _, _, scale = ss.rms_norm_fwd(z, out_dtype=E4M3, scale_block=0)
            assert scale[2].isnan().all() and scale[keep].isfinite().all() and q[2].float().isnan().all()


def test_one_dimension_and_refusals(gpu):
    x = torch.randn(64, device=DEV)
    y, s, rstd, _ = ss.rms_norm_fwd(x, gate=x)
    assert y.shape == (64,) and rstd.shape == (1,) and s is None
    with pytest.raises(ValueError, match="not both"):
        ss.rms_norm_fwd(x, residual=x, gate=x)
    with pytest.raises(ValueError, match="evenly"):
        a = torch.randn(2, 3, 4, 8, device=DEV)
        ss.rms_norm_fwd(a, gate=a.transpose(0, 1).contiguous().transpose(0, 1))
    with pytest.raises(TypeError):
        ss.rms_norm_fwd(x, gate=x.bfloat16())
    with pytest.raises(ss.SelscanError):
        ss.rms_norm_fwd(x, groups=3)
    with pytest.raises(ss.SelscanError):
        ss.rms_norm_fwd(x, out_dtype=E4M3, scale_block=48)
    with pytest.raises(TypeError):
        ss.rms_norm_fwd(x.half())


def test_many_short_rows_sum_in_order(gpu):
    """More partial rows than one pass of the column sums takes; terms of one sign."""
    rows, dim = 1 << 22, 16
    s = torch.ones(rows, dim, dtype=BF16, device=DEV)
    dy = torch.full((rows, dim), 1.0 / 3.0, device=DEV)
    rstd = torch.ones(rows, 1, device=DEV)
    a, b = ss.rms_norm_bwd(dy, s, None, rstd), ss.rms_norm_bwd(dy, s, None, rstd)
    third = torch.tensor(1.0 / 3.0).double()
    assert ((a["dweight"].cpu().double() / (rows * third) - 1).abs() <= 97 * 2.0 ** -24).all()
    assert torch.equal(a["dweight"], b["dweight"])


def test_graph_replays(gpu):
    gen = torch.Generator().manual_seed(9)
    x, r, w, dy = rnd(gen, 33, 640, dtype=BF16), rnd(gen, 33, 640), rnd(gen, 640), rnd(gen, 33, 640, dtype=BF16)
    run = lambda: [t for t in (*ss.rms_norm_fwd(x, w, r), *ss.rms_norm_fwd(x, w, gate=x, out_dtype=E4M3, scale_block=128))
                   if t is not None]
    def both():
        outs = run()
        g = ss.rms_norm_bwd(dy, outs[1], w, outs[2], x_dtype=BF16)
        return outs + [g["dx"], g["dresidual"], g["dweight"]]
    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = both()
    for _ in range(3):
        x.copy_(rnd(gen, 33, 640, dtype=BF16))
        graph.replay()
        want = both()
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(outs, want))
