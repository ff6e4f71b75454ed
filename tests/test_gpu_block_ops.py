"""Layer norm (with dropout and residual) and dropout on the GPU against the
fp64 oracle."""
import numpy as np
import pytest
import torch

import selective_state_space_25_amd as ss
from oracle import block_ops as ref
from parity import check_close, host

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16

# fp32 sums of up to 2^13 terms in a tree: 2^-24 x log2 of the terms, a few
# stages and one division and square root: 2^-19 of the values' scale
TOL = 2.0 ** -19


def _tol(dtype, ref_values, tol=TOL):
    """|err| <= tol (rms + |ref|), plus half a bf16 step of a bf16 output."""
    rms = float(np.sqrt(np.mean(np.square(ref_values)))) + 1e-30
    return tol * max(rms, 1.0), tol + (2.0 ** -8 if dtype == BF16 else 0.0)


def _normal(shape, seed, dtype=F32, shift=0.0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale + shift).to(dtype).to(DEV)


@pytest.mark.parametrize("n", [1, 3, 4, 5, 1023, 4099])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("p", [0.0, 0.3, 1.0])
def test_dropout_matches_oracle(gpu, n, dtype, p):
    x = _normal((n,), n, dtype)
    seed, offset = (5 << 40) + 77, (1 << 33) + 1
    y = ss.dropout(x, p, seed, offset)
    want = ref.dropout(x, p, seed, offset)
    # one rounding of the scale, one of the product
    check_close(host(y).double().numpy(), want, (0.0, 2.0 ** -22 + (2.0 ** -8 if dtype == BF16 else 0.0)))
    assert np.array_equal(host(y).double().numpy() == 0.0, want == 0.0)


@pytest.mark.parametrize("shift", [0, 1])
def test_dropout_in_place_unaligned_and_backward(gpu, shift):
    """Starting off a 16-byte boundary, in place, on another stream; the
    gradient's mask is the output's; dropped NaN is zero."""
    buf = _normal((1000 + shift,), 3)
    x = buf[shift:]
    x[10:20] = float("nan")
    keep = torch.from_numpy(ref.keep(1000, 0.5, 9, 0)).to(DEV)
    want = torch.where(keep, x * 2, torch.zeros(()).to(DEV))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = ss.dropout(x, 0.5, 9, out=x)
        d = ss.dropout(torch.ones_like(x), 0.5, 9)
    torch.cuda.synchronize()
    assert y.data_ptr() == x.data_ptr()
    assert torch.equal(torch.nan_to_num(y, nan=7.0), torch.nan_to_num(want, nan=7.0))
    assert torch.equal(d, 2.0 * keep.float())


NORM_SHAPES = [(1, 1), (3, 2), (1, 768), (5, 64), (7, 100), (4, 101), (130, 256), (3, 1000), (2, 2560), (3, 5121),
               (2, 8192), (2, 9001)]


@pytest.mark.parametrize("rows,dim", NORM_SHAPES)
@pytest.mark.parametrize("types", [(F32, F32, F32), (BF16, F32, BF16), (BF16, BF16, BF16), (F32, F32, BF16)])
@pytest.mark.parametrize("p", [0.0, 0.25])
def test_layer_norm_matches_oracle(gpu, rows, dim, types, p):
    tin, tres, tout = types
    x, r = _normal((rows, dim), 1, tin), _normal((rows, dim), 2, tres, 0.5, 2.0)
    w, b = _normal((dim,), 3, shift=1.0, scale=0.1), _normal((dim,), 4)
    kw = dict(p=p, seed=12345678901, offset=3)
    eps = 1e-3
    y, s, mean, rstd = ss.layer_norm_fwd(x, w, b, residual=r, eps=eps, out_dtype=tout, **kw)
    torch.cuda.synchronize()
    yr, sr, mr, rr = ref.layer_norm(x, w, b, r, eps, **kw)
    f = lambda t: host(t).double().numpy()
    # a rounding of s (2^-24 of it, twice) is carried into y times rstd weight
    amp = float(np.max(rr)) * 2.0 ** -21 * float(np.max(np.abs(sr)))
    ay, ry = _tol(tout, yr)
    check_close(f(y), yr, (ay + amp, ry), "y")
    check_close(f(s), sr, _tol(tres, sr), "s")
    check_close(f(mean), mr, _tol(F32, sr), "mean")
    # rstd's relative error is half the variance's, to which 2^-23 of s adds
    # in proportion to rstd
    check_close(f(rstd), rr, (0.0, TOL + amp), "rstd")

    dy, dr = _normal((rows, dim), 5, tout), _normal((rows, dim), 6, tres)
    g = ss.layer_norm_bwd(dy, s, w, mean, rstd, dresidual=dr, x_dtype=tin, **kw)
    torch.cuda.synchronize()
    gr = ref.layer_norm_bwd(dy, s, w, mean, rstd, dr, **kw)
    big = float(np.max(host(rstd).double().numpy()))   # the terms that cancel are rstd times larger
    for name, t in (("dx", tin), ("dresidual", tres), ("dweight", F32), ("dbias", F32)):
        atol, rtol = _tol(t, gr[name])
        check_close(f(g[name]), gr[name], (atol * max(1.0, big), rtol), name)


@pytest.mark.parametrize("dim", [96, 333])
def test_layer_norm_options(gpu, dim):
    """No weight, no bias, no residual: s is x itself; gradients without the
    residual's; fp32 copy of a bf16 x on request; reproducible bit for bit."""
    x = _normal((65, dim), 11, BF16)
    y, s, mean, rstd = ss.layer_norm_fwd(x, out_dtype=F32)
    assert s is x
    yr, _, _, _ = ref.layer_norm(x)
    check_close(host(y).double().numpy(), yr, _tol(F32, yr), "y")
    assert ss.layer_norm_fwd(x, res_dtype=F32)[1].dtype == F32
    dy = _normal((65, dim), 12)
    g = ss.layer_norm_bwd(dy, s, None, mean, rstd)
    assert g["dx"] is g["dresidual"]
    gr = ref.layer_norm_bwd(dy, s, None, mean, rstd)
    check_close(host(g["dx"]).double().numpy(), gr["dx"], _tol(BF16, gr["dx"]), "dx")
    again = ss.layer_norm_bwd(dy, s, None, mean, rstd)
    assert all(torch.equal(g[n], again[n]) for n in g)


def test_layer_norm_extreme_rows(gpu):
    """A constant row (variance zero), a large offset, NaN confined to its row."""
    x = _normal((4, 512), 13)
    x[0] = 3.0
    x[1] += 1000.0
    x[2, 7] = float("nan")
    y, s, mean, rstd = ss.layer_norm_fwd(x, eps=1e-5)
    yr, _, mr, rr = ref.layer_norm(x)
    yh = host(y).double().numpy()
    assert np.all(yh[0] == 0.0) and np.isnan(yh[2]).all()
    assert float(host(rstd)[0]) == pytest.approx(1e-5 ** -0.5, rel=1e-6)
    # the mean of values near 1000 is off by up to 2^-24 x 1000 x a few
    check_close(yh[1], yr[1], (1000.0 * 2.0 ** -21, 2.0 ** -19), "offset row")
    check_close(yh[3], yr[3], _tol(F32, yr[3]), "plain row")


def test_layer_norm_does_not_touch_neighbours(gpu):
    buf = torch.full((3 * 77 + 8,), 5.0, device=DEV)
    out = buf[:3 * 77].view(3, 77)
    ss.layer_norm_fwd(_normal((3, 77), 14), out=out)
    torch.cuda.synchronize()
    assert torch.equal(host(buf[3 * 77:]), torch.full((8,), 5.0))


def test_workspace_too_small_is_refused(gpu):
    x = _normal((64, 128), 15)
    _, s, mean, rstd = ss.layer_norm_fwd(x)
    with pytest.raises(ss.SelscanError) as e:
        ss.layer_norm_bwd(x, s, None, mean, rstd, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    assert e.value.status == ss.ERR_WORKSPACE


@pytest.mark.parametrize("rows,dim", [(3, 3200), (2, 4096), (3, 5120), (2, 7000), (5000, 64), (2100, 3208)])
def test_layer_norm_longer_rows_and_many_rows(gpu, rows, dim):
    """Rows spread over a workgroup; more rows than one pass of the
    gradients' workgroups."""
    x, r = _normal((rows, dim), 21, BF16), _normal((rows, dim), 22)
    w = _normal((dim,), 23, shift=1.0, scale=0.1)
    y, s, mean, rstd = ss.layer_norm_fwd(x, w, None, residual=r, out_dtype=F32)
    yr, sr, _, rr = ref.layer_norm(x, w, None, r)
    amp = float(np.max(rr)) * 2.0 ** -21 * float(np.max(np.abs(sr)))
    ay, ry = _tol(F32, yr)
    check_close(host(y).double().numpy(), yr, (ay + amp, ry), "y")
    dy = _normal((rows, dim), 24)
    g = ss.layer_norm_bwd(dy, s, w, mean, rstd, x_dtype=BF16)
    gr = ref.layer_norm_bwd(dy, s, w, mean, rstd)
    for name, t in (("dx", BF16), ("dresidual", F32), ("dweight", F32), ("dbias", F32)):
        atol, rtol = _tol(t, gr[name])
        # (sums over the rows: their magnitudes add up where the result does not)
        check_close(host(g[name]).double().numpy(), gr[name], (atol * max(1.0, float(np.max(rr))), rtol), name)


@pytest.mark.parametrize("rows,dim", [((1 << 24) + 3, 5), ((1 << 24) + 5, 16)])
def test_layer_norm_more_rows_than_a_grid_dimension(gpu, rows, dim):
    """Rows past 2^32 threads in one dimension of the grid: the last rows equal those of their own call."""
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn((rows, dim), generator=g, device=DEV, dtype=torch.bfloat16)
    dy = torch.randn((rows, dim), generator=g, device=DEV, dtype=torch.bfloat16)
    y, s, mean, rstd = ss.layer_norm_fwd(x)
    d = ss.layer_norm_bwd(dy, s, None, mean, rstd)
    tail = slice(rows - 1000, rows)
    yt, st, mt, rt = ss.layer_norm_fwd(x[tail].contiguous())
    dt = ss.layer_norm_bwd(dy[tail].contiguous(), st, None, mt, rt)
    torch.cuda.synchronize()
    assert torch.equal(y[tail], yt) and torch.equal(mean[tail], mt) and torch.equal(rstd[tail], rt)
    assert torch.equal(d["dx"][tail], dt["dx"])


def test_dropout_past_32_bits(gpu):
    """Elements past 2^34, a grid of more than 2^32 threads: the last ones' words by their own counters."""
    n = (1 << 34) + 22
    x = torch.ones(n, dtype=torch.bfloat16, device=DEV)
    y = ss.dropout(x, 0.5, 9, 4, out=x)
    got = host(y[n - 22:]).double().numpy()
    first = n // 4 - 5
    words = np.asarray([w for c in range(first, first + 6) for w in ref.philox((c & 0xFFFFFFFF, c >> 32, 4, 0), (9, 0))])
    want = np.where(words >= (1 << 31), 2.0, 0.0)[(n - 22) - 4 * first:][:22]
    assert np.array_equal(got, want)
