"""Comparison with the fp64 oracle, element by element, under a bound that is
a number of fp32 roundings of the terms and one rounding of the result."""
import torch


def close(got, ref, size, roundings, what):
    """|got - ref| <= roundings 2^-24 size + half a step of the result's type."""
    g = got.detach().cpu().double()
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    half = torch.finfo(got.dtype).eps / 2
    bound = roundings * 2.0 ** -24 * size + half * ref.abs() + 1e-38
    off = (g - ref).abs()
    bad = ~(off <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {(off / bound).max():.3g} times the bound"
