"""The fp64 oracle of the gated delta rule, layer norm and dropout, pinned:
closed forms, published vectors of the generator, finite differences (CPU)."""
import numpy as np
import pytest

from oracle import block_ops as ref


def _delta_inputs(B, L, H, G, P, N, seed):
    r = np.random.default_rng(seed)
    unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)
    return dict(q=unit(r.standard_normal((B, L, G, N))), k=unit(r.standard_normal((B, L, G, N))),
                v=r.standard_normal((B, L, H, P)), g=-r.uniform(0, 0.5, (B, L, H)), beta=r.uniform(0, 1, (B, L, H)))


def test_delta_writes_and_reads_back():
    """With orthonormal keys, no decay and beta 1, reading with a key returns
    what was last written under it."""
    N = P = 4
    k = np.eye(N)[[0, 1, 2, 0]][None, :, None, :]
    v = np.random.default_rng(1).standard_normal((1, 4, 1, P))
    y, S = ref.delta(k, k, v, np.zeros((1, 4, 1)), np.ones((1, 4, 1)), scale=1.0)
    np.testing.assert_allclose(y, v, atol=1e-14)
    np.testing.assert_allclose(S[0, 0] @ k[0, 0, 0], v[0, 3, 0], atol=1e-14)


def test_delta_without_erasing_is_the_mamba2_recurrence():
    """Keys of one token orthogonal to every state: the rule is a plain decayed sum."""
    i = _delta_inputs(1, 3, 2, 1, 3, 6, 2)
    i["k"] = np.eye(6)[:3].reshape(1, 3, 1, 6)
    _, S = ref.delta(**i)
    want = np.zeros((2, 3, 6))
    for h in range(2):
        for t in range(3):
            want[h] = np.exp(i["g"][0, t, h]) * want[h] + i["beta"][0, t, h] * np.outer(i["v"][0, t, h], i["k"][0, t, 0])
    np.testing.assert_allclose(S[0], want, atol=1e-14)


def test_delta_split_equals_whole_and_lengths():
    i = _delta_inputs(2, 9, 2, 2, 3, 5, 3)
    y, S = ref.delta(**i)
    a = {n: x[:, :4] for n, x in i.items()}
    b = {n: x[:, 4:] for n, x in i.items()}
    y1, S1 = ref.delta(**a)
    y2, S2 = ref.delta(**b, h0=S1)
    np.testing.assert_allclose(np.concatenate([y1, y2], 1), y, atol=1e-13)
    np.testing.assert_allclose(S2, S, atol=1e-13)
    yl, Sl = ref.delta(**i, lengths=[4, 0])
    np.testing.assert_allclose(yl[0, :4], y[0, :4], atol=1e-14)
    assert not yl[0, 4:].any() and not yl[1].any() and not Sl[1].any()
    np.testing.assert_allclose(Sl[0], S1[0], atol=1e-14)


@pytest.mark.parametrize("name", ["q", "k", "v", "g", "beta", "h0"])
def test_delta_gradient_matches_differences(name):
    i = _delta_inputs(2, 6, 4, 2, 3, 5, 4)
    r = np.random.default_rng(5)
    i["h0"] = r.standard_normal((2, 4, 3, 5))
    dout, dlast = r.standard_normal((2, 6, 4, 3)), r.standard_normal((2, 4, 3, 5))
    lengths = [6, 3]
    grad = ref.delta_bwd(**i, dout=dout, dlast=dlast, lengths=lengths)["d" + name]

    def loss(x):
        y, S = ref.delta(**{**i, name: x}, lengths=lengths)
        return (y * dout).sum() + (S * dlast).sum()

    for _ in range(6):
        d = r.standard_normal(i[name].shape)
        e = 1e-5
        num = (loss(i[name] + e * d) - loss(i[name] - e * d)) / (2 * e)
        assert abs(num - (grad * d).sum()) <= 1e-7 * max(1.0, abs(num))


@pytest.mark.parametrize("counter,key,words", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))])
def test_philox_known_answers(counter, key, words):
    """The generator's published test vectors."""
    assert tuple(ref.philox(counter, key)) == words


def test_dropout_rate_and_edges():
    assert ref.keep(20000, 0.3, 7, 0).mean() == pytest.approx(0.7, abs=4 * (0.21 / 20000) ** 0.5)
    assert ref.keep(100, 0.0, 7, 0).all() and not ref.keep(100, 1.0, 7, 0).any()
    assert not np.array_equal(ref.keep(100, 0.5, 7, 0), ref.keep(100, 0.5, 7, 1))


@pytest.mark.parametrize("name", ["x", "weight", "bias", "residual"])
def test_layer_norm_gradient_matches_differences(name):
    r = np.random.default_rng(6)
    i = dict(x=r.standard_normal((5, 7)), weight=r.standard_normal(7), bias=r.standard_normal(7),
             residual=r.standard_normal((5, 7)))
    kw = dict(p=0.4, seed=3, offset=9)
    dy, ds = r.standard_normal((5, 7)), r.standard_normal((5, 7))
    _, s, mean, rstd = ref.layer_norm(**i, **kw)
    grad = ref.layer_norm_bwd(dy, s, i["weight"], mean, rstd, ds, **kw)["d" + name]

    def loss(x):
        y, s, _, _ = ref.layer_norm(**{**i, name: x}, **kw)
        return (y * dy).sum() + (s * ds).sum()

    for _ in range(4):
        d = r.standard_normal(i[name].shape)
        num = (loss(i[name] + 1e-5 * d) - loss(i[name] - 1e-5 * d)) / 2e-5
        assert abs(num - (grad * d).sum()) <= 1e-7 * max(1.0, abs(num))
