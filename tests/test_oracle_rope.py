"""The fp64 rotation and norms against their definitions: rotations compose and undo, gradients match differences; and
the frequencies that Rope makes."""
import math

import numpy as np
import pytest

import oracle
from learned_kv_cache_gb300 import Rope

rng = np.random.default_rng(5)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_the_complex_product(interleaved):
    x = rng.standard_normal((3, 7, 64))
    pos = rng.integers(-50, 1000, (3, 7))
    inv = Rope(32, theta=1e4).inv_freq
    y = oracle.rotate(x, pos, inv, interleaved, gain=1.3)
    a, b = (x[..., 0:32:2], x[..., 1:32:2]) if interleaved else (x[..., :16], x[..., 16:32])
    z = 1.3 * (a + 1j * b) * np.exp(1j * pos[..., None] * np.array(inv))
    ya, yb = (y[..., 0:32:2], y[..., 1:32:2]) if interleaved else (y[..., :16], y[..., 16:32])
    assert np.abs(ya + 1j * yb - z).max() < 1e-12
    assert (y[..., 32:] == x[..., 32:]).all()
    back = oracle.rotate(y, pos, inv, interleaved, gain=1 / 1.3, inverse=True)
    assert np.abs(back - x).max() < 1e-12


def test_logits_depend_on_the_distance_only():
    inv = Rope(64, theta=1e6).inv_freq
    q, k = rng.standard_normal((2, 1, 64))
    dots = [(oracle.rotate(q, [p + 11], inv) * oracle.rotate(k, [p], inv)).sum() for p in (0, 5, 131072, 2 ** 31 - 12)]
    assert np.ptp(dots) < 1e-11


@pytest.mark.parametrize("weighted", [False, True])
def test_norm_gradient_matches_differences(weighted):
    x, dy = rng.standard_normal((2, 2, 3, 64))
    w = rng.uniform(0.2, 2, 64) if weighted else None
    pos, inv = np.array([7, 1, 900]), Rope(32).inv_freq
    dx, dw = oracle.norm_rope_backward(dy, x, w, 1e-3, pos, inv, True, 1.1)

    def loss(x, w):
        return (oracle.norm_rope(x, w, 1e-3, pos, inv, True, 1.1) * dy).sum()
    h = 1e-6
    for _ in range(20):
        at = tuple(rng.integers(0, n) for n in x.shape)
        e = np.zeros_like(x)
        e[at] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[at]) < 1e-7
        if weighted:
            e = np.zeros(64)
            e[at[-1]] = h
            assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[at[-1]]) < 1e-7


def test_frequencies():
    plain = Rope(128, theta=5e5)
    assert plain.inv_freq[0] == 1.0 and plain.gain == 1.0
    assert plain.inv_freq[63] == pytest.approx(5e5 ** (-126 / 128), rel=1e-14)
    assert Rope(128, theta=5e5, scaling="linear", factor=4.0).inv_freq[5] == plain.inv_freq[5] / 4
    ntk = Rope(128, theta=5e5, scaling="ntk", factor=4.0)
    assert ntk.inv_freq[0] == 1.0 and ntk.inv_freq[63] == pytest.approx(plain.inv_freq[63] / 4, rel=1e-12)
    bands = Rope(128, theta=5e5, scaling="bands", factor=8.0, original_len=8192)
    for f, g in zip(plain.inv_freq, bands.inv_freq):
        wave = 2 * math.pi / f
        if wave < 8192 / 4:
            assert g == pytest.approx(f, rel=1e-14)
        elif wave > 8192:
            assert g == pytest.approx(f / 8, rel=1e-14)
        else:
            assert f / 8 <= g <= f
    yarn = Rope(128, theta=1e6, scaling="yarn", factor=4.0, original_len=32768)
    assert yarn.gain == pytest.approx(0.1 * math.log(4) + 1)
    assert yarn.inv_freq[0] == 1.0
    assert yarn.inv_freq[63] == pytest.approx(Rope(128, theta=1e6).inv_freq[63] / 4, rel=1e-14)
    given = Rope(16, inv_freq=[0.5] * 8, gain=2.0)
    assert given.inv_freq == (0.5,) * 8 and given.gain == 2.0


@pytest.mark.parametrize("kw", [dict(rotary_dim=24), dict(rotary_dim=0), dict(rotary_dim=256), dict(theta=1.0),
                                dict(theta=math.nan), dict(scaling="cubic"), dict(scaling="yarn", factor=2.0),
                                dict(scaling="bands", factor=2.0, original_len=100, low=4.0, high=4.0),
                                dict(scaling="linear", factor=0.0), dict(inv_freq=[1.0]), dict(inv_freq=[-1.0] * 32),
                                dict(inv_freq=[math.inf] * 32), dict(inv_freq=[1.0] * 32, scaling="linear", factor=2.0),
                                dict(gain=math.inf)])
def test_bad_frequencies_are_refused(kw):
    with pytest.raises(ValueError):
        Rope(**{"rotary_dim": 64, **kw})
