"""The float64 oracle of the cache in 4 bits, pinned by hand and by brute force (CPU only)."""

import math

import numpy as np
import pytest

from oracle import batch as ob
from oracle import kvq as ok


def test_e4m3_values_and_rounding():
    torch = pytest.importorskip("torch")
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, ok.E4M3) and ok.E4M3[-1] == 448 and ok.E4M3[1] == 2.0 ** -9
    assert np.array_equal(ok.e4m3(ok.E4M3), np.arange(127))
    mid = (ok.E4M3[:-1] + ok.E4M3[1:]) / 2
    assert np.array_equal(ok.e4m3(mid), np.arange(126) + np.arange(126) % 2)      # ties to even
    assert np.array_equal(ok.e4m3(mid * (1 - 1e-12)), np.arange(126))
    assert np.array_equal(ok.e4m3(mid * (1 + 1e-12)), np.arange(126) + 1)
    assert ok.e4m3(1e9) == 126


def test_encode_by_hand():
    y = np.zeros(32)
    y[:16] = [7, -7, 3.5, 2.5, -0.5, 0.49, 0.51, 1, 0, 0, 0, 0, 0, 0, 0, -6.6]
    codes, scales = ok.encode(y[None])
    n = [codes[0, i // 2] >> 4 * (i & 1) & 15 for i in range(32)]
    assert n[:8] == [15, 1, 12, 10, 8, 8, 9, 9] and n[15] == 1 and n[16:] == [8] * 16  # halves to even
    assert ok.E4M3[scales[0]].tolist() == [1.0, 0.0]
    assert ok.decode(codes, scales)[0, :4].tolist() == [7, -7, 4, 2]
    c2, s2 = ok.encode(y[None] * 8, e=np.array([3]))
    assert np.array_equal(c2, codes) and np.array_equal(s2, scales)


def test_encode_extremes():
    y = np.zeros((4, 16))
    y[0, 3], y[1, 5], y[2, 0], y[3, 0] = np.inf, np.nan, 7 * 2.0 ** -10, 7.1 * 2.0 ** -10
    y[0, 4], y[0, 5] = -np.inf, 448 * 3
    codes, scales = ok.encode(y)
    assert scales[:, 0].tolist() == [126, 127, 0, 1]
    n = [codes[0, i // 2] >> 4 * (i & 1) & 15 for i in range(16)]
    assert n[3:6] == [15, 0, 11] and np.all(codes[1] == 0x88) and np.all(codes[2] == 0x88)
    assert np.isnan(ok.decode(codes, scales)[1]).all()


def test_encode_is_the_nearest_value():
    rng = np.random.default_rng(0)
    y = rng.standard_normal((50, 64)) * np.exp(rng.uniform(-3, 3, (50, 1)))
    codes, scales = ok.encode(y)
    got, s = ok.decode(codes, scales), np.repeat(ok.E4M3[scales], 16, -1)
    grid = (np.arange(16) - 8)[None, None] * s[..., None]
    best = np.abs(grid - y[..., None]).min(-1)
    assert np.allclose(np.abs(got - y), best, rtol=0, atol=1e-12)
    top = np.abs(y).reshape(50, 4, 16).max(-1)
    assert np.all(np.abs(ok.E4M3[scales] - top / 7) <= top / 7 / 16 + 2.0 ** -10)


def test_scale_ties():
    """A largest value that is seven times the middle between two scales."""
    for k in range(8, 100):
        mid = (ok.E4M3[k] + ok.E4M3[k + 1]) / 2
        y = np.zeros((1, 16))
        y[0, 0] = 7 * mid
        assert ok.encode(y)[1][0, 0] == k + k % 2


def test_norm_and_rotation():
    rng = np.random.default_rng(1)
    x, w = rng.standard_normal((3, 2, 16)), rng.standard_normal(16)
    n = ok.norm(x, w, 1e-6)
    assert math.isclose(n[1, 1, 4], x[1, 1, 4] * w[4] / math.sqrt((x[1, 1] ** 2).mean() + 1e-6), rel_tol=1e-14)
    f, m = ob.rope_frequencies(16)
    y, mag = ok.norm_rope(x, w, 1e-6, [0, 5, 9], 16, "half", f, m)
    assert np.allclose(y[0], n[0]) and np.all(np.abs(y) <= mag + 1e-12)
    a = 9 * f[3]
    assert math.isclose(y[2, 0, 11], n[2, 0, 11] * math.cos(a) + n[2, 0, 3] * math.sin(a), rel_tol=1e-12)


def test_linear():
    x, w = np.array([[1.0, -2.0]]), np.array([[3.0, 1.0], [0.5, 0.5], [0.0, 0.0]])
    y, s = ok.linear(x, w, np.array([1.0, 0.0, 0.0]), "silu", np.array([[0.0, 10.0, 1.0]]))
    assert np.allclose(y, [[2 / (1 + math.exp(-2)), 10 - 0.5 / (1 + math.exp(0.5)), 1.0]]) and np.allclose(s, [[5, 1.5, 0]])
    g, _ = ok.linear(x, w, act="gelu")
    assert math.isclose(g[0, 0], 0.5 * (1 + math.erf(1 / math.sqrt(2))))
    t, _ = ok.linear(x, w, act="gelu_tanh")
    assert abs(t[0, 0] - g[0, 0]) < 1e-3
