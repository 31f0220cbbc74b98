"""Pins for the oracle's batched operators (CPU only): library routines, closed
forms and the single-sequence oracle."""

import math

import numpy as np
import pytest
import torch

from oracle import batch as ob
from oracle import layer as ol


def test_slots_by_hand():
    # pages of 4; request 0: 6 cached, 3 new (page 7 holds 4..7, one new page);
    # 1: nothing new; 2: 0 cached, 4 new (one page); 3: 4 cached, 1 new (one page, none left)
    table = np.array([[5, 7, -1], [2, -1, -1], [-1, -1, -1], [3, -1, -1]])
    r = ob.build_slots([6, 1, 0, 4], [3, 0, 4, 1], [9, 8, 6], 1, table, 10, 4, 10, prefix=100)
    assert r["table"].tolist() == [[5, 7, 8], [2, -1, -1], [6, -1, -1], [3, -1, -1]]
    assert r["cu_rows"].tolist() == [0, 3, 3, 7, 8]
    assert r["lens"].tolist() == [9, 1, 4, 4]
    assert r["positions"].tolist() == [106, 107, 108, 100, 101, 102, 103, 104, 0, 0]
    assert r["slots"].tolist() == [30, 31, 32, 24, 25, 26, 27, -1, -1, -1]
    assert r["row_request"].tolist() == [0, 0, 0, 2, 2, 2, 2, 3, -1, -1]
    assert r["summary"].tolist() == [3, 8, 1, 3]


def test_slots_are_distinct_and_consistent():
    rng = np.random.default_rng(3)
    B, page, width = 40, 16, 12
    cached, new = rng.integers(0, 100, B), rng.integers(0, 60, B)
    pages = rng.permutation(2000)
    table = pages[:B * width].reshape(B, width).copy()
    held = -(-cached // page)
    table[np.arange(width)[None] >= held[:, None]] = -1
    r = ob.build_slots(cached, new, pages[B * width:], 0, table, int(new.sum()), page, 2000)
    assert (r["slots"] >= 0).all() and len(set(r["slots"].tolist())) == new.sum()
    for row in range(int(new.sum())):
        b = r["row_request"][row]
        assert r["table"][b, r["positions"][row] // page] == r["slots"][row] // page
        assert r["positions"][row] % page == r["slots"][row] % page


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_is_complex_multiplication_and_relative(layout):
    rng = np.random.default_rng(4)
    rot, d = 16, 24
    f, m = ob.rope_frequencies(rot)
    assert m == 1.0 and f[0] == 1.0 and math.isclose(f[4], 0.01)
    x = rng.standard_normal((5, 2, d))
    pos = np.array([0, 1, 7, 1000, 123456])
    y = ob.rope(x, pos, rot, layout, f, m)
    assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., rot:], x[..., rot:])
    pick = (lambda v: v[..., :8] + 1j * v[..., 8:16]) if layout == "half" else \
        (lambda v: v[..., 0:16:2] + 1j * v[..., 1:16:2])
    z = pick(x) * np.exp(1j * pos[:, None] * f)[:, None]
    assert np.allclose(pick(y), z, atol=1e-12)
    # a score depends on the distance of the positions only
    k = rng.standard_normal((1, 1, d))
    q = rng.standard_normal((1, 1, d))
    s = [float((ob.rope(q, [a + 13], rot, layout, f, m) * ob.rope(k, [a], rot, layout, f, m)).sum())
         for a in (0, 5, 4000)]
    assert np.allclose(s, s[0], atol=1e-9)


def test_rope_scalings():
    f, _ = ob.rope_frequencies(64)
    lin, m = ob.rope_frequencies(64, scaling="linear", factor=4.0)
    assert np.allclose(lin, f / 4) and m == 1.0
    base, _ = ob.rope_frequencies(64, scaling="base", factor=4.0)
    assert base[0] == 1.0 and math.isclose(base[-1], f[-1] / 4)  # the slowest pair is stretched by `factor`
    parts, m = ob.rope_frequencies(64, scaling="parts", factor=4.0, orig_ctx=4096)
    turns = 4096 * f / (2 * math.pi)
    assert np.allclose(parts[turns >= 32], f[turns >= 32]) and np.allclose(parts[turns <= 1], f[turns <= 1] / 4)
    assert np.all(parts <= f) and np.all(parts >= f / 4 * (1 - 1e-15)) and math.isclose(m, 1 + 0.1 * math.log(4))
    assert ob.rope_frequencies(64, scaling="parts", factor=4.0, orig_ctx=4096, attn_factor=0.5)[1] == 0.5


@pytest.mark.parametrize("window,tree", [(0, None), (9, None), (0, [1, 3, 5, 11]), (64, [1, 3, 5, 11])])
def test_attention_of_one_request_is_the_layers(window, tree):
    rng = np.random.default_rng(5)
    T, Hq, Hkv, d, prefix, cached, page = 4, 4, 2, 8, 16, 13, 16
    kc, vc = rng.standard_normal((64, Hkv, d)), rng.standard_normal((64, Hkv, d))
    q = rng.standard_normal((T, Hq, d))
    ref = ol.attention(q, kc, vc, prefix + cached, window, tree)
    pool = lambda x: x.reshape(-1, page, Hkv, d)  # noqa: E731
    out, lse, _ = ob.prefix_attn(q, pool(kc), pool(vc), [0], prefix, np.array([[1, 2]]), [cached + T],
                                 [0, T], window, tree=tree)
    assert np.allclose(out, ref, atol=1e-13)
    if window == 0 and tree is None:
        k = torch.from_numpy(kc[:prefix + cached + T, 0])
        s = torch.from_numpy(q[T - 1, 0]) @ k.T / math.sqrt(d)
        assert math.isclose(lse[T - 1, 0], float(torch.logsumexp(s, 0)))


def test_attention_rows_without_keys_and_pages_outside():
    q = np.ones((3, 1, 4))
    pool = np.ones((2, 16, 1, 4))
    out, lse, _ = ob.prefix_attn(q, pool, pool, [], 0, np.array([[0], [7]]), [0, 2], [0, 1, 2])
    assert np.all(out[0] == 0) and lse[0, 0] == -np.inf
    assert np.all(out[1] == 0) and math.isclose(lse[1, 0], math.log(2))  # two keys of zeros
    assert np.isnan(out[2]).all()
