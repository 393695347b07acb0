"""Pins of the oracle's integer 4-bit and expert functions: hand-worked
weights and routes, torch's softmax and topk, exact rationals."""
from fractions import Fraction

import numpy as np
import torch

import oracle


def test_dequant_by_hand():
    codes = np.zeros((1, 32), dtype=np.uint8)
    codes[0, 0] = 0x3F  # elements 0, 1 = 15, 3
    codes[0, 16] = 0x80  # elements 32, 33 = 0, 8
    scale = np.array([[0.5, 2.0]], dtype=np.float16)
    zero = np.array([[4, 8]], dtype=np.uint8)
    w = oracle.w4g_dequant(codes, scale, zero)
    assert w.shape == (1, 64)
    assert list(w[0, :3]) == [5.5, -0.5, -2.0] and list(w[0, 32:35]) == [-16.0, 0.0, -16.0]
    # without zero points the codes are centred on 8
    assert list(oracle.w4g_dequant(codes, scale, None)[0, :2]) == [3.5, -2.5]


def test_proj_is_the_rational_sum():
    r = np.random.default_rng(3)
    a = r.integers(-9, 10, (2, 64)) / 8.0
    codes = r.integers(0, 256, (3, 32)).astype(np.uint8)
    scale = (r.integers(1, 30, (3, 2)) / 64.0).astype(np.float32)
    zero = r.integers(0, 16, (3, 2)).astype(np.uint8)
    out, mag = oracle.w4g_proj(a, codes, scale, zero)
    for m in range(2):
        for n in range(3):
            s = t = Fraction(0)
            for k in range(64):
                q = (int(codes[n, k // 2]) >> (4 * (k % 2))) & 15
                p = Fraction(a[m, k]) * (q - int(zero[n, k // 32])) * Fraction(float(scale[n, k // 32]))
                s += p
                t += abs(p)
            assert Fraction(out[m, n]) == s and Fraction(mag[m, n]) == t


def test_route_by_hand():
    inf = float("inf")
    x = np.array([[1.0, 3.0, 3.0, 2.0], [-inf, float("nan"), 0.0, -inf], [-inf] * 4, [0.0, -0.0, inf, inf]])
    ids, w, off, rows, pos = oracle.moe_route(x, 2)
    assert ids.tolist() == [[1, 2], [2, -1], [-1, -1], [2, 3]]
    assert np.allclose(w, [[0.5, 0.5], [1, 0], [0, 0], [0.5, 0.5]])
    assert off.tolist() == [0, 0, 1, 4, 5]
    assert rows.tolist() == [0, 0, 1, 3, 3, -1, -1, -1]
    assert pos.tolist() == [[0, 1], [2, -1], [-1, -1], [3, 4]]
    _, w, _, _, _ = oracle.moe_route(x, 2, renormalize=False)
    assert np.allclose(w[0], np.exp(3.0) / np.exp([1.0, 3.0, 3.0, 2.0]).sum()) and np.allclose(w[1], [1, 0])


def test_route_matches_torch():
    x = torch.randn(50, 12, generator=torch.Generator().manual_seed(1), dtype=torch.float64)
    p, i = torch.softmax(x, 1).topk(3, dim=1)
    ids, w, off, rows, pos = oracle.moe_route(x.numpy(), 3, renormalize=False)
    assert np.array_equal(ids, i.numpy()) and np.allclose(w, p.numpy(), rtol=1e-12)
    ids, w, off, rows, pos = oracle.moe_route(x.numpy(), 3)
    assert np.allclose(w, (p / p.sum(1, keepdim=True)).numpy(), rtol=1e-12)
    assert np.array_equal(np.diff(off), np.bincount(ids.ravel(), minlength=12))
    for t in range(50):
        for s in range(3):
            assert rows[pos[t, s]] == t and off[ids[t, s]] <= pos[t, s] < off[ids[t, s] + 1]


def test_combine_by_hand():
    y = np.array([[1.0, -2.0], [4.0, 8.0]])
    out, mag = oracle.moe_combine(y, np.array([[1, 0], [-1, 2], [1, 1]]),
                                  np.array([[0.5, 0.25], [1.0, 1.0], [1.0, -0.5]]), np.array([[1.0, 1], [2, 3], [0, 0]]))
    assert out.tolist() == [[3.25, 4.5], [2.0, 3.0], [2.0, 4.0]]
    assert mag.tolist() == [[3.25, 5.5], [2.0, 3.0], [6.0, 12.0]]
