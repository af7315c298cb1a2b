"""Pins of the MXFP4 quantisation oracle against what the format fixes (CPU)."""
import numpy as np
import pytest

from oracle import mx4
from oracle.mxfp4 import E2M1_VALUES, dequant


@pytest.mark.parametrize("rule", ["fit", "ocp"])
def test_nearest_code_by_brute_force(rule):
    """Every value of a fine grid over two binades of block maxima: no code is nearer, ties go to the even code."""
    top = np.concatenate([np.linspace(1, 8, 57), 2.0 ** np.arange(-6, 7), 6 * 2.0 ** np.arange(-6, 7)])
    x = np.zeros((len(top) * 65, 32))
    x[:, 0] = np.repeat(top, 65)
    x[:, 1] = np.tile(np.linspace(-1, 1, 65), len(top)) * x[:, 0]
    q, s = mx4.quantize(x, rule)
    v = mx4.dequantize(q, s, 32)
    scale = 2.0 ** (s[:, 0].astype(float) - 127)
    assert (scale == [2.0 ** (np.floor(np.log2(t)) - 2) if rule == "ocp" else
                      min(2.0 ** e for e in range(-20, 20) if t <= 6 * 2.0 ** e) for t in x[:, 0]]).all()
    near = np.abs(x[:, 1:2] / scale[:, None] - E2M1_VALUES[None, :])
    off = np.abs(v[:, 1] - x[:, 1]) / scale
    assert (off == near.min(1)).all()
    ties = [(0.25, 0.0), (0.75, 1.0), (1.25, 1.0), (1.75, 2.0), (2.5, 2.0), (3.5, 4.0), (5.0, 4.0)]
    assert all(mx4.grid(np.array([a, -a])).tolist() == [b, -b] for a, b in ties)
    assert np.signbit(mx4.grid(np.array([-0.0, -0.1]))).all()


def test_packing_is_the_weights():
    rng = np.random.default_rng(0)
    q, s = mx4.quantize(rng.normal(size=(5, 96)))
    assert (mx4.dequantize(q, s, 96) == dequant(q, s)).all()
    x = rng.normal(size=(3, 45))
    q, s = mx4.quantize(x)
    assert q.shape == (3, 23) and s.shape == (3, 2) and (q[:, -1] >> 4 == 0).all()
    padded = np.zeros((3, 64))
    padded[:, :45] = x
    q2, s2 = mx4.quantize(padded)
    assert (q == q2[:, :23]).all() and (s == s2).all()


def test_ends_of_the_range():
    x = np.zeros((6, 32))
    x[1, 3], x[2, 4], x[3, 5], x[4, 6], x[5, 7] = 1e-45, 3.4e38, np.inf, np.nan, -2.0 ** -126
    for rule in ("fit", "ocp"):
        q, s = mx4.quantize(x, rule)
        assert s[:, 0].tolist() == [2, 2, 253 if rule == "fit" else 252, 255, 255, 2]
        assert (q[[0, 1, 3, 4]] == 0).all()
        assert mx4.dequantize(q, s, 32)[5, 7] == -2.0 ** -126
    assert mx4.quantize(np.full((1, 32), 7.9), "ocp")[0][0, 0] == 0x77  # saturates at 6
    assert mx4.dequantize(*mx4.quantize(np.full((1, 32), 7.9), "fit"), 32)[0, 0] == 8.0


def test_expert_product_is_one_product_per_row():
    rng = np.random.default_rng(1)
    w, w3, x = rng.normal(size=(3, 4, 6)), rng.normal(size=(3, 4, 6)), rng.normal(size=(5, 6))
    rows, off, pw = np.array([4, 0, 0, 2]), [0, 1, 1, 3], np.array([1.0, 2.0, 0.0, 9.0])
    out, gate, _ = mx4.expert_product(x, w, off, rows=rows, pair_weight=pw)
    for p, e in ((0, 0), (1, 2), (2, 2)):
        assert np.allclose(gate[p], [x[rows[p]] @ w[e, n] for n in range(4)])
        assert np.allclose(out[p], pw[p] * gate[p])
        for n in range(4):
            g, u = x[rows[p]] @ w[e, n], x[rows[p]] @ w3[e, n]
            f = 4 * np.tanh(g / 4) / (1 + np.exp(-g)) * 25 * np.tanh(u / 25)
            assert np.isclose(mx4.expert_product(x, w, off, w3, rows)[0][p, n], f)
    assert np.isnan(out[3]).all()
