"""Pins of the routed oracle: small cases worked by hand, and its gradients against central
differences."""
import numpy as np
import pytest

from oracle import routed as R


def test_choice_by_hand():
    l = np.array([[1.0, 3.0, 3.0, -np.inf], [-np.inf] * 4])
    assert R.choose(l, 3, "softmax").tolist() == [[1, 2, 0], [-1, -1, -1]]
    # a bias moves the choice but not the weights
    ids = R.choose(l, 1, "softmax", bias=[1.0, 0.0, 0.0, 5.0])
    assert ids.tolist() == [[0], [-1]]
    w = R.weights(l, ids, "softmax", False)
    assert np.isclose(w[0, 0], np.exp(1) / (np.exp(1) + 2 * np.exp(3))) and w[1, 0] == 0
    # groups of two: sums 1 + 0.5 against 1.25 + 0.1; best single 1.25
    s = np.log(np.array([[1.0, 0.5, 1.25, 0.1]]))
    assert R.choose(s, 2, "softmax", n_groups=2, top_groups=1, group_top=2).tolist() == [[0, 1]]
    assert R.choose(s, 2, "softmax", n_groups=2, top_groups=1, group_top=1).tolist() == [[2, 3]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_renormalised_weights_survive_underflow(score):
    l = np.array([[-1000.0, -1001.0, 0.0]])
    w = R.weights(l, np.array([[0, 1]]), score, True)
    e = np.exp(-1.0)
    assert np.allclose(w, [[1 / (1 + e), e / (1 + e)]], rtol=1e-12)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_against_differences(score, renorm):
    g = np.random.default_rng(3)
    l, gw = g.normal(size=(5, 9)), g.normal(size=(5, 4))
    ids = R.choose(l, 4, score)
    ids[1, 3] = -1
    ids[4] = -1
    d = R.route_grad(l, ids, gw, score, renorm, 1.5)
    h = 1e-5
    for t in range(5):
        for e in range(9):
            up, dn = l.copy(), l.copy()
            up[t, e] += h
            dn[t, e] -= h
            f = [(gw * R.weights(v, ids, score, renorm, 1.5)).sum() for v in (up, dn)]
            assert abs((f[0] - f[1]) / (2 * h) - d[t, e]) <= 1e-8


def test_mixture_gradient_against_differences():
    g = np.random.default_rng(4)
    d_in, d_out, ranks = 6, 5, [2, 1, 3]
    oA, oB = np.cumsum([0] + [k * d_in for k in ranks]), np.cumsum([0] + [k * d_out for k in ranks])
    A, B = g.normal(size=oA[-1]), g.normal(size=oB[-1])
    ids = np.array([[0, 2], [1, 1], [-1, 2], [-1, -1]])
    x, w, dy, base = g.normal(size=(4, d_in)), g.normal(size=(4, 2)), g.normal(size=(4, d_out)), g.normal(size=(4, d_out))
    f = lambda x_, w_: (dy * R.mixture(x_, base, ids, w_, ranks, oA, oB, A, B, 0.5, [1.0, 2.0, -3.0])[0]).sum()  # noqa: E731
    dx, _, dw, _ = R.mixture_grad(x, dy, ids, w, ranks, oA, oB, A, B, 0.5, [1.0, 2.0, -3.0])
    h = 1e-6
    for idx in np.ndindex(*x.shape):
        up, dn = x.copy(), x.copy()
        up[idx] += h
        dn[idx] -= h
        assert abs((f(up, w) - f(dn, w)) / (2 * h) - dx[idx]) <= 1e-6
    for idx in np.ndindex(*w.shape):
        up, dn = w.copy(), w.copy()
        up[idx] += h
        dn[idx] -= h
        assert abs((f(x, up) - f(x, dn)) / (2 * h) - dw[idx]) <= 1e-6


def test_w4_by_hand():
    W = np.zeros((2, 32))
    W[0, :4] = [7.0, -7.0, 3.5, 2.5]      # scale 1; halves go to even
    c, s, z = R.w4_quantize(W, 32, False)
    assert s[0, 0] == 1.0 and c[0, :5].tolist() == [15, 1, 12, 10, 8] and (c[1] == 8).all() and s[1, 0] == 0
    c, s, z = R.w4_quantize(np.abs(W) - 0.0, 32, True)
    assert z[0, 0] == 0 and c[0, 0] == 15
    q = R.w4_pack(c)
    assert (R.w4_unpack(q) == c).all()
    back = R.w4_matrix(q, s, z.astype(np.uint8), 32)
    assert np.abs(back[0] - np.abs(W[0])).max() <= s[0, 0] / 2 + 15 * s[0, 0] * 2.0 ** -8
