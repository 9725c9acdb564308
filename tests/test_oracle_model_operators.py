"""The oracle of routing by scores, the norm and the 8-bit values: gradients
against central differences of the forward in float64 (the difference's own
error as in test_oracle_operators), and known values."""
import itertools

import numpy as np
import pytest

import oracle
from test_oracle_operators import TOL, diff


def test_route_scored_is_route_for_the_kept_softmax():
    rng = np.random.default_rng(1)
    logits = rng.standard_normal((40, 24)).astype(np.float32)
    logits[3] = 0.0
    ids, w = oracle.route(logits, 5)
    got_ids, got_w = oracle.route_scored(logits, 5)
    np.testing.assert_array_equal(got_ids, ids)
    np.testing.assert_allclose(got_w, w, atol=1e-12)


def test_route_scored_by_hand():
    # sigmoid(0) = 0.5; groups {0, 1}, {2, 3}, {4, 5}
    logits = np.array([[0.0, 0.0, 2.0, -9.0, 1.0, 1.0]])
    s = 1 / (1 + np.exp(-logits[0]))
    ids, w = oracle.route_scored(logits, 2, "sigmoid", n_groups=3, top_groups=1, group_top=1, renormalise=False)
    assert ids.tolist() == [[2, 3]]  # the group of the highest score, whatever else is in it
    np.testing.assert_allclose(w[0], s[[2, 3]])
    ids, _ = oracle.route_scored(logits, 2, "sigmoid", n_groups=3, top_groups=1, group_top=2)
    assert ids.tolist() == [[4, 5]]  # by the sum of two; equal logits in order
    bias = np.array([0.0, 1.0, 0, 0, 0, 0])
    ids, w = oracle.route_scored(logits, 2, "sigmoid", bias=bias, scale=3.0)
    assert ids.tolist() == [[1, 2]]
    np.testing.assert_allclose(w[0], 3.0 * s[[1, 2]] / (s[1] + s[2]), rtol=1e-12)  # the bias is not in the weights


def test_route_scored_absent_and_nan():
    x = np.array([[1.0, -np.inf, 3.0, -np.inf], [-np.inf] * 4, [0.0, np.nan, 5.0, 1.0]])
    ids, w = oracle.route_scored(x, 3, "sigmoid")
    assert ids.tolist() == [[2, 0, -1], [-1, -1, -1], [1, 2, 3]]
    assert w[0, 2] == 0 and not w[1].any() and np.isnan(w[2]).all()
    ids, _ = oracle.route_scored(x, 2, "softmax", n_groups=2, top_groups=1, group_top=2)
    assert ids[0].tolist() == [2, -1] and ids[1].tolist() == [-1, -1]
    assert oracle.route_scored(x, 2, valid=[0, 0, 1])[0].tolist()[0] == [-1, -1]


def test_align_dropped_is_align_without_drops():
    ids = np.random.default_rng(2).integers(0, 9, (30, 3))
    al = oracle.align(ids, 9, 16)
    rows, blocks, off = oracle.align_dropped(ids, 9, 16)
    np.testing.assert_array_equal(rows, al["sorted_token_ids"])
    np.testing.assert_array_equal(blocks, al["block_expert_ids"])
    np.testing.assert_array_equal(off, al["expert_offsets"])


@pytest.mark.parametrize("scoring,renormalise", itertools.product(("softmax", "sigmoid"), (True, False)))
def test_route_scored_gradient(scoring, renormalise):
    rng = np.random.default_rng(3)
    logits = rng.standard_normal((3, 7))
    ids, _ = oracle.route_scored(logits, 3, scoring)
    ids[1, 2], ids[2] = -1, -1
    g = rng.standard_normal((3, 3))

    def loss():
        total = 0.0
        for t in range(3):
            at = [j for j in range(3) if ids[t, j] >= 0]
            if at:
                e = ids[t, at]
                s = oracle.scores(logits[t], scoring)[e]
                s = s / s.sum() if renormalise else s
                total += 2.5 * float(g[t, at] @ s)
        return total

    got, mag = oracle.route_scored_backward(logits, ids, g, scoring, renormalise, 2.5)
    np.testing.assert_allclose(got, diff(loss, logits), atol=TOL)
    assert (np.abs(got) <= mag * (1 + 1e-12)).all() and not got[2].any()


def test_norm_gradient():
    rng = np.random.default_rng(4)
    h, w, g, d = rng.standard_normal((3, 6)), rng.standard_normal(6), rng.standard_normal((3, 6)), rng.standard_normal((3, 6))
    loss = lambda: float((oracle.rms_norm(h, w, 1e-3)[0] * g).sum() + (h * d).sum())  # noqa: E731
    dh, dw, mag, wmag = oracle.rms_norm_backward(g, h, oracle.rms_norm(h, w, 1e-3)[1], w, d)
    np.testing.assert_allclose(dh, diff(loss, h), atol=TOL)
    np.testing.assert_allclose(dw, diff(loss, w), atol=TOL)
    assert (np.abs(dh) <= mag * (1 + 1e-12)).all() and (np.abs(dw) <= wmag * (1 + 1e-12)).all()


def test_e4m3_by_enumeration():
    """Every finite code keeps its value, the middle between two goes to the even one, the rest to the nearer."""
    values = []
    for code in range(0x7f):
        e, m = code >> 3, code & 7
        values.append((m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    values = np.array(values)
    assert values[-1] == 448 and (np.diff(values) > 0).all()
    np.testing.assert_array_equal(oracle.e4m3(values), values)
    np.testing.assert_array_equal(oracle.e4m3(-values), -values)
    middle = (values[:-1] + values[1:]) / 2
    even = values[np.arange(len(middle)) + (np.arange(len(middle)) % 2)]
    np.testing.assert_array_equal(oracle.e4m3(middle), even)
    np.testing.assert_array_equal(oracle.e4m3(np.nextafter(middle, 0)), values[:-1])
    np.testing.assert_array_equal(oracle.e4m3(np.nextafter(middle, 1e9)), values[1:])
    assert oracle.e4m3(1e9) == 448


def test_quantise_scales():
    y = np.zeros((2, 64))
    y[0, :32] = np.linspace(-3, 7, 32)
    q, s = oracle.quantise(y, 32)
    assert s.dtype == np.float32 and s[0, 0] == np.float32(7 / 448) and s[0, 1] == np.float32(2.0 ** -126)
    assert q[0, 31] == 448 and not q[1].any()
