"""The oracle of the balance loss and the adapters: its gradients against
central differences of its forward in float64 (step h: the difference's own
error is O(h^2) of third derivatives of order 1, plus 2^-52 / h of rounding;
with h = 1e-5 both are below 1e-9 of the values' scale), and known values."""
import numpy as np
import pytest

import oracle

H = 1e-5
TOL = 1e-8


def diff(f, x):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + H
        up = f()
        x[i] = keep - H
        down = f()
        x[i] = keep
        g[i] = (up - down) / (2 * H)
    return g


def test_balance_uniform_is_one():
    ids = np.arange(12).reshape(6, 2) % 4
    got = oracle.balance(np.zeros((6, 4)), ids)
    np.testing.assert_array_equal(got["counts"], [[3, 3, 3, 3]])
    assert abs(got["loss"][0] - 1.0) < 1e-15


def test_balance_empty_and_masked():
    logits = np.zeros((5, 3))
    logits[2] = np.nan
    ids = np.zeros((5, 1), np.int64)
    got = oracle.balance(logits, ids, offsets=[0, 0, 5], valid=[1, 1, 0, 1, 0])
    assert got["tokens"].tolist() == [0, 3] and got["loss"][0] == 0
    assert abs(got["loss"][1] - 1.0) < 1e-15  # all three choose expert 0, whose probability is 1/3


@pytest.mark.parametrize("k", [1, 3])
def test_balance_gradient_against_differences(k):
    rng = np.random.default_rng(5)
    M, E = 11, 7
    logits = rng.standard_normal((M, E))
    ids = np.stack([rng.permutation(E)[:k] for _ in range(M)])
    off, valid = [0, 4, 4, 9], rng.random(M) > 0.2
    gl = rng.standard_normal(3)
    st = oracle.balance(logits, ids, off, valid)

    got = oracle.balance_backward(logits, k, st["counts"], st["tokens"], gl, off, valid)
    want = diff(lambda: float(gl @ oracle.balance(logits, ids, off, valid)["loss"]), logits)
    np.testing.assert_allclose(got[:9], want[:9], atol=TOL, rtol=0)
    assert np.isnan(got[9:]).all() and np.abs(want[9:]).max() == 0


def test_lora_gradients_against_differences():
    rng = np.random.default_rng(6)
    M, K, N, r, L = 7, 5, 4, 3, 3
    x, a, b = rng.standard_normal((M, K)), rng.standard_normal((L, r, K)), rng.standard_normal((L, N, r))
    ids, scales = np.array([0, 2, -1, 0, 3, 2, 2]), np.array([0.5, 1.0, -2.0])
    base, g = rng.standard_normal((M, N)), rng.standard_normal((M, N))
    _, h = oracle.lora_forward(x, ids, a, b, scales, base)
    dx, da, db = oracle.lora_backward(g, x, ids, h, a, b, scales, np.zeros((M, K)))

    def loss():
        return float((g * oracle.lora_forward(x, ids, a, b, scales, base)[0]).sum())

    for got, leaf in ((dx, x), (da, a), (db, b)):
        np.testing.assert_allclose(got, diff(loss, leaf), atol=TOL, rtol=0)
    assert np.abs(da[1]).max() == 0 and np.abs(dx[2]).max() == 0
