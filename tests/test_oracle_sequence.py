"""The sequence operators' float64 definitions: hand-worked values, and every
gradient formula against central differences of its forward."""
import numpy as np
import pytest

from oracle import sequence_oracle as so


def differences(f, a, eps=1e-6):
    g = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        up, dn = a.copy(), a.copy()
        up[i] += eps
        dn[i] -= eps
        g[i] = (f(up) - f(dn)) / (2 * eps)
    return g


# central differences of O(1) functions: eps^2 f'''/6 ~ 1e-12 and rounding
# 1e-16 * |f| / eps ~ 1e-9 for |f| ~ 10
TOL = 1e-7


def test_embed_by_hand():
    t = np.array([[1.0, 2.0], [3.0, 4.0]])
    out = so.embed(t, np.array([1, -1, 0, 2]), 2.0)
    assert np.array_equal(out[:3], [[6, 8], [0, 0], [2, 4]]) and np.isnan(out[3]).all()


def test_embed_grad_matches_differences():
    rng = np.random.default_rng(0)
    ids = np.array([[0, 2, 2], [-1, 4, 5]])
    d = rng.standard_normal((2, 3, 3))
    t = rng.standard_normal((5, 3))

    def f(table):
        return np.nansum(so.embed(table, ids, 1.5) * d)
    assert np.abs(differences(f, t) - so.embed_grad(d, ids, 5, 1.5)).max() < TOL


def test_scan_by_hand():
    x = np.array([[[1.0], [5.0], [7.0]]])
    g = np.array([[[0.0], [-np.inf], [np.inf]]])
    h, last, before = so.gated_scan(x, g, np.array([[3.0]]))
    assert np.allclose(h[0, :, 0], [2.0, 5.0, 5.0]) and last[0, 0] == 5.0
    h, last, _ = so.gated_scan(x, g, np.array([[3.0]]), lengths=np.array([0]))
    assert not h.any() and last[0, 0] == 3.0


@pytest.mark.parametrize("lengths", [None, [5, 0, 3]])
def test_scan_grad_matches_differences(lengths):
    rng = np.random.default_rng(1)
    x, g, dh = (rng.standard_normal((3, 5, 2)) for _ in range(3))
    h0, dl = rng.standard_normal((3, 2)), rng.standard_normal((3, 2))

    def f(x=x, g=g, h0=h0):
        h, last, _ = so.gated_scan(x, g, h0, lengths)
        return (h * dh).sum() + (last * dl).sum()
    dx, dg, dh0 = so.gated_scan_grad(x, g, dh, dl, h0, lengths)
    assert np.abs(differences(lambda v: f(x=v), x) - dx).max() < TOL
    assert np.abs(differences(lambda v: f(g=v), g) - dg).max() < TOL
    assert np.abs(differences(lambda v: f(h0=v), h0) - dh0).max() < TOL


def test_logprobs_by_hand():
    z = np.array([[0.0, np.log(3.0), -np.inf], [-np.inf] * 3, [1.0, 1.0, 1.0]])
    logp, h, lse, tlp, ids = so.token_logprobs(z, np.array([1, 0, -1]), 3, 1.0)
    assert np.allclose(logp[0], np.log(0.75)) and logp[1] == -np.inf and logp[2] == 0.0
    assert np.allclose(h, [-(0.25 * np.log(0.25) + 0.75 * np.log(0.75)), 0.0, np.log(3.0)])
    assert np.array_equal(ids, [[1, 0, -1], [-1, -1, -1], [0, 1, 2]])


def test_logprobs_grad_matches_differences():
    rng = np.random.default_rng(2)
    z = rng.standard_normal((4, 6))
    tok = np.array([3, -1, 0, 5])
    w, q = rng.standard_normal(4), rng.standard_normal(4)

    def f(z):
        logp, h, *_ = so.token_logprobs(z, tok, 0, 0.7)
        return (w * logp).sum() + (q * h).sum()
    assert np.abs(differences(f, z) - so.token_logprobs_grad(z, tok, w, q, 0.7)).max() < TOL


def test_log_softmax_of_rows_of_the_lowest_value():
    """Every column alike, however far from zero the row lies."""
    for low in (np.finfo(np.float32).min, -65504.0, 0.0, 3e38):
        lp, lse, h = so.log_softmax(np.full((2, 5), low), 1.0)
        assert np.allclose(lp, -np.log(5), rtol=1e-12) and np.allclose(h, np.log(5), rtol=1e-12)
