"""The layer oracle: gradients against differences, the step against the sequence,
turns against complex numbers, AdamW by hand."""
import numpy as np
import pytest

from oracle import layers_oracle as lo


@pytest.mark.parametrize("lengths", [None, [5, 0, 3]])
@pytest.mark.parametrize("G", [4, 2, 1])
def test_attention_gradient_against_differences(lengths, G):
    rng = np.random.default_rng(G)
    B, T, H, dk, dv, scale = 3, 5, 4, 3, 2, 0.7
    x = {"q": rng.standard_normal((B, T, H, dk)), "k": rng.standard_normal((B, T, G, dk)),
         "v": rng.standard_normal((B, T, G, dv)), "state": rng.standard_normal((B, H, dk, dv))}
    decay = -rng.random(H)
    do, dlast = rng.standard_normal((B, T, H, dv)), rng.standard_normal((B, H, dk, dv))

    def loss(x):
        o, last = lo.linear_attention(x["q"], x["k"], x["v"], decay, x["state"], lengths, scale)
        return (o * do).sum() + (last * dlast).sum()

    got = dict(zip(("q", "k", "v", "state"), lo.linear_attention_grad(
        x["q"], x["k"], x["v"], decay, do, dlast, x["state"], lengths, scale)))
    h = 1e-3  # the loss is a quadratic in each input along a line: central differences are exact
    for name in x:
        d = rng.standard_normal(x[name].shape)
        hi, lo_ = dict(x), dict(x)
        hi[name], lo_[name] = x[name] + h * d, x[name] - h * d
        assert abs((loss(hi) - loss(lo_)) / (2 * h) - (got[name] * d).sum()) < 1e-9 * 1e3


def test_attention_by_hand_and_in_parts():
    q = np.array([2.0, 3.0]).reshape(1, 2, 1, 1)
    k, v = np.array([1.0, 5.0]).reshape(1, 2, 1, 1), np.array([7.0, 11.0]).reshape(1, 2, 1, 1)
    o, S = lo.linear_attention(q, k, v, [np.log(0.5)], scale=10.0)
    assert np.allclose(o.ravel(), [10 * 2 * 7, 10 * 3 * (3.5 + 55)]) and np.allclose(S, 58.5)
    rng = np.random.default_rng(0)
    q, k, v = (rng.standard_normal((2, 9, 2, 3)) for _ in range(3))
    o, S = lo.linear_attention(q, k, v, [-0.1, -0.5])
    o1, S1 = lo.linear_attention(q[:, :4], k[:, :4], v[:, :4], [-0.1, -0.5])
    o2, S2 = lo.linear_attention(q[:, 4:], k[:, 4:], v[:, 4:], [-0.1, -0.5], S1)
    assert np.allclose(o, np.concatenate([o1, o2], 1)) and np.allclose(S, S2)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_against_complex_numbers(interleaved):
    rng = np.random.default_rng(1)
    x, pos, f = rng.standard_normal((6, 2, 10)), np.arange(-2, 4), np.array([1.0, 0.3, 0.01])
    got = lo.rotary(x, pos, f, interleaved, 1.5)
    one, two = (x[..., 0:6:2], x[..., 1:6:2]) if interleaved else (x[..., 0:3], x[..., 3:6])
    w = (one + 1j * two) * 1.5 * np.exp(1j * pos[:, None, None] * f)
    want = np.empty((6, 2, 6))
    if interleaved:
        want[..., 0::2], want[..., 1::2] = w.real, w.imag
    else:
        want[..., :3], want[..., 3:] = w.real, w.imag
    assert np.allclose(got[..., :6], want) and np.array_equal(got[..., 6:], x[..., 6:])
    back = lo.rotary(got, pos, f, interleaved, 1 / 1.5, inverse=True)
    assert np.allclose(back, x)


def test_adamw_by_hand():
    p, m, v = lo.adamw([1.0, 2.0], [0.5, 0.0], [0.0, 0.0], [0.0, 0.0], 1, 0.1, 0.9, 0.99, 0.0, 0.2)
    assert np.allclose(m, [0.05, 0]) and np.allclose(v, [0.0025, 0])
    assert np.allclose(p[0], 0.98 - 0.1) and np.isnan(p[1])  # 0 / 0 without eps
    p, m, v = lo.adamw(1.0, 0.3, 0.2, 0.04, 3, 0.01, 0.5, 0.5, 1e-8, 0.0)
    assert np.allclose(m, 0.25) and np.allclose(v, 0.065)
    assert np.allclose(p, 1 - 0.01 * (0.25 / 0.875) / np.sqrt(0.065 / 0.875))
