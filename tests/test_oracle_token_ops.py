"""Pins of the token operators' oracle: rotary positions against complex
multiplication and worked values, decayed linear attention against the sum it
stands for and its gradients against differences."""

import math

import numpy as np
import pytest

from oracle import token_ops as tok


def test_plain_frequencies_are_a_geometric_row_per_axis():
    w, amp = tok.rotary_frequencies([4, 2], base=10000.0)
    np.testing.assert_allclose(w, [1, 0.1, 0.01, 0.001, 1, 0.01], rtol=1e-14)
    assert amp == 1.0


def test_scalings_at_their_ends():
    P, f = 64, 8.0
    plain, _ = tok.rotary_frequencies([P])
    linear, _ = tok.rotary_frequencies([P], scaling="linear", factor=f)
    np.testing.assert_allclose(linear, plain / f)
    ntk, _ = tok.rotary_frequencies([P], scaling="ntk", factor=f)
    np.testing.assert_allclose([ntk[0], ntk[-1]], [plain[0], plain[-1] / f], rtol=1e-13)
    yarn, amp = tok.rotary_frequencies([P], scaling="yarn", factor=f, trained_length=4096.0)
    turns = 4096 * plain / (2 * math.pi)
    np.testing.assert_allclose(yarn[turns > 64], plain[turns > 64])
    np.testing.assert_allclose(yarn[turns < 0.5], plain[turns < 0.5] / f)
    assert (np.diff(yarn) < 0).all() and amp == pytest.approx(0.1 * math.log(8) + 1)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotation_is_complex_multiplication(layout):
    r = np.random.default_rng(0)
    x = r.standard_normal((2, 3, 5, 16))
    w, amp = tok.rotary_frequencies([6], scaling="yarn", factor=4.0, trained_length=64.0)
    pos = r.integers(0, 1000, (2, 1, 5))
    y = tok.rotate(x, pos, [6], w, amp, layout)
    a, b = (x[..., :6], x[..., 6:12]) if layout == "half" else (x[..., 0:12:2], x[..., 1:12:2])
    z = (a + 1j * b) * amp * np.exp(1j * pos[:, 0, None, :, None] * w)
    got = (y[..., :6], y[..., 6:12]) if layout == "half" else (y[..., 0:12:2], y[..., 1:12:2])
    np.testing.assert_allclose(got[0], z.real, atol=1e-12)
    np.testing.assert_allclose(got[1], z.imag, atol=1e-12)
    np.testing.assert_array_equal(y[..., 12:], x[..., 12:])
    # the inverse is the transpose
    u = r.standard_normal(x.shape)
    back = tok.rotate(u, pos, [6], w, amp, layout, inverse=True)
    assert np.sum(u * y) == pytest.approx(np.sum(back * x), rel=1e-12)


def test_grid_positions():
    p = tok.grid_positions((2, 2, 3), origin=(5, 0, 1))
    assert p[:, 0].tolist() == [5, 0, 1] and p[:, 11].tolist() == [6, 1, 3] and p[:, 4].tolist() == [5, 1, 2]


def _case(seed, B=2, H=2, N=7, d=4):
    r = np.random.default_rng(seed)
    t = [r.standard_normal((B, H, N, d)) for _ in range(4)]
    return t, np.log(np.array([0.9, 0.4])), r.standard_normal((B, H, d, d)), r.standard_normal((B, H, d, d)), np.array([7, 4])


def test_decay_forward_is_the_masked_sum():
    (q, k, v, _), g, s0, _, lens = _case(1)
    out, S = tok.decay_forward(q, k, v, g, lens, s0, scale=0.7)
    for b in range(2):
        for h in range(2):
            n, f = lens[b], math.exp(g[h])
            for t in range(7):
                want = np.zeros(4)
                if t < n:
                    want = sum(f ** (t - s) * (q[b, h, t] @ k[b, h, s]) * v[b, h, s] for s in range(t + 1))
                    want = 0.7 * (want + f ** (t + 1) * q[b, h, t] @ s0[b, h])
                np.testing.assert_allclose(out[b, h, t], want, atol=1e-12)
            end = f ** n * s0[b, h] + sum(f ** (n - 1 - s) * np.outer(k[b, h, s], v[b, h, s]) for s in range(n))
            np.testing.assert_allclose(S[b, h], end, atol=1e-12)


def test_decay_of_zero_keeps_only_the_token_itself():
    (q, k, v, _), _, s0, _, _ = _case(2)
    out, S = tok.decay_forward(q, k, v, np.array([-np.inf, -np.inf]), None, s0, scale=1.0)
    np.testing.assert_allclose(out, np.sum(q * k, -1, keepdims=True) * v, atol=1e-12)
    np.testing.assert_allclose(S, k[:, :, -1, :, None] * v[:, :, -1, None, :])


def test_decay_backward_against_differences():
    (q, k, v, do), g, s0, ds, lens = _case(3)
    grads = tok.decay_backward(q, k, v, g, do, lens, s0, ds, scale=0.7)

    def loss(q, k, v, s0):
        out, S = tok.decay_forward(q, k, v, g, lens, s0, scale=0.7)
        return np.sum(out * do) + np.sum(S * ds)

    r = np.random.default_rng(4)
    args = [q, k, v, s0]
    for i, gr in enumerate(grads):
        x = r.standard_normal(args[i].shape)
        e = 1e-5
        up, dn = list(args), list(args)
        up[i], dn[i] = args[i] + e * x, args[i] - e * x
        # the loss is a polynomial of low degree in each argument: the central
        # difference is off by e^2 and by rounding over e
        assert (loss(*up) - loss(*dn)) / (2 * e) == pytest.approx(np.sum(gr * x), rel=1e-7, abs=1e-7)
    for gr in grads[:3]:
        assert (gr[1, :, 4:] == 0).all()
