"""Pins of the gated delta rule's and the layer norms' oracle: closed forms,
and gradients against central differences in fp64."""
import numpy as np
import pytest

from oracle import delta


def _inputs(seed, T=7, hk=2, hv=4, dk=8, dv=8):
    r = np.random.default_rng(seed)
    k = r.standard_normal((T, hk, dk))
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    return (r.standard_normal((T, hk, dk)), k, r.standard_normal((T, hv, dv)), -r.uniform(0, 1, (T, hv)),
            r.uniform(0, 1, (T, hv)), 0.5, r.standard_normal((hv, dk, dv)))


def test_no_decay_and_full_strength_stores_the_last_value_of_a_key():
    """beta = 1, g = 0 and a unit key: after the write S^T k = v (the delta
    rule replaces what the key held)."""
    q, k, v, g, beta, scale, S = _inputs(0)
    o, last = delta.sequence(k, k, v, 0 * g, 0 * beta + 1, 1.0, S)
    np.testing.assert_allclose(o, v, atol=1e-12)


def test_zero_strength_only_decays():
    q, k, v, g, beta, scale, S = _inputs(1)
    o, last = delta.sequence(q, k, v, g, 0 * beta, scale, S)
    np.testing.assert_allclose(last, np.exp(g.sum(0))[:, None, None] * S, rtol=1e-12)


def test_orthogonal_keys_are_linear_attention():
    q, k, v, g, beta, scale, S = _inputs(2, T=8)
    k = np.repeat(np.eye(8)[:, None], 2, axis=1)
    o, last = delta.sequence(q, k, v, 0 * g, beta, scale, 0 * S)
    kk = np.repeat(k, 2, axis=1)
    np.testing.assert_allclose(last, np.einsum("thk,th,thv->hkv", kk, beta, v), atol=1e-12)


def test_two_halves_are_the_whole():
    q, k, v, g, beta, scale, S = _inputs(3)
    o, last = delta.sequence(q, k, v, g, beta, scale, S)
    o1, mid = delta.sequence(q[:3], k[:3], v[:3], g[:3], beta[:3], scale, S)
    o2, last2 = delta.sequence(q[3:], k[3:], v[3:], g[3:], beta[3:], scale, mid)
    np.testing.assert_allclose(np.concatenate([o1, o2]), o, rtol=1e-13)
    np.testing.assert_allclose(last2, last, rtol=1e-13)


@pytest.mark.parametrize("which", ["q", "k", "v", "g", "beta", "initial_state"])
def test_gradients_are_the_differences(which):
    names = ["q", "k", "v", "g", "beta", "scale", "initial_state"]
    args = list(_inputs(4))
    r = np.random.default_rng(5)
    do, ds = r.standard_normal(args[2].shape), r.standard_normal(args[6].shape)
    grad = delta.sequence(*args, do=do, dstate=ds)[2][which]
    i = names.index(which)
    d = r.standard_normal(args[i].shape)

    def loss(h):
        a = list(args)
        a[i] = a[i] + h * d
        o, last = delta.sequence(*a)
        return (o * do).sum() + (last * ds).sum()

    h = 1e-5   # the error of a central difference is of order h^2 = 1e-10 times third derivatives, and 1e-16 / h
    diff = (loss(h) - loss(-h)) / (2 * h)
    assert abs(diff - (grad * d).sum()) < 1e-6 * max(1.0, abs(diff))


def test_layer_norm_gradients_are_the_differences():
    r = np.random.default_rng(6)
    x, dz, gamma, eps = r.standard_normal((5, 9)) + 2, r.standard_normal((5, 9)), r.standard_normal(9), 1e-5
    _, _, _, dx, dg, _ = delta.layer_norm_backward(dz, x, gamma, eps)
    d, dgam = r.standard_normal(x.shape), r.standard_normal(9)
    loss = lambda h: (delta.layer_norm_backward(dz, x + h * d, gamma + h * dgam, eps)[0] * dz).sum()  # noqa: E731
    h = 1e-5
    diff = (loss(h) - loss(-h)) / (2 * h)
    assert abs(diff - (dx * d).sum() - (dg * dgam).sum()) < 1e-6 * max(1.0, abs(diff))
