"""Pins of the gated delta rule's and the residual norm's oracle: special
cases that reduce to routines pinned elsewhere, worked values, and gradients
against central finite differences of the forward."""
import numpy as np
import pytest

import oracle


def _inputs(rng, B, n, Hk, H, dk, dv):
    q, k = rng.standard_normal((2, B, n, Hk, dk))
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    v = rng.standard_normal((B, n, H, dv))
    g = -rng.random((B, n, H))
    beta = rng.random((B, n, H))
    return q, k, v, g, beta


def test_orthogonal_keys_reduce_to_retention():
    """With orthonormal keys nothing is ever replaced: x = beta v, which is
    retention of (q, k, beta v) with a decay of one rate."""
    rng = np.random.default_rng(0)
    B, n, H, d = 2, 6, 3, 8
    q, _, v, _, beta = _inputs(rng, B, n, H, H, d, 5)
    k = np.broadcast_to(np.eye(d)[None, :n, None, :], (B, n, H, d))
    gam = np.array([0.5, 0.9, 1.0])
    g = np.broadcast_to(np.log(gam), (B, n, H))
    o, S = oracle.delta_recurrent(q, k, v, g, beta, 0.25)
    want, St = oracle.retention_recurrent(q, k, beta[..., None] * v, gam)
    np.testing.assert_allclose(o, 0.25 * want, atol=1e-12)
    np.testing.assert_allclose(S, St, atol=1e-12)


def test_full_strength_write_is_read_back():
    """beta = 1 and |k| = 1: the state answers k_t with v_t right after it."""
    rng = np.random.default_rng(1)
    q, k, v, g, beta = _inputs(rng, 1, 7, 2, 2, 4, 3)
    o, _ = oracle.delta_recurrent(k, k, v, g, np.ones_like(beta), 1.0)
    np.testing.assert_allclose(o, v, atol=1e-12)


def test_lengths_and_states_split_a_run():
    rng = np.random.default_rng(2)
    q, k, v, g, beta = _inputs(rng, 3, 9, 1, 2, 4, 3)
    o, S = oracle.delta_recurrent(q, k, v, g, beta, 1.0)
    cut = [0, 4, 9]
    o1, S1 = oracle.delta_recurrent(q, k, v, g, beta, 1.0, lengths=cut)
    for b, c in enumerate(cut):
        np.testing.assert_array_equal(o1[b, :c], o[b, :c])
        assert not o1[b, c:].any()
        rest = [x[b:b + 1, c:] for x in (q, k, v, g, beta)]
        o2, S2 = oracle.delta_recurrent(*rest, 1.0, state=S1[b:b + 1])
        np.testing.assert_allclose(o2[0], o[b, c:], atol=1e-12)
        np.testing.assert_allclose(S2[0], S[b], atol=1e-12)


@pytest.mark.parametrize("H,Hk,lengths", [(1, 1, None), (4, 2, [5, 3])])
def test_delta_gradients_against_differences(H, Hk, lengths):
    rng = np.random.default_rng(3)
    B, n, dk, dv, scale = 2, 5, 4, 3, 0.7
    args = list(_inputs(rng, B, n, Hk, H, dk, dv))
    do = rng.standard_normal((B, n, H, dv))

    def loss(a):
        return (oracle.delta_recurrent(*a, scale, lengths=lengths)[0] * do).sum()

    grads = oracle.delta_backward(*args, do, scale, lengths)
    for i, grad in enumerate(grads):
        for _ in range(3):
            way = rng.standard_normal(args[i].shape)
            step = 1e-5
            up, down = list(args), list(args)
            up[i], down[i] = args[i] + step * way, args[i] - step * way
            diff = (loss(up) - loss(down)) / (2 * step)
            # central differences: O(step^2) truncation, 1e-16 / step rounding
            assert abs(diff - (grad * way).sum()) < 1e-7 * max(1.0, abs(diff)), i


def test_residual_norm_by_hand():
    # rms of (3, 4, 0, 0) is (1.2, 1.6, 0, 0) at eps = 0; h = (1, 1, 1, 1) + 0.5 * that * post
    x, y = np.ones(4), np.array([3.0, 4.0, 0.0, 0.0])
    h, n = oracle.residual_norm(x, y, post=np.array([1.0, 2.0, 1.0, 1.0]), scale=0.5, eps=0.0)
    np.testing.assert_allclose(h, [1.6, 2.6, 1.0, 1.0])
    np.testing.assert_allclose(n, h / np.sqrt((1.6 ** 2 + 2.6 ** 2 + 2) / 4))
    h, _ = oracle.residual_norm(x, y, gate=np.zeros(4), post_norm=False)
    np.testing.assert_array_equal(h, x)                       # swish(0) = 0


@pytest.mark.parametrize("gated,post_norm", [(True, True), (False, True), (True, False)])
def test_residual_norm_gradients_against_differences(gated, post_norm):
    rng = np.random.default_rng(4)
    rows, hidden = 3, 6
    x, y, gate, dn, dh = rng.standard_normal((5, rows, hidden))
    post, pre = 1 + 0.3 * rng.standard_normal((2, hidden))
    kw = dict(post_norm=post_norm, scale=0.6, eps=1e-3)
    args = [x, y, gate if gated else None, post if post_norm else None, pre]

    def loss(a):
        h, n = oracle.residual_norm(a[0], a[1], a[2], post=a[3], pre=a[4], **kw)
        return (h * dh).sum() + (n * dn).sum()

    grads = oracle.residual_norm_backward(x, y, dn, dh, args[2], post=args[3], pre=pre, **kw)
    for i, grad in enumerate(grads):
        if args[i] is None:
            continue
        way = rng.standard_normal(args[i].shape)
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + 1e-5 * way, args[i] - 1e-5 * way
        diff = (loss(up) - loss(down)) / 2e-5
        assert abs(diff - (grad * way).sum()) < 1e-7 * max(1.0, abs(diff)), i
