"""Pins of the attention oracle (oracle/attention.py) to facts that do not
depend on its code."""
import numpy as np
import pytest

from oracle import attention as oa


def test_rotation_keeps_pair_norms_and_depends_on_distance_only():
    """A rotation keeps every pair's length, and q(p).k(s) depends on p - s."""
    r = np.random.RandomState(0)
    f = 10000.0 ** (-np.arange(16) / 16)
    q, k = r.randn(1, 1, 1, 32), r.randn(1, 1, 1, 32)
    for inter in (False, True):
        def at(x, p):
            return oa.qk_norm_rope(x, np.array([[p]]), inv_freq=f, interleaved=inter)[0][0, 0, 0]
        y = at(q, 1234)
        pairs = (lambda z: z.reshape(16, 2)) if inter else (lambda z: z.reshape(2, 16).T)
        np.testing.assert_allclose((pairs(y) ** 2).sum(1), (pairs(q[0, 0, 0]) ** 2).sum(1), rtol=1e-12)
        np.testing.assert_allclose(at(q, 70) @ at(k, 61), at(q, 9) @ at(k, 0), rtol=1e-11)
    np.testing.assert_allclose(at(q, 0), q[0, 0, 0], rtol=1e-14)


def test_rotation_of_a_right_angle_and_norm_of_a_constant():
    x = np.zeros((1, 1, 1, 32))
    x[..., 0], x[..., 16] = 3.0, 4.0
    y = oa.qk_norm_rope(x, np.array([[1]]), inv_freq=np.full(16, np.pi / 2))[0][0, 0, 0]
    np.testing.assert_allclose([y[0], y[16]], [-4.0, 3.0], atol=1e-12)
    z = oa.qk_norm_rope(np.full((1, 1, 1, 32), -7.0), np.array([[0]]), weight=np.arange(32.0), eps=0.0)[0]
    np.testing.assert_allclose(z[0, 0, 0], -np.arange(32.0))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 2), (3, 0), (3, 2), (3, 9), (100, 0), (100, 5)])
def test_uniform_scores_average_the_seen_values(window, sinks):
    """With zero keys all seen keys weigh the same: outputs count them."""
    T = 12
    v = np.eye(T)[None, None]
    o = oa.window(np.ones((1, 1, T, T)), np.zeros((1, 1, T, T)), v, window, sinks, 1.0)[0][0, 0]
    for i in range(T):
        seen = [j for j in range(T) if oa.sees(i, j, T, window, sinks)]
        want = np.zeros(T)
        want[seen] = 1.0 / len(seen)
        np.testing.assert_allclose(o[i], want, atol=1e-15)
    assert oa.sees(0, 0, 1, 1, 0) and not oa.sees(0, 1, 5, 9, 9)


def test_one_key_returns_its_value_and_empty_rows_are_zero():
    r = np.random.RandomState(1)
    q, k, v = r.randn(1, 2, 3, 8), r.randn(1, 1, 2, 8), r.randn(1, 1, 2, 8)
    o, size, _, written = oa.window(q, k, v, 9, 0, 0.3, q_len=[3], k_len=[2])
    assert written.all() and (o[0, :, 0] == 0).all()      # position -1
    np.testing.assert_allclose(o[0, :, 1], np.stack([v[0, 0, 0]] * 2))
    np.testing.assert_allclose(size[0, :, 1], np.abs(o[0, :, 1]))


def test_step_is_the_last_row_of_the_window_form():
    r = np.random.RandomState(2)
    L, page, d = 37, 16, 8
    k, v, q = r.randn(1, 2, L, d), r.randn(1, 2, L, d), r.randn(1, 4, L, d)
    table = np.array([[2, 0, 3]])
    kc, vc = np.full((4, 2, page, d), np.nan), np.full((4, 2, page, d), np.nan)
    for j in range(L):
        kc[table[0, j // page], :, j % page], vc[table[0, j // page], :, j % page] = k[0, :, j], v[0, :, j]
    for window, sinks in ((5, 0), (5, 3), (100, 0)):
        a = oa.window(q, k, v, window, sinks, 0.4)[0][:, :, -1]
        b = oa.step(q[:, :, -1], kc, vc, table, [L], window, sinks, 0.4)[0]
        np.testing.assert_allclose(a, b, rtol=1e-13)
