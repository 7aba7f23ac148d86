"""The attention's and the projection's fp64 oracle against things other than itself."""
import numpy as np
import pytest

from oracle import attention_oracle as ao


def _draw(seed, *shapes):
    rng = np.random.default_rng(seed)
    return [rng.standard_normal(s) for s in shapes]


def test_mask_by_hand():
    m = ao.seen(6, window=2, prefix=1)
    assert m.astype(int).tolist() == [[1, 0, 0, 0, 0, 0], [1, 1, 0, 0, 0, 0], [1, 1, 1, 0, 0, 0], [1, 0, 1, 1, 0, 0],
                                      [1, 0, 0, 1, 1, 0], [1, 0, 0, 0, 1, 1]]
    assert (ao.seen(5) == np.tril(np.ones((5, 5), bool))).all()
    assert (ao.seen(5, 1) == np.eye(5, dtype=bool)).all()


def test_special_cases():
    q, k, v = _draw(1, (4, 7, 5), (2, 7, 5), (2, 7, 3))
    out, lse = ao.attention(q, k, v, 0.3, window=1)          # itself alone
    assert np.allclose(out, np.repeat(v, 2, 0)) and np.allclose(lse, 0.3 * (q * np.repeat(k, 2, 0)).sum(-1))
    out, lse = ao.attention(q, k * 0, v, 0.3)                # equal scores: the mean so far
    mean = np.repeat(v.cumsum(1) / np.arange(1, 8)[:, None], 2, 0)
    assert np.allclose(out, mean) and np.allclose(lse, np.log(np.arange(1, 8)))
    full = ao.attention(q, k, v, 0.3)[0]
    assert np.allclose(full, ao.attention(q, k, v, 0.3, window=7)[0])
    assert np.allclose(full, ao.attention(q, k, v, 0.3, window=2, prefix=7)[0])


@pytest.mark.parametrize("window,prefix", [(0, 0), (3, 0), (2, 2)])
def test_steps_are_the_rows_of_the_prompt(window, prefix):
    q, k, v = _draw(2, (4, 9, 6), (2, 9, 6), (2, 9, 6))
    out = ao.attention(q, k, v, 0.4, window, prefix)[0]
    for n in range(1, 10):
        got = ao.attention_step(q[:, n - 1:n], k[:, :n], v[:, :n], 0.4, window, prefix)
        assert np.allclose(got, out[:, n - 1:n])
    assert np.allclose(ao.attention_step(q[:, 5:], k, v, 0.4, window, prefix), out[:, 5:])
    z = ao.attention_step(q[:, :3], k[:, :2], v[:, :2], 0.4, window, prefix)
    assert (z[:, 0] == 0).all() and np.allclose(z[:, 1:], ao.attention(q[:, 1:3], k[:, :2], v[:, :2], 0.4, window, prefix)[0])
    assert (ao.attention_step(q[:, :2], k[:, :0], v[:, :0], 0.4) == 0).all()


@pytest.mark.parametrize("window,prefix", [(0, 0), (2, 1)])
def test_gradient_against_differences(window, prefix):
    x = _draw(3, (4, 5, 3), (2, 5, 3), (2, 5, 3))
    (do,) = _draw(4, (4, 5, 3))
    got = ao.attention_backward(*x, do, 0.6, window, prefix)
    f = lambda: (ao.attention(*x, 0.6, window, prefix)[0] * do).sum()  # noqa: E731
    for t, g in zip(x, got):
        for at in np.ndindex(t.shape):
            keep, eps = t[at], 1e-5
            t[at] = keep + eps
            hi = f()
            t[at] = keep - eps
            lo = f()
            t[at] = keep
            assert abs((hi - lo) / (2 * eps) - g[at]) < 1e-8


@pytest.mark.parametrize("activation", [False, True])
def test_projection_and_its_gradient(activation):
    x, w, b, r, do = _draw(5, (4, 3), (5, 3), (5,), (4, 5), (4, 5))
    out, z = ao.projection(x, w, b, r, activation)
    for m in range(4):
        for o in range(5):
            t = sum(x[m, i] * w[o, i] for i in range(3)) + b[o]
            assert abs(t - z[m, o]) < 1e-13
            assert abs((t / (1 + np.exp(-t)) if activation else t) + r[m, o] - out[m, o]) < 1e-13
    got = ao.projection_backward(x, w, do, z if activation else None)
    f = lambda: (ao.projection(x, w, b, r, activation)[0] * do).sum()  # noqa: E731
    for t, g in zip((x, w, b), got):
        for at in np.ndindex(t.shape):
            keep, eps = t[at], 1e-5
            t[at] = keep + eps
            hi = f()
            t[at] = keep - eps
            lo = f()
            t[at] = keep
            assert abs((hi - lo) / (2 * eps) - g[at]) < 1e-8
