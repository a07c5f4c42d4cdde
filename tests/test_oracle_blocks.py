"""The float64 oracles of the norms and the recurrence pinned: gradients against
differences, known values, and the recurrence against its own other forms."""
import numpy as np
import pytest

from oracle import norm as N
from oracle import recur as R

H = 1e-6


def _differences(f, arrays):
    """df / d(each array) by central differences of the scalar f()."""
    out = []
    for a in arrays:
        g = np.zeros_like(a)
        for i in np.ndindex(a.shape):
            old = a[i]
            a[i] = old + H
            p = f()
            a[i] = old - H
            q = f()
            a[i] = old
            g[i] = (p - q) / (2 * H)
        out.append(g)
    return out


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("gate", ["none", "scalar", "vector", "token"])
@pytest.mark.parametrize("pre,post,scale", [(True, True, "vector"), (True, False, "scalar"), (False, True, "none")])
def test_join_gradients(kind, gate, pre, post, scale):
    r = np.random.default_rng(3)
    T, D, eps = 3, 5, 1e-3
    n = r.standard_normal
    v = {"R": n((T, D)), "B": n((T, D)), "post_w": n(D) if post else None, "post_b": n(D) if post else None,
         "gate": {"none": None, "scalar": n(1), "vector": n(D), "token": n((T, D))}[gate],
         "scale": {"none": None, "scalar": n(1), "vector": n(D)}[scale], "w": n(D) if pre else None, "b": n(D) if pre else None}
    dX, d1 = n((T, D)), n((T, D))

    def f():
        R1, X = N.join(v["R"], v["B"], kind, eps, post, v["post_w"], v["post_b"], v["gate"], gate == "token", v["scale"],
                       v["w"], v["b"])
        return (R1 * d1).sum() + ((X * dX).sum() if pre else 0.0)

    R1, _ = N.join(v["R"], v["B"], kind, eps, post, v["post_w"], v["post_b"], v["gate"], gate == "token", v["scale"])
    g = N.join_backward(v["R"], v["B"], R1, dX, d1, kind, eps, pre, post, v["post_w"], v["post_b"], v["gate"],
                        gate == "token", v["scale"], v["w"])
    names = [k for k in v if v[k] is not None]
    for k, want in zip(names, _differences(f, [v[k] for k in names])):
        np.testing.assert_allclose(g["d" + k], want, rtol=1e-6, atol=1e-7, err_msg=k)


def test_norm_values():
    x = np.array([[3.0, -4.0], [0.0, 0.0]])
    np.testing.assert_allclose(N.forward(x, "rms", 0.5), [[3 / np.sqrt(13.0), -4 / np.sqrt(13.0)], [0, 0]])
    np.testing.assert_allclose(N.forward(x, "layer", 0.75, b=[1.0, 2.0]), [[3.5 / np.sqrt(13.0) + 1, -3.5 / np.sqrt(13.0) + 2], [1, 2]])
    np.testing.assert_allclose(N.sigmoid(np.array([0.0, 1000.0, -1000.0])), [0.5, 1.0, 0.0])


def _inputs(T, D, seed):
    r = np.random.default_rng(seed)
    return [r.standard_normal((T, D)) for _ in range(3)] + [r.standard_normal(D) - 3.0]


@pytest.mark.parametrize("offsets", [None, [0, 4, 4, 9], [2, 5, 8]])
def test_recurrence_gradients(offsets):
    T, D, c = 9, 2, 8.0
    x, r, i, lam = _inputs(T, D, 1)
    n = 1 if offsets is None else len(offsets) - 1
    g = np.random.default_rng(2)
    h0, dhT, dy = g.standard_normal((n, D)), g.standard_normal((n, D)), g.standard_normal((T, D))

    def f():
        y, hT, _ = R.forward(x, r, i, lam, c, offsets, h0)
        return (y * dy).sum() + (hT * dhT).sum()

    got = R.backward(x, r, i, lam, c, dy, offsets, h0, dhT)
    for k, want in zip(("dx", "dr", "di", "dlam", "dh0"), _differences(f, [x, r, i, lam, h0])):
        np.testing.assert_allclose(got[k], want, rtol=1e-6, atol=1e-7, err_msg=k)


def test_recurrence_values():
    # r = 0: a = exp(-c / 2 log 2) for lam = 0; c = 2: a = 1/2, and i = 0: u = sqrt(3) / 4 x
    y, hT, before = R.forward(np.ones((3, 1)), np.zeros((3, 1)), np.zeros((3, 1)), np.zeros(1), 2.0)
    u = np.sqrt(3.0) / 4
    np.testing.assert_allclose(y[:, 0], [u, 1.5 * u, 1.75 * u])
    np.testing.assert_allclose(before[:, 0], [0, u, 1.5 * u])
    assert hT[0, 0] == y[2, 0]


def test_step_is_the_recurrence():
    T, D, c = 7, 3, 8.0
    x, r, i, lam = _inputs(T, D, 5)
    y, hT, _ = R.forward(x, r, i, lam, c)
    state = np.zeros((2, D))
    got, after = R.step(x, r, i, lam, c, state, np.ones(T, int))    # one state, its positions in order
    np.testing.assert_allclose(got, y)
    np.testing.assert_allclose(after[1], hT[0])
    assert (after[0] == 0).all()
    got, after = R.step(x, r, i, lam, c, state, np.array([-1, 2, 9, -5, 2, 3, 7]))
    assert (got == 0).all() and (after == 0).all()
