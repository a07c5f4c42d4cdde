"""Pins of the feed-forward oracle (oracle/ffn.py): torch's own functions and
autograd in float64, differences, closed forms."""
import numpy as np
import pytest
import torch

from oracle import ffn as orc

KINDS = ["silu", "gelu", "relu2"]


def _case(T=5, D=12, F=9, seed=0):
    r = np.random.default_rng(seed)
    return [r.standard_normal(s) for s in ((T, D), (F, D), (F, D), (D, F), (T, D))]


def _torch_act(g, kind):
    if kind == "silu":
        return torch.nn.functional.silu(g)
    if kind == "gelu":
        return torch.nn.functional.gelu(g, approximate="tanh")
    return torch.relu(g).square()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dropped", [False, True])
def test_against_autograd(kind, dropped):
    X, Wg, Wu, Wd, dY = _case()
    f = (np.random.default_rng(1).random(dY.shape) < 0.5) * 2.0 if dropped else None
    t = [torch.tensor(v, requires_grad=True) for v in (X, Wg, Wu, Wd)]
    y = (_torch_act(t[0] @ t[1].T, kind) * (t[0] @ t[2].T)) @ t[3].T
    if dropped:
        y = y * torch.tensor(f)
    res = np.ones_like(dY)
    np.testing.assert_allclose(orc.forward(X, Wg, Wu, Wd, kind, f, res), y.detach().numpy() + 1, rtol=1e-12, atol=1e-12)
    y.backward(torch.tensor(dY))
    got = orc.backward(X, Wg, Wu, Wd, dY, kind, f)
    for k, v in zip(("dX", "dWg", "dWu", "dWd"), t):
        np.testing.assert_allclose(got[k], v.grad.numpy(), rtol=1e-11, atol=1e-12)


@pytest.mark.parametrize("kind", KINDS)
def test_against_differences(kind):
    X, Wg, Wu, Wd, dY = _case(seed=2)
    got = orc.backward(X, Wg, Wu, Wd, dY, kind)
    args = {"dX": X, "dWg": Wg, "dWu": Wu, "dWd": Wd}
    h = 1e-6
    for k, a in args.items():
        for i in [(0, 0), tuple(n - 1 for n in a.shape), (a.shape[0] // 2, 1)]:
            keep = a[i]
            a[i] = keep + h
            up = (orc.forward(X, Wg, Wu, Wd, kind) * dY).sum()
            a[i] = keep - h
            down = (orc.forward(X, Wg, Wu, Wd, kind) * dY).sum()
            a[i] = keep
            assert (up - down) / (2 * h) == pytest.approx(got[k][i], rel=1e-6, abs=1e-7)


def test_closed_forms():
    # one unit, one input: y = d a(g x) u x
    y = orc.forward([[2.0]], [[3.0]], [[5.0]], [[7.0]], "relu2")
    assert y[0, 0] == 7 * 36 * 10
    assert orc.act(np.array([0.0]), "silu")[1][0] == 0.5 and orc.act(np.array([0.0]), "gelu")[1][0] == 0.5
    a, d = orc.act(np.array([40.0, -800.0]), "silu")
    assert a[0] == pytest.approx(40) and d[0] == pytest.approx(1) and a[1] == 0 and d[1] == 0
    g = np.linspace(-5, 5, 11)
    for kind in KINDS:
        num = (orc.act(g + 1e-6, kind)[0] - orc.act(g - 1e-6, kind)[0]) / 2e-6
        np.testing.assert_allclose(orc.act(g, kind)[1], num, atol=2e-6)
