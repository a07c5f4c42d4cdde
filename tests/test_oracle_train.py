"""The oracles' gradients chained as a training step chains them (embedding,
dropout, feed-forward block with residual and dropout, loss, and back) against
differences of the whole step's loss, in float64."""
import numpy as np

from oracle import drop as orcd
from oracle import ffn as orcf
from oracle import ssm as orcs


def test_chained_gradients_against_differences():
    r = np.random.default_rng(3)
    R, T, F, V, C = 12, 40, 24, 90, 60
    rows = r.integers(0, R, T)
    sign = r.choice([-1.0, 1.0], T)[:, None]
    tgt = r.integers(0, V, T).astype(np.int32)
    cand, slot, _, ok = orcs.candidates(tgt, r.permutation(V).astype(np.int32), V, C)
    assert ok
    g = r.random(T) / T
    fe, ff = (orcd.keep(T, 768, p, 5, o) * (65536 / (65536 - orcd.threshold(p))) for p, o in ((0.1, 1), (0.3, 2)))
    P = {"table": r.standard_normal((R, 768)), "Wg": r.standard_normal((F, 768)) / 28,
         "Wu": r.standard_normal((F, 768)) / 28, "Wd": r.standard_normal((768, F)) / 5,
         "U": r.standard_normal((V, 768)) / 28}

    def loss(P):
        E = sign * P["table"][rows] * fe
        Y = orcf.forward(E, P["Wg"], P["Wu"], P["Wd"], "gelu", ff, E)
        return (orcs.loss_fwd(Y, P["U"], cand, slot)[0] * g).sum(), E, Y

    _, E, Y = loss(P)
    dY, dUc = orcs.loss_bwd(Y, P["U"], cand, slot, g)
    f = orcf.backward(E, P["Wg"], P["Wu"], P["Wd"], dY, "gelu", ff)
    dE = (dY + f["dX"]) * fe * sign
    grad = {"table": np.zeros((R, 768)), "U": np.zeros((V, 768)), **{k: f["d" + k] for k in ("Wg", "Wu", "Wd")}}
    np.add.at(grad["table"], rows, dE)
    grad["U"][cand] = dUc
    for k in P:
        D = r.standard_normal(P[k].shape)
        h = 1e-5
        ends = [loss({**P, k: P[k] + s * h * D})[0] for s in (1, -1)]
        want = (grad[k] * D).sum()
        # third derivatives are O(1) of these sizes: h^2 = 1e-10; fp64 noise 1e-16 |loss| / h
        assert abs((ends[0] - ends[1]) / (2 * h) - want) <= 1e-6 * (abs(want) + np.linalg.norm(grad[k])), k
