"""GPU parity of the feed-forward block where it keeps two bf16 values of H, dG
and dU (include/ffn.h), against the float64 oracle."""
import numpy as np
import pytest
import torch

from oracle import ffn as orc
from test_gpu_ffn import M, NAMES, _bf16, _f64, _real

pytestmark = pytest.mark.gpu


def _same_kind(got, want, name):
    """Infinite with the oracle's sign where it is infinite, NaN where NaN, else finite."""
    g = _f64(got)
    for test in (np.isposinf, np.isneginf, np.isnan):
        bad = int((test(g) != test(want)).sum())
        assert bad == 0, (name, test.__name__, bad)


@pytest.mark.parametrize("kind", ["silu", "relu2"])
@pytest.mark.parametrize("T,F", [(1, 136), (3, 2056), (32, 256)])
def test_infinite_operands(T, F, kind):
    # an infinity times a value kept as two bf16 values of either sign, or of
    # which nothing was left, is an infinity of the value's sign
    m = M()
    X, W, dY, _ = _real(T, F, 60)
    cfg = m.config(F, T, act=kind)
    ws = m.Workspace(cfg)

    def run(X, Wg, Wu, Wd, dY):
        dev = [_bf16(a).cuda() for a in (X, Wg, Wu, Wd)]
        got = {"Y": m.fwd(cfg, ws, *dev), **m.bwd(cfg, ws, *dev, _bf16(dY).cuda())}
        with np.errstate(invalid="ignore", over="ignore"):
            return got, {"Y": orc.forward(X, Wg, Wu, Wd, kind), **orc.backward(X, Wg, Wu, Wd, dY, kind)}

    for value in (np.inf, -np.inf):
        Wd = W[2].copy()
        Wd[5, 7], Wd[9, F - 1] = value, -value
        got, want = run(X, W[0], W[1], Wd, dY)
        _same_kind(got["Y"], want["Y"], "Y")
        assert np.isinf(want["Y"]).any()
        g = dY.copy()
        g[T // 2, 3] = value
        got, want = run(X, *W, g)
        _same_kind(got["dWd"], want["dWd"], "dWd")
        assert np.isinf(want["dWd"]).sum() >= F // 4
        Wu = W[1].copy()
        Wu[7, 3] = value
        got, want = run(X, W[0], Wu, W[2], dY)
        for k in ("dX", "dWu"):
            _same_kind(got[k], want[k], k)
        assert np.isinf(want["dX"]).any() or kind == "relu2"   # (relu2: the unit may be off)
    assert set(got) == {"Y", *NAMES}
