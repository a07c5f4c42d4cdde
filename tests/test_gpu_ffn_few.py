"""GPU parity of the feed-forward block where it keeps two bf16 values of H, dG
and dU (include/ffn.h), against the float64 oracle."""
import numpy as np
import pytest
import torch

from oracle import drop as orcd
from oracle import ffn as orc
from test_gpu_ffn import D, M, NAMES, _bf16, _f64, _real, _run_whole

pytestmark = pytest.mark.gpu


def _same_kind(got, want, name):
    """Infinite with the oracle's sign where it is infinite, NaN where NaN, else finite."""
    g = _f64(got)
    for test in (np.isposinf, np.isneginf, np.isnan):
        bad = int((test(g) != test(want)).sum())
        assert bad == 0, (name, test.__name__, bad)


@pytest.mark.parametrize("kind", ["silu", "relu2"])
@pytest.mark.parametrize("T,F", [(1, 136), (3, 2056), (32, 256), (64, 128)])
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


@pytest.mark.parametrize("kind", ["silu", "gelu", "relu2"])
@pytest.mark.parametrize("T,F", [(33, 128), (33, 248), (48, 136), (64, 128), (64, 72)])
def test_one_rounding_up_to_64_positions(T, F, kind):
    # 16 bits of H, dG and dU leave a result's own rounding beside the operands'
    # 2^-17 and fp32 sums of at most 1,000 terms (2^-14), together below 2^-13 of the
    # norm.  The rounding's norm is that of the oracle's values but for the few
    # values that lie near a tie: the root of a mean of n squares of values spread
    # evenly strays by 0.45 / sqrt(n), 0.2 % at n = 64 x 768, and 5 % is allowed.
    # (One bf16 value of each would make it 1.41 times that.)
    m = M()
    X, W, dY, _ = _real(T, F, 70)
    cfg = m.config(F, T, act=kind)
    ws, spec = m.Workspace(cfg), D().spec(0.2, 3, 4)
    factor = orcd.keep(T, 768, 0.2, 3, 4) * (65536 / (65536 - orcd.threshold(0.2)))
    Xd, Wc = _bf16(X).cuda(), [_bf16(w).cuda() for w in W]
    got = {"Y": m.fwd(cfg, ws, Xd, *Wc, drop=spec), **m.bwd(cfg, ws, Xd, *Wc, _bf16(dY).cuda(), drop=spec)}
    want = {"Y": orc.forward(X, *W, kind, factor), **orc.backward(X, *W, dY, kind, factor)}
    for k, v in want.items():
        own = np.linalg.norm(_f64(_bf16(v)) - v)
        assert np.linalg.norm(_f64(got[k]) - v) <= 1.05 * own + 2.0 ** -13 * np.linalg.norm(v), k


@pytest.mark.parametrize("T,F,p", [(33, 248, 0.5), (33, 256, 0.0), (64, 128, 0.5), (64, 136, 0.0), (65, 120, 0.5), (50, 8, 0.0)])
def test_whole_numbers_either_side(T, F, p):
    _run_whole(T, F, p, max_tokens=T + 2)


@pytest.mark.parametrize("T,F", [(1, 8192), (1, 8), (64, 128), (31, 264), (65, 1000), (130, 8), (300, 2056)])
def test_nothing_behind_the_workspace(T, F):
    # a workspace of exactly the bytes asked for, guarded; results as with a roomy one
    m = M()
    X, W, dY, _ = _real(T, F, 80)
    Xd, Wc, dYd = _bf16(X).cuda(), [_bf16(w).cuda() for w in W], _bf16(dY).cuda()
    roomy = m.config(F, T + 1000)
    want = m.bwd(roomy, m.Workspace(roomy), Xd, *Wc, dYd)
    wy = m.fwd(roomy, m.Workspace(roomy), Xd, *Wc)
    cfg = m.config(F, T)
    for backward in (False, True):
        n = m.workspace_bytes(cfg, backward)
        buf = torch.full((n + (1 << 20) + 256,), 165, dtype=torch.uint8, device="cuda")
        off = -buf.data_ptr() % 256
        ws = m.Workspace(cfg, backward=backward)
        ws.tensor = buf[off:off + n]
        ws.ptr = ws.tensor.data_ptr()
        assert torch.equal(m.fwd(cfg, ws, Xd, *Wc), wy)
        if backward:
            got = m.bwd(cfg, ws, Xd, *Wc, dYd)
            assert all(torch.equal(got[k], want[k]) for k in NAMES)
        assert torch.all(buf[:off] == 165) and torch.all(buf[off + n:] == 165)
