"""GPU parity of the feed-forward block's kernels of many positions, at sizes
that reach each of them (tests/test_ffn_plan_cpu.py holds the lists below to
that).  Whole-number cases are exact and real-valued ones are held to the
bounds that stand, with their derivation, at the top of test_gpu_ffn.py.
"""
import numpy as np
import pytest
import torch

from oracle import drop as orcd
from oracle import ffn as orc
from test_gpu_ffn import D, M, NAMES, _bf16, _bounds, _hold, _real, _run_whole, _same, _whole

pytestmark = pytest.mark.gpu

# positions, hidden units, share dropped
WHOLE = [(8193, 1000, 0.5), (4001, 1000, 0.0), (1100, 2848, 0.5), (617, 13080, 0.0), (1025, 2992, 0.5)]
# the same for an activation, types of the stream and of the weights' gradients
REAL = [(7823, 1000, 0.1, "silu", "bf16", "bf16"), (7823, 1000, 0.3, "gelu", "f32", "f32"),
        (3001, 2056, 0.0, "gelu", "bf16", "f32"), (3001, 2056, 0.2, "silu", "f32", "bf16")]
# accumulated weights' gradients: in parts on both tiles, and in one part
ACCUM = [(8193, 1000, 0.5), (3500, 264, 0.0), (333, 520, 0.5), (300, 65536, 0.0)]


@pytest.mark.parametrize("T,F,p", WHOLE)
def test_whole_numbers(T, F, p):
    _run_whole(T, F, p)


@pytest.mark.parametrize("dw", ["f32", "bf16"])
@pytest.mark.parametrize("T,F,p", ACCUM)
def test_accumulated_gradients(T, F, p, dw):
    # two micro-steps into gradients that hold whole numbers already.  Every sum is
    # exact in fp32, so bf16 gradients are the rounded sums, once a micro-step
    m = M()
    cfg = m.config(F, T, act="relu2", y_dtype="f32", dw_dtype=dw, accumulate=True)
    ws = m.Workspace(cfg)
    td = cfg.dw_torch_dtype
    r = np.random.default_rng([T, F, 11])
    want = [torch.from_numpy(r.integers(-3, 4, s)).float().to(td) for s in ((F, 768), (F, 768), (768, F))]
    got = [w.cuda() for w in want]
    for step in range(2):
        X, W, dY, _ = _whole(T, F, 20 + step)
        spec = D().spec(p, 5, step) if p else None
        factor = orcd.keep(T, 768, p, 5, step) * 2.0 if p else None
        g = m.bwd(cfg, ws, _bf16(X).cuda(), *(_bf16(w).cuda() for w in W), torch.from_numpy(dY).float().cuda(), spec,
                  None, *got)
        o = orc.backward(X, *W, dY, "relu2", factor)
        _same(g["dX"], o["dX"], "dX")
        for i, k in enumerate(NAMES[1:]):
            want[i] = (want[i].double() + torch.from_numpy(o[k])).float().to(td)
            assert g[k].data_ptr() == got[i].data_ptr()
            _same(g[k], want[i].double().numpy(), f"{k} of step {step}")


@pytest.mark.parametrize("T,F,p,kind,yt,wt", REAL)
def test_real_values(T, F, p, kind, yt, wt):
    m = M()
    X, W, dY, res = _real(T, F)
    cfg = m.config(F, T, act=kind, y_dtype=yt, dw_dtype=wt)
    ws = m.Workspace(cfg)
    spec = D().spec(p, 5, 6) if p else None
    factor = orcd.keep(T, 768, p, 5, 6) * (65536 / (65536 - orcd.threshold(p))) if p else None
    td, b = cfg.y_torch_dtype, 2.0 ** -24
    Xd, Wc = _bf16(X).cuda(), [_bf16(w).cuda() for w in W]
    resd, dYd = torch.from_numpy(res).to(td).cuda(), torch.from_numpy(dY).to(td).cuda()
    o = _bounds(X, W, dY, kind, factor, yt == "f32")
    y = m.fwd(cfg, ws, Xd, *Wc, residual=resd, drop=spec)
    _hold(y, o["Y"][0] + res, o["Y"][1] + 2 * b * np.abs(res), yt == "bf16", "Y")
    g = m.bwd(cfg, ws, Xd, *Wc, dYd, drop=spec)
    for k in NAMES:
        _hold(g[k], *o[k], g[k].dtype == torch.bfloat16, k)
    # and again, over whatever the first pass left in the workspace
    assert torch.equal(y, m.fwd(cfg, ws, Xd, *Wc, residual=resd, drop=spec))
    h = m.bwd(cfg, ws, Xd, *Wc, dYd, drop=spec)
    assert all(torch.equal(g[k], h[k]) for k in NAMES)


@pytest.mark.parametrize("kind", ["silu", "gelu", "relu2"])
def test_nan_and_inf_stay_in_their_rows(kind):
    # 7,823 positions: the last tile of 256 is moved back to 7,567, so rows up to
    # 7,679 are written by two blocks
    m = M()
    T, F = 7823, 1000
    X, W, dY, _ = _real(T, F, 4)
    Xd, Wc, dYd = _bf16(X).cuda(), [_bf16(w).cuda() for w in W], _bf16(dY).cuda()
    cfg = m.config(F, T, act=kind)
    ws = m.Workspace(cfg)
    clean, cdx = m.fwd(cfg, ws, Xd, *Wc), m.bwd(cfg, ws, Xd, *Wc, dYd)["dX"]
    rows = torch.tensor([0, 7566, 7567, 7600, 7679, 7680, 7822], device="cuda")
    bad = Xd.clone()
    bad[rows, 3] = torch.tensor([float("nan"), float("inf"), float("nan"), float("-inf"), float("nan"), float("inf"),
                                 float("nan")], dtype=torch.bfloat16, device="cuda")
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[rows] = False
    y, dx = m.fwd(cfg, ws, bad, *Wc), m.bwd(cfg, ws, bad, *Wc, dYd)["dX"]
    assert torch.equal(y[rest], clean[rest]) and torch.equal(dx[rest], cdx[rest])
    assert torch.all(torch.any(~torch.isfinite(y[rows]), 1))
