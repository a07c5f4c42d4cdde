"""Norms of rows that leave fp32's range of squares: rows of one huge value, whose
deviations from their mean are 0, and rows with an infinity."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")]
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-3


def N():
    from sparse_hashed_gram_amd import norm
    return norm


def _rows(T, D, dt, seed=0):
    return torch.randn(T, D, generator=torch.Generator().manual_seed(D + seed)).to(dt).cuda()


# constants whose D-fold sums and products with 1 / D are rounded, and whose D-fold are not
WIDTHS = [1, 2, 4, 41, 768, 769, 1000, 1024, 1500, 2048, 4095, 4096]


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("D", WIDTHS)
def test_constant_rows(D, types):
    """With mean: xh = 0, so X = b, dw = 0, and the gradient goes through with 1 / sqrt(eps):
    dR = dR1 + (dxh - mean(dxh)) / sqrt(eps).  The mean of at most 4,096 terms is off by 28 u
    of their mean magnitude (16 additions in a lane, 6 across the wavefront, 3 across
    wavefronts, the product with 1 / D and its rounding), rho by 4 u, and the products and
    sums 4 u of their terms.  The rows between them are those of a call without them."""
    n = N()
    xt, rt = (TORCH[k] for k in types)
    cfg = n.config(D, "layer", *types, eps=EPS)
    ws = n.Workspace(cfg)
    big = [2.0 ** 70, -2.0 ** 127, float(torch.finfo(rt).min), 1.2345e30]
    T = 2 * len(big)
    R, dX, dR1 = _rows(T, D, rt), _rows(T, D, xt, 1), _rows(T, D, rt, 2)
    R[5] *= 2.0 ** 70   # huge, but not constant
    w, b = 1 + 0.1 * _rows(1, D, torch.float32, 3)[0], _rows(1, D, torch.float32, 4)[0]
    plain = n.fwd(cfg, R, w, b), n.bwd(cfg, ws, R, dX, w, b, dR1=dR1)
    for k, v in enumerate(big):
        R[2 * k] = v
    X = n.fwd(cfg, R, w, b)
    g = n.bwd(cfg, ws, R, dX, w, b, dR1=dR1)
    assert torch.equal(X[::2], b.to(xt).expand(len(big), D))
    assert torch.equal(X[1::2], plain[0][1::2]) and torch.equal(g["dR"][1::2], plain[1]["dR"][1::2])
    d = (dX.double() * w.double())[::2]
    rho = float(np.float32(EPS)) ** -0.5
    size = d.abs().mean(1, keepdim=True)
    want = dR1[::2].double() + rho * (d - d.mean(1, keepdim=True))
    lim = U * (rho * (10 * d.abs() + 36 * size) + 2 * dR1[::2].double().abs())
    lim = 1.01 * (lim + torch.finfo(rt).eps / 2 * (want.abs() + lim))
    assert ((g["dR"][::2].double() - want).abs() <= lim).all()
    assert torch.isfinite(g["dw"]).all() and torch.isfinite(g["db"]).all()
    only = n.bwd(cfg, ws, R[::2].contiguous(), dX[::2].contiguous(), w, b)
    assert (only["dw"] == 0).all() and torch.equal(only["dR"].float(), n.bwd(
        cfg, ws, torch.zeros_like(R[::2]), dX[::2].contiguous(), w, b)["dR"].float())


@pytest.mark.parametrize("D", [1, 41, 768, 1000, 1500, 4096])
def test_constant_rows_of_a_block(D):
    """The same of a block's output, behind the block."""
    n = N()
    cfg = n.config(D, "layer", gate="vector", eps=EPS)
    ws = n.Workspace(cfg)
    T = 6
    R, B, dX = _rows(T, D, torch.float32), _rows(T, D, torch.bfloat16, 1), _rows(T, D, torch.bfloat16, 2)
    B[1], B[4] = 2.0 ** 80, torch.finfo(torch.bfloat16).min
    zero = B.clone()
    zero[1] = zero[4] = 0.0
    p = {k: 1 + 0.1 * _rows(1, D, torch.float32, 5 + j)[0] for j, k in enumerate(("post_w", "post_b", "gate", "w", "b"))}
    a, z = n.join_fwd(cfg, R, B, **p), n.join_fwd(cfg, R, zero, **p)
    assert torch.equal(a[0], z[0]) and torch.equal(a[1], z[1])
    g, h = (n.join_bwd(cfg, ws, None, v, a[0], dX, R, **p) for v in (B, zero))
    assert all(torch.equal(g[k], h[k]) for k in h)


@pytest.mark.parametrize("D", [5, 64, 768, 1000, 1500, 4096])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_not_finite_rows(kind, D):
    """A NaN or an infinity in a row makes its norm NaN, all of it, and the row's gradient;
    no other row."""
    n = N()
    T = 9
    cfg = n.config(D, kind)
    ws = n.Workspace(cfg)
    R, dX = _rows(T, D, torch.float32), _rows(T, D, torch.bfloat16, 1)
    w, b = 1 + 0.1 * _rows(1, D, torch.float32, 3)[0], _rows(1, D, torch.float32, 4)[0]
    X0, g0 = n.fwd(cfg, R, w, b), n.bwd(cfg, ws, R, dX, w, b)
    keep = torch.arange(T, device="cuda") != 4
    for where in (0, D // 2, D - 1, slice(None)):
        for v in (float("inf"), -float("inf"), float("nan")):
            S = R.clone()
            S[4, where] = v
            X, g = n.fwd(cfg, S, w, b), n.bwd(cfg, ws, S, dX, w, b)
            assert torch.equal(X[keep], X0[keep]) and torch.equal(g["dR"][keep], g0["dR"][keep])
            assert torch.isnan(X[4]).all() and torch.isnan(g["dR"][4]).all() and torch.isnan(g["dw"]).all()
            assert torch.equal(g["db"], g0["db"])
    S = R.clone()
    S[4, 0], S[4, 1:] = float("inf"), 2.0 ** 100
    assert torch.isnan(n.fwd(cfg, S, w, b)[4]).all()


@pytest.mark.parametrize("D", [64, 1000])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_not_finite_rows_of_a_block(kind, D):
    n = N()
    T = 9
    cfg = n.config(D, kind, gate="token")
    ws = n.Workspace(cfg)
    R, B, dX, G = (_rows(T, D, t, k) for k, t in enumerate((torch.float32, *3 * (torch.bfloat16,))))
    clean = n.join_fwd(cfg, R, B, gate=G)
    keep = torch.arange(T, device="cuda") != 2
    for v in (float("inf"), -float("inf"), float("nan")):
        S = B.clone()
        S[2, D // 3] = v
        R1, X = n.join_fwd(cfg, R, S, gate=G)
        assert torch.equal(R1[keep], clean[0][keep]) and torch.equal(X[keep], clean[1][keep])
        assert torch.isnan(R1[2]).all() and torch.isnan(X[2]).all()
        g = n.join_bwd(cfg, ws, None, S, clean[0], dX, R, gate=G)
        h = n.join_bwd(cfg, ws, None, B, clean[0], dX, R, gate=G)
        assert torch.isnan(g["dB"][2]).all() and torch.isnan(g["dgate"][2]).all()
        assert torch.equal(g["dR"], h["dR"]) and torch.equal(g["dB"][keep], h["dB"][keep])
