"""Dropped places hold nothing: what a NaN or an infinity there does to the
operators that drop (include/drop.h), and both ends of p inside them."""
import pytest
import torch

from oracle import drop as orcd
from test_gpu_ffn import D, M, NAMES, _bf16, _real

pytestmark = pytest.mark.gpu

SIZES = [(5, 136), (64, 128), (40, 1000), (130, 520), (3001, 2056)]


@pytest.mark.parametrize("yt", ["bf16", "f32"])
@pytest.mark.parametrize("T,F", SIZES)
def test_nan_in_dropped_places_of_dy_reaches_no_gradient(T, F, yt):
    m = M()
    X, W, dY, _ = _real(T, F, 90)
    cfg = m.config(F, T, y_dtype=yt, dw_dtype="f32")
    ws, spec = m.Workspace(cfg), D().spec(0.4, 8, 9)
    Xd, Wc = _bf16(X).cuda(), [_bf16(w).cuda() for w in W]
    clean = torch.from_numpy(dY).to(cfg.y_torch_dtype).cuda()
    keep = torch.from_numpy(orcd.keep(T, 768, 0.4, 8, 9)).cuda()
    bad = torch.where(torch.arange(768, device="cuda") % 2 == 0, float("nan"), float("-inf")).to(clean.dtype)
    dirty = torch.where(keep, clean, bad).contiguous()
    want = m.bwd(cfg, ws, Xd, *Wc, clean, drop=spec)
    got = m.bwd(cfg, ws, Xd, *Wc, dirty, drop=spec)
    assert all(torch.isfinite(want[k]).all() and torch.equal(got[k], want[k]) for k in NAMES)


@pytest.mark.parametrize("T,F", SIZES)
def test_nan_rows_leave_the_residual_in_dropped_places(T, F):
    m = M()
    X, W, _, res = _real(T, F, 91)
    cfg = m.config(F, T, act="gelu")
    Xd, Wc, r = _bf16(X).cuda(), [_bf16(w).cuda() for w in W], _bf16(res).cuda()
    Xd[T // 2] = float("nan")
    y = m.fwd(cfg, m.Workspace(cfg), Xd, *Wc, residual=r, drop=D().spec(0.4, 8, 9))
    keep = torch.from_numpy(orcd.keep(T, 768, 0.4, 8, 9)).cuda()
    assert torch.equal(y[~keep], r[~keep])
    assert torch.isnan(y[T // 2][keep[T // 2]]).all()


@pytest.mark.parametrize("T,F", SIZES)
def test_everything_and_nothing_dropped(T, F):
    m, d = M(), D()
    X, W, dY, res = _real(T, F, 92)
    cfg = m.config(F, T)
    ws = m.Workspace(cfg)
    Xd, Wc, r, g = _bf16(X).cuda(), [_bf16(w).cuda() for w in W], _bf16(res).cuda(), _bf16(dY).cuda()
    assert torch.equal(m.fwd(cfg, ws, Xd, *Wc, residual=r, drop=d.spec(1.0, 1, 2)), r)
    out = m.bwd(cfg, ws, Xd, *Wc, g, drop=d.spec(1.0, 1, 2))
    assert all(torch.count_nonzero(out[k]) == 0 for k in NAMES)
    least = d.spec(2.0 ** -18, 1, 2)       # rounds to a threshold of 0
    assert torch.equal(m.fwd(cfg, ws, Xd, *Wc, residual=r, drop=least), m.fwd(cfg, ws, Xd, *Wc, residual=r))
    plain, out = m.bwd(cfg, ws, Xd, *Wc, g), m.bwd(cfg, ws, Xd, *Wc, g, drop=least)
    assert all(torch.equal(out[k], plain[k]) for k in NAMES)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nan_table_rows_are_zero_in_dropped_places(dtype):
    from sparse_hashed_gram_amd import ngram as N
    cfg = N.config(300, 7, (211, 389), dtype, max_tokens=500)
    W = [torch.full((r, 768), float("nan"), dtype=cfg.torch_dtype, device="cuda") for r in (211, 389)]
    tok = torch.randint(0, 300, (500,), dtype=torch.int32, device="cuda")
    y = N.embed_fwd_drop(cfg, W[0], W[1], tok, D().spec(0.4, 8, 9))
    keep = torch.from_numpy(orcd.keep(500, 768, 0.4, 8, 9)).cuda()
    assert torch.count_nonzero(y[~keep]) == 0 and torch.isnan(y[keep]).all()


def test_residual_in_place_of_another_type():
    # fp32 residual stream updated in place by a bf16 branch, rows that end inside a group
    d = D()
    x = torch.randn(37, 771).bfloat16()
    r = torch.randn(37, 771, device="cuda")
    want = d.fwd(d.spec(0.3, 1, 2), x.cuda(), residual=r)
    assert d.fwd(d.spec(0.3, 1, 2), x.cuda(), residual=r, out=r) is r and torch.equal(r, want)
