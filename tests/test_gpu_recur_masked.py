"""Positions that the recurrence's gate r closes (s(r) = 0: a = 1, the state goes
on as it is), whatever finite value x holds there, and gates that are all but closed."""
import numpy as np
import pytest
import torch

from oracle import recur as orc

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def M():
    from sparse_hashed_gram_amd import recur
    return recur


def _run(x, r, i, lam, h0, dy, t, c=8.0):
    m = M()
    T, D = x.shape
    cfg = m.config(D, T, t, c)
    ws = m.Workspace(cfg)
    y, hT, saved = m.fwd(cfg, ws, x, r, i, lam, h0=h0, keep=True, final=True)
    return {"y": y, "hT": hT, **m.bwd(cfg, ws, x, r, i, lam, saved, dy, h0=h0)}


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("closed", [-float("inf"), -200.0, "lowest"])
@pytest.mark.parametrize("T", [20, 300])
def test_what_stands_in_closed_positions(T, closed, t):
    """The type's lowest and largest values where r closes a position: every result is the
    one with zeros there, and dx and di are 0."""
    dt = torch.float32 if t == "f32" else torch.bfloat16
    D = 70
    gen = torch.Generator().manual_seed(T)
    x, r, i, dy = (torch.randn(T, D, generator=gen).to(dt).cuda() for _ in range(4))
    h0 = torch.randn(1, D, generator=gen).cuda()
    lam = torch.linspace(-7, 2, D).cuda()
    shut = torch.zeros(T, dtype=torch.bool)
    shut[3:7] = shut[T - 2] = True
    r[shut] = torch.finfo(dt).min if closed == "lowest" else closed
    x[shut] = 0.0
    want = _run(x, r, i, lam, h0, dy, t)
    assert all(torch.isfinite(v).all() for v in want.values())
    for v in (1e21, torch.finfo(dt).max, torch.finfo(dt).min):
        x[shut] = v
        got = _run(x, r, i, lam, h0, dy, t)
        for k in want:
            assert torch.equal(got[k], want[k]), (k, v)
        assert (got["dx"][shut] == 0).all() and (got["di"][shut] == 0).all()


@pytest.mark.parametrize("r,lam,c", [(-87.0, 1.0, 8.0), (0.0, -86.0, 8.0), (0.5, 0.0, 1e-37)])
def test_all_but_closed(r, lam, c):
    """m = sqrt(1 - a^2) below 1e-18: dr, whose part from the input is z / m of x, and
    dlam.  T = 1 without a state, so that part is all there is, and its relative error is
    z's, 1 / m's half of it, and those of the products: (2 |r| + 26) 1.5 u for z and m,
    (2 |r| + 8) 2 u for s(r) and 1 - s(r), 40 u for the rest, and |lam| 4 u for sp and s(lam)."""
    D = 64
    f = lambda v: torch.full((1, D), v, device="cuda")   # noqa: E731
    x = torch.linspace(0.5, 2, D, device="cuda")[None]
    got = _run(x, f(r), f(0.3), f(lam)[0], None, f(0.25), "f32", c)
    h = [v.double().cpu().numpy() for v in (x, f(r), f(0.3), f(lam)[0])]
    o = orc.backward(*h, float(np.float32(c)), np.full((1, D), 0.25))
    # -expm1(2 z) and a^2 / m are exact enough in 64 bits for z of 1e-37
    rel = (1.5 * (2 * abs(r) + 26) + 2 * (2 * abs(r) + 8) + 40 + 4 * abs(lam)) * U
    for k in ("dx", "dr", "dlam"):
        g = got[k].double().cpu().numpy()
        assert (np.abs(o[k]) > 0).all()
        assert (np.abs(g - o[k]) <= rel * np.abs(o[k]) + 2.0 ** -140).all(), k
