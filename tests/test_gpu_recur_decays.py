"""Fast decays of the gated linear recurrence (include/recur.h): a = exp(z) far
from 1, where a state falls by many powers of ten within a position and what is
left of it still has to be right to a few roundings of itself.

The cases hold products only: x = 0 and dy = 0, h0 and dhT positive, so
h_t = a_1 ... a_t h0 and G_t = a_{t+1} ... a_T dhT, and no sum hides a factor's
relative error.  Tolerances, u = 2^-24, relative:
- z = -c sp(lam) s(r): (2 |r| + 16) u (exp's argument |r| u and exp, sum, reciprocal a
  few u for s(r), twice |r| for the product with log2(e) and its constant; 8 u more for
  sp and the products);
- a = exp(z): z's error times |z|, the product with log2(e) and its constant 2 u |z|,
  exp2 itself 2 u; near 1, where a = 1 + e, (2 |r| + 26) u of |e|, and |e| / a is at most
  1.2 |z|, and 1 u: both are below 1.2 (2 |r| + 26) |z| u + 3 u;
- a product over positions: its factors' errors and 2 u a position, 42 u for the joining
  of pieces;
- s(r) and 1 - s(r): (2 |r| + 8) u; m = sqrt(1 - a^2): half of 1 - a^2's, at most (2 |r| +
  30) u, and s(i) (2 |i| + 8) u;
- dlam: all its terms have one sign, so the largest relative error of a term, T / 64 + 90 u
  of the sum and 40 u of c s(lam).
"""
import numpy as np
import pytest
import torch

from oracle import recur as orc

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def M():
    from sparse_hashed_gram_amd import recur
    return recur


def _dev(a, t="f32"):
    x = torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(TORCH[t])
    return x.cuda(), x.double().numpy()


def _near(got, want, rel, t, name):
    g = got.double().cpu().numpy()
    lim = 1.01 * (rel * U + HALF[t] * (1 + rel * U)) * np.abs(want)
    off = np.abs(g - want)
    assert (off <= lim).all(), (name, np.max(off / np.maximum(lim, 1e-300)))


def _inputs(T, D, t, seed):
    r = np.random.default_rng([T, D, seed])
    rr, hr = _dev(np.clip(r.standard_normal((T, D)), -2.0, 0.5), t)
    i, hi = _dev(r.standard_normal((T, D)), t)
    return r, rr, hr, i, hi, torch.zeros(T, D, dtype=TORCH[t], device="cuda")


def _relative(hr, hlam, c):
    """(a, the relative bound of a in u)."""
    z = c * orc.softplus(hlam) * orc.sigmoid(hr)
    return np.exp(-z), 1.2 * (2 * np.abs(hr) + 26) * z + 3, z


# lam of 1 to 4 and c of 8: z of -1 to -20; c of 64: -3 to -19, from lam of -2 to -0.5
@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("c,lo,hi", [(8.0, 1.0, 4.0), (64.0, -2.0, -0.5)])
@pytest.mark.parametrize("T,D", [(3, 70), (100, 33), (400, 70), (1500, 2000)])
def test_what_fast_decays_leave(T, D, c, lo, hi, t):
    m = M()
    r, rr, hr, i, hi_, x = _inputs(T, D, t, 1)
    lam, hlam = _dev(np.linspace(lo, hi, D))
    off = [0]
    while off[-1] < T:   # sequences of one to three positions
        off.append(min(T, off[-1] + len(off) % 3 + 1))
    n = len(off) - 1
    h0, hh0 = _dev(1 + r.random((n, D)))
    dhT, hdhT = _dev(1 + r.random((n, D)))
    cfg = m.config(D, T, t, c)
    ws = m.Workspace(cfg)
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    y, hT, saved = m.fwd(cfg, ws, x, rr, i, lam, offsets, h0, keep=True, final=True)
    g = m.bwd(cfg, ws, x, rr, i, lam, saved, x, offsets, h0, dhT)
    a, ra, z = _relative(hr, hlam, c)
    oy, ohT, _ = orc.forward(0 * hr, hr, hi_, hlam, c, off, hh0)
    o = orc.backward(0 * hr, hr, hi_, hlam, c, 0 * hr, off, hh0, hdhT)
    total = np.zeros((n, D))
    through = np.zeros((T, D))   # of the whole sequence's product, which h_{t-1} a_t G_t is
    upto, behind = np.zeros((T, D)), np.zeros((T, D))
    for k in range(n):
        s = slice(off[k], off[k + 1])
        assert z[s].sum(0).max() < 80   # nothing leaves fp32's normal range
        upto[s] = np.cumsum(ra[s] + 2, 0) + 42
        total[k] = (ra[s] + 2).sum(0) + 42
        through[s] = total[k]
        behind[s] = total[k] - np.cumsum(ra[s] + 2, 0) + 42
    assert (a < 2.0 ** -24).any() or T < 10
    _near(y, oy, upto, t, "y")
    _near(hT, ohT, total, "f32", "hT")
    _near(g["dh0"], o["dh0"], total, "f32", "dh0")
    ar = np.abs(hr)
    _near(g["dr"], o["dr"], through + 6 * ar + 60, t, "dr")
    _near(g["dx"], o["dx"], behind + 2 * ar + 30 + 2 * np.abs(hi_) + 12, t, "dx")
    assert (g["di"] == 0).all()
    _near(g["dlam"], o["dlam"], (through + 2 * ar + 16).max(0) + T / 64 + 90 + 40, "f32", "dlam")


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("n,D", [(1, 64), (5, 65), (700, 258)])
def test_what_a_step_leaves(n, D, t):
    m = M()
    r, rr, hr, i, hi, x = _inputs(n, D, t, 2)
    lam, hlam = _dev(np.linspace(1.0, 4.0, D))
    st, hst = _dev(1 + r.random((n, D)))
    y = m.step(m.config(D, 1, t), x, rr, i, lam, st)
    a, ra, _ = _relative(hr, hlam, 8.0)
    _near(st, a * hst, ra + 2, "f32", "state")
    _near(y, a * hst, ra + 2, t, "y")


def test_an_infinite_state_stays():
    """a h of an infinite h is infinite while a is not 0."""
    m = M()
    T, D = 3, 8
    lam, r = torch.full((D,), 4.0, device="cuda"), torch.full((T, D), 0.5, device="cuda")   # z of -20
    x = torch.ones(T, D, device="cuda")
    h0 = torch.full((1, D), float("inf"), device="cuda")
    cfg = m.config(D, T, "f32")
    ws = m.Workspace(cfg)
    y, hT, _ = m.fwd(cfg, ws, x, r, x, lam, h0=h0, final=True)
    assert (y == float("inf")).all() and (hT == float("inf")).all()
    st = h0.clone()
    assert (m.step(cfg, x[:1], r[:1], x[:1], lam, st) == float("inf")).all() and (st == float("inf")).all()
