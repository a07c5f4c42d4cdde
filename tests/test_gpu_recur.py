"""GPU parity of the gated linear recurrence (include/recur.h) against the float64
oracle, through the C ABI.

Tolerances, u = 2^-24, worst cases of each operation:
- rho = s(r): exp's argument is off by |r| u, and exp, sum, reciprocal, product by a
  few u: (2 |r| + 8) u; g alike;
- z = -c sp(lam) rho: 8 u more for sp and the products: rz = (2 |r| + 16) u;
- e = exp(z) - 1: an error of z carries over at most as it is, the series or the
  difference from 1 (exp at most 0.71 beside 0.29) adds 10 u: re = (2 |r| + 26) u;
- a = 1 + e: ra = u + re |e| / a (e / a reaches far only where a is small, and the
  absolute error of a, u + re |e|, is what counts); m = sqrt(-e (2 + e)): re + 4 u;
- u_t = m g x: ru = re + (2 |i| + 14) u;
- h: a sum of terms u_s a_{s+1} ... a_t.  However the scan groups them, a term's
  relative error is that of its factors and a rounding for each product and sum on
  its way, at most two a position and 40 for the joining of pieces.  With S_t = a_t
  S_{t-1} + |u_t|: E_t = a_t E_{t-1} + S_{t-1} (ea_t + 2 u a_t) + |u_t| ru, and the
  bound is E + 42 u S.  The same for G backwards, from |dy|.
- the gradients carry these on by the product rule (bounds.py).
A norm bound on top: the errors of many independent roundings do not add up the
worst way.  A rounding's square is at most 1/3 of its half step's on average, so the
error's 2-norm over the value's is at most 1 / sqrt(3) of 2^-8 on average, and held to
0.6 of it.  That needs many values that count: the square of that ratio strays by 0.9
/ sqrt(N), N = (sum v^2)^2 / sum v^4, and with mantissas spread over an octave its
mean is 0.18; from N = 256 on, 0.36 is over ten times 5.6 % of 0.18 away.  Below (one
position's few values, of which one may carry the norm) the element-wise bound stands
alone.
"""
import numpy as np
import pytest
import torch

from bounds import U, V, within
from oracle import recur as orc

pytestmark = pytest.mark.gpu

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}


def M():
    from sparse_hashed_gram_amd import recur
    return recur


def _dev(a, t="f32"):
    x = torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(TORCH[t])
    return x.cuda(), x.double().numpy()


def _scan_bound(a, ea, u, eu, cut, first, efirst, reverse=False):
    """(E, S) of the scan; cut[t]: the state in front of position t (behind it, if
    reverse) is first[t]."""
    T = u.shape[0]
    E, S = np.zeros(u.shape), np.zeros(u.shape)
    e = s = np.zeros(u.shape[1])
    for t in (range(T - 1, -1, -1) if reverse else range(T)):
        if cut[t]:
            e, s = efirst[t], np.abs(first[t])
        E[t] = a[t] * e + s * (ea[t] + 2 * U * a[t]) + eu[t]
        S[t] = a[t] * s + np.abs(u[t])
        e, s = E[t], S[t]
    return E, S


class Case:
    def __init__(self, T, D, t, offsets=None, h0=False, dhT=False, seed=0, c=8.0, decay=(0.9, 0.999), spread=1.0):
        r = np.random.default_rng([T, D, seed])
        self.T, self.D, self.t, self.c = T, D, t, float(np.float32(c))
        for k in ("x", "r", "i"):
            a, h = _dev(r.standard_normal((T, D)) * (1.0 if k == "x" else spread), t)
            setattr(self, k, a), setattr(self, "h" + k, h)
        self.dy, self.hdy = _dev(r.standard_normal((T, D)) / 16, t)
        u = r.uniform(*decay, D)
        self.lam, self.hlam = _dev(np.log(np.expm1(-np.log(u) / c)))
        self.off = None if offsets is None else np.asarray(offsets, np.int32)
        self.offsets = None if offsets is None else torch.from_numpy(self.off).cuda()
        self.n = 1 if offsets is None else len(offsets) - 1
        self.h0, self.hh0 = _dev(r.standard_normal((self.n, D))) if h0 else (None, None)
        self.dhT, self.hdhT = _dev(r.standard_normal((self.n, D)) / 16) if dhT else (None, None)
        self.cfg = M().config(D, max(T, 1), t, c)

    def bounds(self):
        z = self.hr, self.hi
        a, m, g, rho = orc.gates(*z, self.hlam, self.c)
        sp = orc.softplus(self.hlam)
        re = (2 * np.abs(self.hr) + 26) * U
        ea = U + re * np.abs(np.expm1(-self.c * sp * rho))
        A, Mv = V(a, ea), V(m, m * (re + 4 * U))
        Gi = V(g, g * (2 * np.abs(self.hi) + 8) * U)
        Gn = V(1 - g, (1 - g) * (2 * np.abs(self.hi) + 8) * U)
        Rh = V(rho, rho * (2 * np.abs(self.hr) + 8) * U)
        Rn = V(orc.sigmoid(-self.hr), orc.sigmoid(-self.hr) * (2 * np.abs(self.hr) + 8) * U)
        u = Mv * Gi * self.hx
        spans = [(0, self.T)] if self.off is None else list(zip(self.off[:-1], self.off[1:]))
        shape = (self.T, self.D)
        cut, last = np.zeros(self.T, bool), np.zeros(self.T, bool)
        first, behind = np.zeros(shape), np.zeros(shape)
        for k, (lo, hi) in enumerate(spans):
            if hi > lo:
                cut[lo] = last[hi - 1] = True
                if self.hh0 is not None:
                    first[lo] = self.hh0[k]
                if self.hdhT is not None:
                    behind[hi - 1] = self.hdhT[k]
        zero = np.zeros(shape)
        E, S = _scan_bound(a, ea, u.v, u.e, cut, first, zero)
        self.eh = E + 42 * U * S
        y, hT, before = orc.forward(self.hx, *z, self.hlam, self.c, self.off, self.hh0)
        eb = np.zeros(shape)
        eb[1:] = self.eh[:-1]
        eb[cut] = 0
        Hb = V(before, eb)
        # backwards the state that comes in at t is a_{t+1} G_{t+1}
        an, ean = np.zeros(shape), np.zeros(shape)
        an[:-1], ean[:-1] = a[1:], ea[1:]
        G, Eg, Sg = np.zeros(shape), np.zeros(shape), np.zeros(shape)
        gg = e = s = np.zeros(self.D)
        for t in range(self.T - 1, -1, -1):
            at, eat = an[t], ean[t]
            if last[t]:
                gg, e, s, at, eat = behind[t], 0 * e, np.abs(behind[t]), 1.0, 0.0
            G[t] = self.hdy[t] + at * gg
            Eg[t] = at * e + s * (eat + 2 * U * at)
            Sg[t] = np.abs(self.hdy[t]) + at * s
            gg, e, s = G[t], Eg[t], Sg[t]
        Gv = V(G, Eg + 42 * U * Sg)
        inside = np.zeros(self.T, bool)
        for lo, hi in spans:
            inside[lo:hi] = True
        Gv = V(Gv.v * inside[:, None], Gv.e * inside[:, None])
        with np.errstate(divide="ignore", invalid="ignore"):
            over = np.where(m > 0, a * a / m, 0.0)
        eo = over * (2 * ea / np.maximum(a, 1e-30) + re + 8 * U)
        K = V(-self.c * sp, self.c * sp * 8 * U)
        dz = A * Gv * Hb - Gv * Gi * self.hx * V(over, eo)
        out = {"dx": Gv * Mv * Gi, "di": Gv * Mv * self.hx * Gi * Gn, "dr": K * dz * Rh * Rn}
        sl = orc.sigmoid(self.hlam)
        out["dlam"] = (Rh * dz).total(self.T / 64 + 90) * V(-self.c * sl, self.c * sl * 40 * U)
        ag = A * Gv
        h0v, h0e = np.zeros((self.n, self.D)), np.zeros((self.n, self.D))
        eT = np.zeros((self.n, self.D))
        for k, (lo, hi) in enumerate(spans):
            if hi > lo:
                h0v[k], h0e[k], eT[k] = ag.v[lo], ag.e[lo], self.eh[hi - 1]
            elif self.hdhT is not None:
                h0v[k] = self.hdhT[k]
        out["dh0"] = V(h0v, h0e)
        out["y"], out["hT"] = V(y, self.eh * inside[:, None]), V(hT, eT)
        return out, inside

    def run(self, ws=None):
        m = M()
        ws = ws or m.Workspace(self.cfg)
        ws.tensor.fill_(0xFF)
        y = torch.full((self.T, self.D), 7.0, dtype=TORCH[self.t], device="cuda")
        g = {k: torch.full_like(y, 7.0) for k in ("dx", "dr", "di")}
        y, hT, saved = m.fwd(self.cfg, ws, self.x, self.r, self.i, self.lam, self.offsets, self.h0, keep=True, final=True,
                             out=y)
        ws.tensor.fill_(0xFF)
        g = m.bwd(self.cfg, ws, self.x, self.r, self.i, self.lam, saved, self.dy, self.offsets, self.h0, self.dhT, **g)
        return {"y": y, "hT": hT, **g}

    def check(self, ws=None):
        got = self.run(ws)
        b, inside = self.bounds()
        o = orc.backward(self.hx, self.hr, self.hi, self.hlam, self.c, self.hdy, self.off, self.hh0, self.hdhT)
        o["y"], o["hT"], _ = orc.forward(self.hx, self.hr, self.hi, self.hlam, self.c, self.off, self.hh0)
        assert set(got) == {"y", "hT", "dx", "dr", "di", "dlam"} | ({"dh0"} if self.h0 is not None else set())
        rows = torch.from_numpy(inside)
        for k, v in got.items():
            t = self.t if k in ("y", "dx", "dr", "di") else "f32"
            if t == self.t and v.dim() == 2 and k not in ("hT", "dh0"):
                assert (v.cpu()[~rows] == 7.0).all(), f"{k}: a row outside the sequences was written"
                v = torch.where(rows[:, None].cuda(), v, torch.zeros_like(v))
                square = o[k] ** 2
                if t == "bf16" and square.sum() ** 2 >= 256 * (square ** 2).sum() > 0:
                    off = np.linalg.norm(v.double().cpu().numpy() - o[k]) / np.sqrt(square.sum())
                    assert off <= 0.6 * 2.0 ** -8, (k, off)
            within(v, o[k], b[k], t, k)
        return got


LENGTHS = [1, 2, 7, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 511, 513, 1000]


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("T", LENGTHS)
def test_one_sequence(T, t):
    Case(T, 70, t).check()


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("D", [1, 2, 3, 63, 64, 65, 127, 128, 129, 255, 257, 768, 1001])
def test_widths(D, t):
    Case(150, D, t, [0, 40, 41, 150], h0=True, dhT=True).check()


def _pack(r, T, mean, gap=0, empty=0.2):
    out, at = [gap], gap
    while at < T - gap:
        at = min(T - gap, at + (0 if r.random() < empty else 1 + int(r.exponential(mean))))
        out.append(at)
    return out


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("mean", [0.5, 3, 20, 64, 300])
@pytest.mark.parametrize("T,gap", [(70, 0), (500, 9), (1500, 70)])
def test_packed(T, gap, mean, t):
    r = np.random.default_rng([T, int(10 * mean)])
    off = _pack(r, T, mean, gap)
    Case(T, 66, t, off, h0=True, dhT=True).check()
    Case(T, 33, t, off + [off[-1]] * 5).check()


@pytest.mark.parametrize("off", [[0, 0], [5, 5, 5], [0, 64], [64, 128], [0, 64, 128, 192], [63, 64, 65], [128, 130],
                                 [0, 0, 0, 200], [200, 200], [0, 1, 2, 3, 4]])
def test_edges_of_pieces(off):
    for t in ("f32", "bf16"):
        Case(200, 40, t, off, h0=True, dhT=True).check()


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("T", [31, 32, 33, 64, 65, 128, 129, 256, 257, 512, 513])
def test_lengths_where_pieces_change(T, t):
    """Sequences that cross the borders, with all that they may have; a workspace of a
    longer call serves, and an accumulated dlam gets every channel's sum once."""
    m = M()
    ws = m.Workspace(m.config(90, 2000, t))
    for off in ([0, T // 3, T // 3, T], [1, T - 1], [0, T]):
        c = Case(T, 90, t, off, h0=True, dhT=True)
        c.cfg.max_tokens = 2000
        got = c.check(ws)
        acc = m.config(90, 2000, t, accumulate=True)
        old = torch.full((90,), 3.0, device="cuda")
        _, _, saved = m.fwd(acc, ws, c.x, c.r, c.i, c.lam, c.offsets, c.h0, keep=True)
        m.bwd(acc, ws, c.x, c.r, c.i, c.lam, saved, c.dy, c.offsets, c.h0, c.dhT, dlam=old)
        assert torch.equal(old, got["dlam"] + 3.0)


@pytest.mark.parametrize("T", [40, 200, 600])
def test_widest(T):
    Case(T, 16384, "bf16", [0, T // 2, T], h0=True, dhT=True).check()
    Case(T, 16383, "f32").check()


@pytest.mark.parametrize("T", [20, 200, 700])
@pytest.mark.parametrize("n", [1500, 5000, 70000])
def test_more_sequences_than_positions(n, T):
    r = np.random.default_rng([n, T])
    off = np.sort(r.integers(3, T - 2, n + 1))
    Case(T, 20, "f32", off, h0=True, dhT=True).check()


@pytest.mark.parametrize("T,lo,hi", [(60, 5, 50), (200, 33, 100), (1500, 100, 1000)])
def test_padding_counts_for_nothing(T, lo, hi):
    """Whatever stands in the rows in front of the first sequence and behind the last."""
    m, D = M(), 70
    for t in ("f32", "bf16"):
        c = Case(T, D, t, [lo, (lo + hi) // 2, hi], h0=True, dhT=True)
        want = c.check()
        for v in (float("nan"), float("inf"), -float("inf")):
            for x in (c.x, c.r, c.i, c.dy):
                x[:lo], x[hi:] = v, v
            got = c.run()
            assert all(torch.equal(got[k], want[k]) for k in want), v


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("T,D,off", [(4000, 70, None), (5000, 30, [0, 4100, 5000]), (3001, 130, [0, 1, 2999, 3001])])
def test_long(T, D, off, t):
    Case(T, D, t, off, h0=True, dhT=True).check()


@pytest.mark.parametrize("decay", [(0.5, 0.6), (0.9999, 0.99999), (1e-6, 0.1)])
def test_fast_and_slow_decays(decay):
    for t in ("f32", "bf16"):
        Case(700, 50, t, decay=decay, spread=3.0, h0=True, dhT=True).check()


def test_gates_far_out():
    """r and i where their sigmoids are 0 or 1 to the last bit: nothing is NaN."""
    T, D = 130, 24
    c = Case(T, D, "f32", h0=True)
    for r, i in ((-200.0, 3.0), (200.0, -200.0), (-90.0, 200.0), (-float("inf"), float("inf")), (float("inf"), 0.0)):
        c.r.fill_(r), c.i.fill_(i)
        got = c.run()
        assert all(torch.isfinite(v).all() for v in got.values()), (r, i)
        if r == -float("inf"):   # a = 1, u = 0
            assert torch.equal(got["y"], c.h0.expand(T, D)) and (got["dr"] == 0).all() and (got["dlam"] == 0).all()


@pytest.mark.parametrize("T,off", [(300, [0, 100, 164, 300]), (2000, [0, 900, 1000, 2000])])
def test_not_finite_stays_in_its_sequence(T, off):
    D = 70
    for v in (float("nan"), float("inf")):
        c = Case(T, D, "bf16", off, h0=True, dhT=True)
        ref = c.run()
        lo, hi = off[1], off[2]
        c.x[lo + 3, 5] = v
        c.dy[hi - 2, 6] = v
        c.h0[1, 7] = v
        c.dhT[1, 8] = v
        got = c.run()
        keep = torch.ones(T, dtype=torch.bool, device="cuda")
        keep[lo:hi] = False
        for k in ("y", "dx", "dr", "di"):
            assert torch.equal(got[k][keep], ref[k][keep]), k
        ok = torch.ones(D, dtype=torch.bool, device="cuda")
        ok[5:9] = False
        for k in got:
            assert torch.equal(got[k][..., ok], ref[k][..., ok]), k
        assert not torch.isfinite(got["y"][lo + 3:hi, 5]).any() and not torch.isfinite(got["y"][lo:hi, 7]).any()
        assert not torch.isfinite(got["dx"][lo:hi - 1, 6]).any() and not torch.isfinite(got["dx"][lo:hi, 8]).any()


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_columns_of_one_projection(t):
    m, T, D = M(), 333, 100
    c = Case(T, D, t, [0, 50, 333])
    ref = c.run()
    p = torch.full((T, 3 * D + 7), float("nan"), dtype=TORCH[t], device="cuda")
    cols = [p[:, k * D + 1:(k + 1) * D + 1] for k in range(3)]
    for v, w in zip(cols, (c.x, c.r, c.i)):
        v.copy_(w)
    g = torch.full((T, 3 * D + 5), 9.0, dtype=TORCH[t], device="cuda")
    out = [g[:, k * D + 3:(k + 1) * D + 3] for k in range(3)]
    ws = m.Workspace(c.cfg)
    y, _, saved = m.fwd(c.cfg, ws, *cols, c.lam, c.offsets, keep=True)
    got = m.bwd(c.cfg, ws, *cols, c.lam, saved, c.dy, c.offsets, dx=out[0], dr=out[1], di=out[2])
    assert torch.equal(y, ref["y"])
    for k in ("dx", "dr", "di", "dlam"):
        assert torch.equal(got[k], ref[k]), k
    assert (g[:, :3] == 9.0).all() and (g[:, 3 * D + 3:] == 9.0).all()


def test_prompt_in_pieces():
    """A sequence in two calls, the state handed over, is the sequence in one."""
    m = M()
    c = Case(900, 96, "f32", h0=True)
    ws = m.Workspace(c.cfg)
    y, hT, _ = m.fwd(c.cfg, ws, c.x, c.r, c.i, c.lam, h0=c.h0, final=True)
    b, _ = c.bounds()
    for at in (1, 64, 333, 899):
        y0, h, _ = m.fwd(c.cfg, ws, c.x[:at], c.r[:at], c.i[:at], c.lam, h0=c.h0, final=True)
        y1, h, _ = m.fwd(c.cfg, ws, c.x[at:], c.r[at:], c.i[at:], c.lam, h0=h, final=True)
        lim = torch.from_numpy(2.02 * b["y"].e).cuda() + 2 * U * y.double().abs()
        assert ((torch.cat([y0, y1]) - y).double().abs() <= lim).all() and ((h - hT).double().abs() <= lim[-1:]).all()


def test_accumulates_and_no_positions():
    m = M()
    c = Case(100, 40, "bf16", [0, 60, 60, 100], h0=True, dhT=True)
    ws = m.Workspace(c.cfg)
    y, hT, saved = m.fwd(c.cfg, ws, c.x, c.r, c.i, c.lam, c.offsets, c.h0, keep=True, final=True)
    a = m.bwd(c.cfg, ws, c.x, c.r, c.i, c.lam, saved, c.dy, c.offsets, c.h0, c.dhT)
    acc = m.config(40, 100, "bf16", accumulate=True)
    old = torch.full((40,), 3.0, device="cuda")
    b = m.bwd(acc, ws, c.x, c.r, c.i, c.lam, saved, c.dy, c.offsets, c.h0, c.dhT, dlam=old)
    assert b["dlam"] is old and torch.equal(old, a["dlam"] + 3.0)
    e = Case(0, 40, "bf16", [0, 0, 0], h0=True, dhT=True)
    got = e.run()
    assert torch.equal(got["hT"], e.h0) and torch.equal(got["dh0"], e.dhT) and (got["dlam"] == 0).all()
    e = Case(0, 40, "f32")
    got = e.run()
    assert (got["hT"] == 0).all() and (got["dlam"] == 0).all()
    old.fill_(2.0)
    z = e.x.bfloat16()
    m.bwd(acc, ws, z, z, z, e.lam, torch.empty(0, 40, device="cuda"), z, dlam=old)
    assert (old == 2.0).all()
    n0 = Case(50, 40, "f32", [7])   # no sequence at all
    got = n0.run()
    assert (got["dlam"] == 0).all() and (got["y"] == 7.0).all() and (got["dx"] == 7.0).all()


def test_offsets_that_do_not_ascend_touch_nothing_else():
    """Unspecified results, but inside the buffers: guards of NaN stay."""
    m, T, D = M(), 300, 65
    for off in ([0, 200, 100, 300], [300, 0], [-5, 1000], [2 ** 31 - 1, -2 ** 31, 7], [250, 260, 10, 20, 5000]):
        c = Case(T, D, "f32", [0] * len(off), h0=True, dhT=True)
        c.offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
        bufs = {}

        def guarded(name, rows):
            bufs[name] = torch.full((rows + 4, D), 5.0, device="cuda")
            return bufs[name][2:2 + rows]

        ws = m.Workspace(c.cfg)
        y, hT, saved = m.fwd(c.cfg, ws, c.x, c.r, c.i, c.lam, c.offsets, c.h0, keep=True, final=True, out=guarded("y", T))
        saved.zero_()
        m.bwd(c.cfg, ws, c.x, c.r, c.i, c.lam, saved, c.dy, c.offsets, c.h0, c.dhT, dx=guarded("dx", T),
              dr=guarded("dr", T), di=guarded("di", T), dh0=guarded("dh0", c.n))
        torch.cuda.synchronize()
        for k, v in bufs.items():
            assert (v[:2] == 5.0).all() and (v[-2:] == 5.0).all(), k


def test_same_bits_every_time_other_streams_and_threads():
    import threading
    m = M()
    c = Case(3000, 200, "bf16", [0, 1000, 1001, 3000], h0=True, dhT=True)
    ref = c.run()
    torch.cuda.synchronize()
    bad = []

    def work():
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            ws = m.Workspace(c.cfg)
            for _ in range(4):
                y, hT, saved = m.fwd(c.cfg, ws, c.x, c.r, c.i, c.lam, c.offsets, c.h0, keep=True, final=True)
                g = m.bwd(c.cfg, ws, c.x, c.r, c.i, c.lam, saved, c.dy, c.offsets, c.h0, c.dhT)
                s.synchronize()
                if not (torch.equal(y, ref["y"]) and all(torch.equal(g[k], ref[k]) for k in g)):
                    bad.append(1)

    th = [threading.Thread(target=work) for _ in range(3)]
    [t.start() for t in th]
    [t.join() for t in th]
    assert not bad


def test_captured():
    """Replays take the offsets and values of the moment; two graphs share a workspace."""
    m, T, D = M(), 700, 96
    c = Case(T, D, "bf16", [0, 100, 700], h0=True, dhT=True)
    ws = m.Workspace(c.cfg)

    def call():
        y, hT, saved = m.fwd(c.cfg, ws, c.x, c.r, c.i, c.lam, c.offsets, c.h0, keep=True, final=True)
        return {"y": y, "hT": hT, **m.bwd(c.cfg, ws, c.x, c.r, c.i, c.lam, saved, c.dy, c.offsets, c.h0, c.dhT)}

    call()
    torch.cuda.synchronize()
    graphs, got = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(call())
    for k, off in enumerate(([0, 1, 700], [0, 640, 700], [0, 0, 700])):
        c.offsets.copy_(torch.tensor(off, dtype=torch.int32))
        c.x.copy_(torch.randn(T, D, generator=torch.Generator().manual_seed(k)))
        for g in graphs:
            g.replay()
        want = call()
        torch.cuda.synchronize()
        for h in got:
            assert all(torch.equal(h[q], want[q]) for q in want), k
        torch.randn(1 << 16, device="cuda").sum().item()


def _check_step(c, r, slots, states):
    m, n, D = M(), c.T, c.D
    st, hst = _dev(r.standard_normal((states, D)))
    sd = None if slots is None else torch.from_numpy(slots.astype(np.int32)).cuda()
    y = m.step(m.config(D, 1, c.t), c.x, c.r, c.i, c.lam, st, sd)
    oy, ost = orc.step(c.hx, c.hr, c.hi, c.hlam, 8.0, hst, slots)
    # the bound of a sequence: the slot's positions in order
    a, mm, g, rho = orc.gates(c.hr, c.hi, c.hlam, 8.0)
    re = (2 * np.abs(c.hr) + 26) * U
    ea = U + re * np.abs(np.expm1(-8.0 * orc.softplus(c.hlam) * rho))
    u = np.abs(mm * g * c.hx)
    E, S = np.zeros((states, D)), np.abs(hst)
    ey = np.zeros((n, D))
    for k in range(n):
        s = k if slots is None else slots[k]
        if 0 <= s < states:
            E[s] = a[k] * E[s] + S[s] * (ea[k] + 2 * U * a[k]) + u[k] * (re[k] + (2 * np.abs(c.hi[k]) + 14) * U)
            S[s] = a[k] * S[s] + u[k]
            ey[k] = E[s] + 2 * U * S[s]
    within(st, ost, V(ost, E + 2 * U * S), "f32", "state")
    within(y, oy, V(oy, ey), c.t, "y")


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("n,D", [(1, 768), (1, 1), (5, 65), (33, 129), (70, 768), (300, 40), (512, 9), (1100, 66)])
def test_step(n, D, t):
    r = np.random.default_rng([n, D])
    c = Case(n, D, t)
    states = n + 7
    for slots in (None, r.permutation(states)[:n], r.integers(-2, states + 2, n), np.zeros(n, int), np.full(n, -1)):
        _check_step(c, r, slots, states)


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("D", [129, 257, 258])
def test_step_of_more_rows_than_run_at_once(D, t):
    """Every channel's state moves on once, by whichever wavefront and whenever it runs."""
    r = np.random.default_rng(D)
    n = 20000
    c = Case(n, D, t)
    _check_step(c, r, None, n)
    _check_step(c, r, r.permutation(n + 50)[:n], n + 50)


def test_steps_continue_a_prompt():
    m, D = M(), 130
    c = Case(140, D, "f32", [0, 90, 140], h0=True)
    ws = m.Workspace(c.cfg)
    b, _ = c.bounds()
    y, hT, _ = m.fwd(c.cfg, ws, c.x, c.r, c.i, c.lam, c.offsets, c.h0, final=True)
    part = torch.tensor([0, 70, 120], dtype=torch.int32, device="cuda")
    rows = torch.cat([torch.arange(70), torch.arange(90, 140)]).cuda()
    _, st, _ = m.fwd(c.cfg, ws, c.x[rows], c.r[rows], c.i[rows], c.lam, part, c.h0, final=True)
    more = torch.arange(70, 90).cuda()
    # the 20 positions that the first sequence still has, as rows of one call
    slots = torch.zeros(20, dtype=torch.int32, device="cuda")
    out = m.step(c.cfg, c.x[more], c.r[more], c.i[more], c.lam, st, slots)
    lim = torch.from_numpy(2.02 * b["y"].e).cuda() + 2 * U * y.double().abs()
    assert ((out - y[70:90]).double().abs() <= lim[70:90]).all()
    assert ((st - hT).double().abs() <= torch.stack([lim[89], lim[139]])).all()


def test_gradients_against_differences():
    """dL / d(everything) of L = sum(y dy) + sum(hT dhT) along random directions."""
    m = M()
    c = Case(300, 33, "f32", [0, 130, 300], h0=True, dhT=True)
    ws = m.Workspace(c.cfg)
    got = c.run(ws)
    r = np.random.default_rng(5)

    def loss(x, rr, i, lam, h0):
        y, hT, _ = orc.forward(x, rr, i, lam, c.c, c.off, h0)
        return (y * c.hdy).sum() + (hT * c.hdhT).sum()

    base = [c.hx, c.hr, c.hi, c.hlam, c.hh0]
    for k, name in enumerate(("dx", "dr", "di", "dlam", "dh0")):
        d = r.standard_normal(base[k].shape)
        p, q = list(base), list(base)
        p[k], q[k] = base[k] + 1e-5 * d, base[k] - 1e-5 * d
        want = (loss(*p) - loss(*q)) / 2e-5
        g = got[name].double().cpu().numpy()
        # the difference's own error is 1e-10 of the third derivative's scale; fp32 sums: 1e-5 of the terms' norm
        assert abs((g * d).sum() - want) <= 1e-5 * np.linalg.norm(g) * np.linalg.norm(d) + 1e-6, name


def test_rows_past_32_bits():
    """Element offsets past 2^32: the last rows against the same rows alone."""
    m = M()
    T, D = (1 << 20) + 100, 4100
    cfg = m.config(D, T)
    ws = m.Workspace(cfg)
    x = torch.zeros(T, D, dtype=torch.bfloat16, device="cuda")
    r, i = torch.zeros_like(x), torch.zeros_like(x)
    gen = torch.Generator(device="cuda").manual_seed(3)
    for t in (x, r, i):
        t[-100:].normal_(generator=gen)
    lam = torch.full((D,), -4.0, device="cuda")
    off = torch.tensor([0, T - 100, T], dtype=torch.int32, device="cuda")
    y, _, saved = m.fwd(cfg, ws, x, r, i, lam, off, keep=True)
    assert (y[:1000] == 0).all() and (y[-1100:-100] == 0).all()
    dy = x
    g = m.bwd(cfg, ws, x, r, i, lam, saved, dy, off)
    tail = [v[-100:].contiguous() for v in (x, r, i)]
    y2, _, s2 = m.fwd(cfg, ws, *tail, lam, keep=True)
    g2 = m.bwd(cfg, ws, *tail, lam, s2, tail[0])
    # two roundings to bf16 of values that differ by fp32 sums' errors: a step apart at most
    for p, q in ((y, y2), *((g[k], g2[k]) for k in ("dx", "dr", "di"))):
        p, q = p[-100:].double(), q.double()
        assert (q.abs().sum(1) > 0).all() and ((p - q).abs() <= 2.0 ** -7 * q.abs() + 1e-5 * q.abs().max()).all()
