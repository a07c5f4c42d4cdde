"""GPU parity of the gated feed-forward block (include/ffn.h) against the
float64 oracle, through the C ABI.

Whole-number cases: X has two non-zero entries of +-1 a row, the weights are in
{-1, 0, 1}, dY is sparse, the activation is relu2 and a dropout of p = 1/2
scales by 2.  Every G, U lies in [-2, 2], every H, dG, dU is a whole number of
at most 256 (checked on the oracle's), which bf16 holds, and every sum is below
2^24: the results are exact, whatever the tiling, the order of the sums or the
parts of k, and are compared for equality.

Real-valued cases: with u = 2^-24 and b = 2^-8 (half a bf16 step)
  eG = 768 u |X| |Wg|^T, eU alike           (fp32 sums of exact products)
  ea = (|a'| + 2 eG) eG + 2^-19 (|a| + |g| 2^-4)      a'' is at most 2; the fast
       exp's argument is off by u |g| and the exp, sum, reciprocal and product
       by a few u: 2^-19 relative holds to |g| of 16
  ea' = 2 eG + 2^-19 (1 + |g|)               the same for the derivative
  eH = ea |U| + |a| eU + ea eU + b |H|       (rounded once)
  e(dH) = 768 u |dY'| |Wd| (+ b |dY'| |Wd| where dY was fp32)
  e(dU) = e(dH) |a| + |dH| ea + e(dH) ea + b |dU|
  e(dG) = e(dH) |U a'| + |dH| (eU |a'| + |U| ea' + eU ea') + b |dG|   (first order, and 1 %)
and each product C = A B carries eA |B| + |A| eB + K u |A| |B|.  The result's
own rounding is u or b of it.  These are worst cases, so the errors' 2-norm is
held too: independent roundings have at most b / sqrt(3) of the value each, and
an output sees two (its operand's, its own) or, for dWd of an fp32 dY and for
all of an fp32 dY's gradients, three: sqrt(3) b / sqrt(3) = b of the norm.
"""
import numpy as np
import pytest
import torch

from oracle import drop as orcd
from oracle import ffn as orc

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
B = 2.0 ** -8
NAMES = ("dX", "dWg", "dWu", "dWd")


def M():
    from sparse_hashed_gram_amd import ffn
    return ffn


def D():
    from sparse_hashed_gram_amd import drop
    return drop


def _bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16)


def _f64(t):
    return t.detach().float().cpu().double().numpy()


def _same(got, want, name):
    g = _f64(got)
    at = np.argwhere(~(g == want))
    if len(at):
        i = tuple(at[0])
        pytest.fail(f"{name}: {len(at)} of {g.size} differ, first at {i}: {g[i]} instead of {want[i]}; last at {tuple(at[-1])}")


# ----------------------------------------------------- whole numbers: exact

def _whole(T, F, seed):
    r = np.random.default_rng([T, F, seed])
    X = np.zeros((T, 768))
    for _ in range(2):
        X[np.arange(T), r.integers(0, 768, T)] = r.choice([-1.0, 1.0], T)
    W = [r.integers(-1, 2, s).astype(np.float64) for s in ((F, 768), (F, 768), (768, F))]
    dY = r.integers(-1, 2, (T, 768)) * (r.random((T, 768)) < 0.03)
    res = r.integers(-3, 4, (T, 768)).astype(np.float64)
    return X, W, dY.astype(np.float64), res


def _run_whole(T, F, p, max_tokens=None, accumulate=False, ws=None):
    m = M()
    X, W, dY, res = _whole(T, F, 0)
    cfg = m.config(F, max_tokens or max(T, 1), act="relu2", y_dtype="f32", dw_dtype="f32", accumulate=accumulate)
    ws = ws or m.Workspace(cfg)
    seed, off = 1234567 + T, (9 << 32) + F
    spec = D().spec(p, seed, off) if p else None
    factor = orcd.keep(T, 768, p, seed, off) * 2.0 if p else None
    Xd, Wd_ = _bf16(X).cuda(), [_bf16(w).cuda() for w in W]
    dYd, resd = torch.from_numpy(dY).float().cuda(), torch.from_numpy(res).float().cuda()
    y = m.fwd(cfg, ws, Xd, *Wd_, residual=resd, drop=spec)
    _same(y, orc.forward(X, *W, "relu2", factor, res), "Y")
    old = {k: torch.full(s, 5.0, device="cuda") for k, s in zip(NAMES[1:], ((F, 768), (F, 768), (768, F)))}
    g = m.bwd(cfg, ws, Xd, *Wd_, dYd, drop=spec, **(old if accumulate else {}))
    o = orc.backward(X, *W, dY, "relu2", factor)
    for k in NAMES:
        _same(g[k], o[k] + (5.0 if accumulate and k != "dX" else 0.0), k)
    a, da = orc.act(X @ W[0].T, "relu2")
    dH = (dY if factor is None else dY * factor) @ W[2]
    u = X @ W[1].T
    for v in (a * u, dH * a, dH * u * da):
        assert np.abs(v).max(initial=0) <= 256, "the case is not exact"
    return g, y


@pytest.mark.parametrize("T", [1, 2, 3, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 200, 257])
@pytest.mark.parametrize("F,p", [(8, 0.0), (72, 0.5), (64, 0.0), (200, 0.5), (1000, 0.0), (2056, 0.5)])
def test_whole_numbers(T, F, p):
    _run_whole(T, F, p)


@pytest.mark.parametrize("T,F,p", [(1000, 2048, 0.5), (2049, 264, 0.0), (3001, 2056, 0.5), (4096, 128, 0.0),
                                   (9000, 640, 0.5), (513, 8192, 0.0), (300, 65536, 0.0), (20000, 8, 0.5)])
def test_whole_numbers_larger(T, F, p):
    _run_whole(T, F, p)


@pytest.mark.parametrize("T,F,p", [(1, 65536, 0.0), (1, 8192, 0.5), (1, 8200, 0.0), (20, 12288, 0.5), (32, 8192, 0.0),
                                   (12, 8192, 0.5), (13, 8192, 0.0), (4, 2048, 0.5), (4, 2056, 0.0),
                                   (33, 1984, 0.5), (33, 1992, 0.0), (64, 1024, 0.5), (64, 1032, 0.0), (49, 1336, 0.0)])
def test_whole_numbers_few_positions(T, F, p):
    # either side of the rules that pick the kernels of few positions and of few values
    _run_whole(T, F, p, max_tokens=T + 3)


def test_whole_numbers_accumulate_and_a_roomy_workspace():
    _run_whole(333, 520, 0.5, max_tokens=5000, accumulate=True)
    _run_whole(70, 520, 0.0, max_tokens=5000, accumulate=True)


def test_one_workspace_for_several_sizes_and_rows_behind():
    # nothing of a larger call shows in a smaller one, and no row behind T changes
    m = M()
    cfg = m.config(2056, 3001, act="relu2", y_dtype="f32", dw_dtype="f32")
    ws = m.Workspace(cfg)
    ws.tensor.fill_(255)                       # NaN in every format
    for T in (3001, 5, 700, 1):
        X, W, dY, res = _whole(T, 2056, 1)
        Wc = [_bf16(w).cuda() for w in W]
        Y = torch.full((T + 40, 768), 9.0, device="cuda")
        dX = torch.full((T + 40, 768), 9.0, device="cuda")
        m.fwd(cfg, ws, _bf16(X).cuda(), *Wc, out=Y[:T])
        _same(Y[:T], orc.forward(X, *W, "relu2"), f"Y at {T}")
        assert torch.all(Y[T:] == 9)
        g = m.bwd(cfg, ws, _bf16(X).cuda(), *Wc, torch.from_numpy(dY).float().cuda(), dX=dX[:T])
        o = orc.backward(X, *W, dY, "relu2")
        for k in NAMES:
            _same(g[k], o[k], f"{k} at {T}")
        assert torch.all(dX[T:] == 9)


# ------------------------------------------------------------- real values

def _real(T, F, seed=0):
    r = np.random.default_rng([T, F, seed, 7])
    q = lambda a: _bf16(a).float().numpy().astype(np.float64)   # noqa: E731
    X = q(r.standard_normal((T, 768)))
    Wg, Wu = (q(r.standard_normal((F, 768)) * 768 ** -0.5) for _ in range(2))
    Wd = q(r.standard_normal((768, F)) * F ** -0.5)
    return X, [Wg, Wu, Wd], q(r.standard_normal((T, 768)) / 64), q(r.standard_normal((T, 768)))


def _bounds(X, W, dY, kind, factor, dy_rounded):
    """{name: (oracle, bound on the fp32 result before its own rounding)}"""
    Wg, Wu, Wd = W
    ab = np.abs
    G, Uu = X @ Wg.T, X @ Wu.T
    eG, eU = 768 * U * ab(X) @ ab(Wg).T, 768 * U * ab(X) @ ab(Wu).T
    a, da = orc.act(G, kind)
    ea = (ab(da) + 2 * eG) * eG + 2.0 ** -19 * (ab(a) + ab(G) / 16)
    eda = 2 * eG + 2.0 ** -19 * (1 + ab(G))
    H = a * Uu
    eH = ea * ab(Uu) + ab(a) * eU + ea * eU
    eH = eH + B * (ab(H) + eH)
    F = H.shape[1]
    y = H @ Wd.T
    ey = eH @ ab(Wd).T + (F + 64) * U * (ab(H) + eH) @ ab(Wd).T
    if factor is not None:
        y, ey = y * factor, ey * factor + U * 2 * ab(y * factor)
        dY = dY * factor
    out = {"Y": (y, ey)}
    edY = B * ab(dY) if dy_rounded else np.zeros_like(dY)
    edY = edY + 2 * U * ab(dY)     # the scale, in fp32
    dH = dY @ Wd
    edH = edY @ ab(Wd) + 768 * U * ab(dY) @ ab(Wd)
    dU, dG = dH * a, dH * Uu * da
    edU = edH * ab(a) + ab(dH) * ea + edH * ea
    edU = edU + B * (ab(dU) + edU)
    edG = 1.01 * (edH * ab(Uu * da) + ab(dH) * (eU * ab(da) + ab(Uu) * eda + eU * eda))
    edG = edG + B * (ab(dG) + edG)
    T = X.shape[0]
    out["dX"] = (dG @ Wg + dU @ Wu, edG @ ab(Wg) + edU @ ab(Wu)
                 + (2 * F + 128) * U * ((ab(dG) + edG) @ ab(Wg) + (ab(dU) + edU) @ ab(Wu)))
    for k, v, e in (("dWg", dG, edG), ("dWu", dU, edU)):
        out[k] = (v.T @ X, e.T @ ab(X) + (T + 64) * U * (ab(v) + e).T @ ab(X))
    out["dWd"] = (dY.T @ H, ab(dY).T @ eH + edY.T @ (ab(H) + eH) + (T + 64) * U * ab(dY).T @ (ab(H) + eH))
    return out


def _hold(got, o, e, bf16, name):
    g = _f64(got)
    e = e + (B if bf16 else 2 * U) * (np.abs(o) + e)
    err = np.abs(g - o)
    assert not np.any(np.isnan(g)) and np.all(err <= e), (name, float((err / np.maximum(e, 1e-300)).max()))
    if o.size >= 1000:
        assert np.linalg.norm(g - o) <= B * np.linalg.norm(o), name


@pytest.mark.parametrize("kind", ["silu", "gelu", "relu2"])
@pytest.mark.parametrize("T,F,p,yt,wt", [(1, 2048, 0.0, "bf16", "bf16"), (7, 1000, 0.3, "f32", "f32"),
                                         (130, 520, 0.0, "bf16", "f32"), (300, 2056, 0.1, "bf16", "bf16"),
                                         (1025, 320, 0.5, "f32", "bf16")])
def test_real_values(T, F, p, yt, wt, kind):
    m = M()
    X, W, dY, res = _real(T, F)
    cfg = m.config(F, T, act=kind, y_dtype=yt, dw_dtype=wt)
    ws = m.Workspace(cfg)
    spec = D().spec(p, 5, 6) if p else None
    factor = orcd.keep(T, 768, p, 5, 6) * (65536 / (65536 - orcd.threshold(p))) if p else None
    td = torch.float32 if yt == "f32" else torch.bfloat16
    Xd, Wd_ = _bf16(X).cuda(), [_bf16(w).cuda() for w in W]
    o = _bounds(X, W, dY, kind, factor, yt == "f32")
    y = m.fwd(cfg, ws, Xd, *Wd_, drop=spec)
    _hold(y, *o["Y"], yt == "bf16", "Y")
    yr = m.fwd(cfg, ws, Xd, *Wd_, residual=torch.from_numpy(res).to(td).cuda(), drop=spec)
    _hold(yr, o["Y"][0] + res, o["Y"][1] + 2 * U * np.abs(res), yt == "bf16", "Y + res")
    g = m.bwd(cfg, ws, Xd, *Wd_, torch.from_numpy(dY).to(td).cuda(), drop=spec)
    for k in NAMES:
        assert g[k].dtype == (td if k == "dX" else torch.float32 if wt == "f32" else torch.bfloat16)
        _hold(g[k], *o[k], g[k].dtype == torch.bfloat16, k)


@pytest.mark.parametrize("kind", ["silu", "gelu", "relu2"])
@pytest.mark.parametrize("T,F", [(1, 128), (1, 2048), (1, 8192), (2, 424), (3, 2056), (7, 136), (16, 512), (17, 480), (32, 256), (31, 128)])
def test_few_positions_round_once(T, F, kind):
    # H, dG and dU keep 16 bits here, so a result's own rounding, of 2^-8 / sqrt(3) of the
    # value at most on average, is what is left: with it the operands' 2^-17 and
    # the fp32 sums (2^-24 times a few hundred).  A root of n values' squares strays
    # from its expectation by about 1 / sqrt(n) of it, n at least 768 here, and a
    # rounding's is well below its most: for mantissas spread evenly 0.7 of it.
    m, d = M(), D()
    X, W, dY, _ = _real(T, F, 50)
    cfg = m.config(F, T, act=kind)
    ws, spec = m.Workspace(cfg), d.spec(0.2, 3, 4)
    factor = orcd.keep(T, 768, 0.2, 3, 4) * (65536 / (65536 - orcd.threshold(0.2)))
    Xd, Wc = _bf16(X).cuda(), [_bf16(w).cuda() for w in W]
    got = {"Y": m.fwd(cfg, ws, Xd, *Wc, drop=spec), **m.bwd(cfg, ws, Xd, *Wc, _bf16(dY).cuda(), drop=spec)}
    want = {"Y": orc.forward(X, *W, kind, factor), **orc.backward(X, *W, dY, kind, factor)}
    for k, v in want.items():
        assert np.linalg.norm(_f64(got[k]) - v) <= (B / np.sqrt(3) + 2.0 ** -12) * np.linalg.norm(v), k


def test_few_positions_past_the_largest_bf16():
    # G = 2^43, U = 2^42 (1 - 2^-10): H = 2^128 (1 - 2^-10) is finite in fp32 and
    # rounds to infinity in bf16; what that leaves is taken as 0, not as -infinity
    m = M()
    F = 64
    X, Wg, Wu = (np.zeros((n, 768)) for n in (2, F, F))
    X[:, 0], X[:, 1] = 2.0 ** 43, 2.0 ** 33
    Wg[:, 0] = 1.0
    Wu[:, 0], Wu[:, 1] = 0.498046875, 1.5
    cfg = m.config(F, 2, act="relu2", y_dtype="f32")
    y = m.fwd(cfg, m.Workspace(cfg), *(_bf16(a).cuda() for a in (X, Wg, Wu, np.ones((768, F)))))
    assert torch.all(torch.isinf(y) & (y > 0))


def test_gradients_against_differences_of_the_forward():
    # along a random direction, with fp32 results: the forward's own rounding of H
    # (2^-8 of it) is the noise, so the step is large and the check coarse
    m = M()
    T, F = 64, 256
    X, W, dY, _ = _real(T, F, 3)
    cfg = m.config(F, T, act="silu", y_dtype="f32", dw_dtype="f32")
    ws = m.Workspace(cfg)
    dev = lambda a: _bf16(a).cuda()   # noqa: E731
    g = m.bwd(cfg, ws, dev(X), *map(dev, W), torch.from_numpy(dY).float().cuda())
    r = np.random.default_rng(5)
    for i, k in enumerate(NAMES):
        args = [X, *W]
        V = r.standard_normal(args[i].shape) * np.abs(args[i]).mean() * 0.25
        ends = []
        for sgn in (1, -1):
            moved = list(args)
            moved[i] = _f64(_bf16(args[i] + sgn * V))
            ends.append((moved[i], (_f64(m.fwd(cfg, ws, *map(dev, moved))) * dY)))
        step = ends[0][0] - ends[1][0]
        want = (_f64(g[k]) * step).sum()
        scale = np.linalg.norm(_f64(g[k]) * step) + 1e-12
        # oracle's own difference over the same step: curvature is the oracle's to say
        o = [orc.forward(*[e[0] if j == i else args[j] for j in range(4)], "silu") * dY for e in ends]
        curve = abs((o[0] - o[1]).sum() - (orc.backward(*args, dY, "silu")[k] * step).sum())
        noise = 2 * B * np.linalg.norm(o[0])
        assert abs((ends[0][1] - ends[1][1]).sum() - want) <= curve + 4 * noise + 4 * B * scale, k


def test_no_positions():
    m = M()
    cfg = m.config(64, 8)
    ws = m.Workspace(cfg)
    z = lambda *s: torch.ones(*s, dtype=torch.bfloat16, device="cuda")   # noqa: E731
    W = [z(64, 768), z(64, 768), z(768, 64)]
    assert m.fwd(cfg, ws, z(0, 768), *W).shape == (0, 768)
    g = m.bwd(cfg, ws, z(0, 768), *W, z(0, 768), dWg=z(64, 768), dWu=z(64, 768), dWd=z(768, 64))
    assert g["dX"].shape == (0, 768) and all(torch.count_nonzero(g[k]) == 0 for k in NAMES[1:])
    cfg = m.config(64, 8, accumulate=True)
    g = m.bwd(cfg, ws, z(0, 768), *W, z(0, 768), dWg=z(64, 768), dWu=z(64, 768), dWd=z(768, 64))
    assert all(torch.all(g[k] == 1) for k in NAMES[1:])
    with pytest.raises(ValueError, match="accumulating"):
        m.bwd(cfg, ws, z(0, 768), *W, z(0, 768))


def test_nan_and_inf_stay_in_their_rows():
    # a row of NaN or Inf reaches its own Y row and dX row, no other
    m = M()
    T, F = 150, 264
    X, W, dY, _ = _real(T, F, 4)
    Xd, Wc = _bf16(X).cuda(), [_bf16(w).cuda() for w in W]
    for kind in ("silu", "gelu", "relu2"):
        cfg = m.config(F, T, act=kind)
        ws = m.Workspace(cfg)
        clean = m.fwd(cfg, ws, Xd, *Wc)
        cdx = m.bwd(cfg, ws, Xd, *Wc, _bf16(dY).cuda())["dX"]
        for row, val in ((0, float("nan")), (149, float("inf")), (64, float("-inf"))):
            bad = Xd.clone()
            bad[row, 3] = val
            y = m.fwd(cfg, ws, bad, *Wc)
            dx = m.bwd(cfg, ws, bad, *Wc, _bf16(dY).cuda())["dX"]
            rest = [t for t in range(T) if t != row]
            assert torch.equal(y[rest], clean[rest]) and torch.equal(dx[rest], cdx[rest])
            assert torch.any(~torch.isfinite(y[row]))


@pytest.mark.parametrize("T,F", [(1, 2048), (40, 520), (2500, 1032)])
def test_bitwise_repeatable_and_on_another_stream(T, F):
    m = M()
    X, W, dY, res = _real(T, F, 6)
    Xd, Wc, dYd, rd = _bf16(X).cuda(), [_bf16(w).cuda() for w in W], _bf16(dY).cuda(), _bf16(res).cuda()
    cfg = m.config(F, T)
    ws, spec = m.Workspace(cfg), D().spec(0.2, 1, 2)
    y = m.fwd(cfg, ws, Xd, *Wc, residual=rd, drop=spec)
    g = m.bwd(cfg, ws, Xd, *Wc, dYd, drop=spec)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ws2 = m.Workspace(cfg)
        inplace = rd.clone()
        y2 = m.fwd(cfg, ws2, Xd, *Wc, residual=inplace, drop=spec, out=inplace)
        g2 = m.bwd(cfg, ws2, Xd, *Wc, dYd, drop=spec)
    side.synchronize()
    assert y2 is inplace and torch.equal(y, y2)
    assert all(torch.equal(g[k], g2[k]) for k in NAMES)


def test_two_streams_at_once():
    # calls of different sizes and masks in flight together, each with its workspace
    m, d = M(), D()
    jobs = []
    for i, (T, F) in enumerate(((1500, 1032), (70, 2048), (4100, 256), (9, 520))):
        X, W, dY, _ = _real(T, F, 30 + i)
        cfg = m.config(F, T)
        jobs.append((cfg, m.Workspace(cfg), _bf16(X).cuda(), [_bf16(w).cuda() for w in W], _bf16(dY).cuda(),
                     d.spec(0.3, i, 5), torch.cuda.Stream()))
    want = [(m.fwd(c, ws, X, *W, drop=s), m.bwd(c, ws, X, *W, dY, drop=s)) for c, ws, X, W, dY, s, _ in jobs]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for c, ws, X, W, dY, s, st in jobs:
            with torch.cuda.stream(st):
                got.append((m.fwd(c, ws, X, *W, drop=s), m.bwd(c, ws, X, *W, dY, drop=s)))
        torch.cuda.synchronize()
        for (y, g), (y0, g0) in zip(got, want):
            assert torch.equal(y, y0) and all(torch.equal(g[k], g0[k]) for k in NAMES)


def test_graph_replays():
    m, d = M(), D()
    T, F = 333, 520
    cfg = m.config(F, T, y_dtype="f32", dw_dtype="f32", accumulate=True)
    ws = m.Workspace(cfg)
    rng = d.rng_state(0, 0)
    spec = d.spec(0.25, rng=rng)
    X, W, dY, _ = _real(T, F, 8)
    Xd, Wc, dYd = _bf16(X).cuda(), [_bf16(w).cuda() for w in W], torch.from_numpy(dY).float().cuda()
    y, dX = torch.empty(T, 768, device="cuda"), torch.empty(T, 768, device="cuda")
    dW = [torch.zeros(s, device="cuda") for s in ((F, 768), (F, 768), (768, F))]

    def step():
        m.fwd(cfg, ws, Xd, *Wc, drop=spec, out=y)
        m.bwd(cfg, ws, Xd, *Wc, dYd, spec, dX, *dW)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for w in dW:
        w.zero_()
    ref = [torch.zeros_like(w) for w in dW]
    ws2 = m.Workspace(cfg)
    for i in range(3):
        Xd.copy_(_bf16(_real(T, F, 20 + i)[0]))
        d.rng_state(i, 77, out=rng)
        g.replay()
        torch.cuda.synchronize()
        s = d.spec(0.25, i, 77)
        assert torch.equal(y, m.fwd(cfg, ws2, Xd, *Wc, drop=s))
        e = m.bwd(cfg, ws2, Xd, *Wc, dYd, s, None, *ref)
        assert torch.equal(dX, e["dX"])
        assert all(torch.equal(a, b) for a, b in zip(dW, ref))


def test_refusals_on_the_gpu():
    m = M()
    cfg = m.config(64, 16)
    ws = m.Workspace(cfg, backward=False)
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")   # noqa: E731
    X, W = z(16, 768), [z(64, 768), z(64, 768), z(768, 64)]
    assert torch.count_nonzero(m.fwd(cfg, ws, X, *W)) == 0
    with pytest.raises(m.FfnError) as e:
        m.bwd(cfg, ws, X, *W, z(16, 768))         # a forward's workspace
    assert e.value.status == -4
    with pytest.raises(m.FfnError) as e:
        m.fwd(cfg, ws, z(17, 768), *W)
    assert e.value.status == -4
    with pytest.raises(ValueError, match="Wd must have shape"):
        m.fwd(cfg, ws, X, W[0], W[1], z(64, 768))
    with pytest.raises(ValueError, match="contiguous"):
        m.fwd(cfg, ws, X, W[0], W[1], z(64, 768).t())
    with pytest.raises(TypeError, match="X must be"):
        m.fwd(cfg, ws, X.float(), *W)
    with pytest.raises(TypeError, match="residual"):
        m.fwd(cfg, ws, X, *W, residual=X.float())
    with pytest.raises(ValueError, match="residual must have shape"):
        m.fwd(cfg, ws, X, *W, residual=z(15, 768))
    with pytest.raises(m.FfnError) as e:
        m.fwd(cfg, ws, X, *W, out=X)
    assert e.value.status == -5
    flat = torch.zeros(16 * 768 + 4, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(m.FfnError) as e:
        m.fwd(cfg, ws, flat[4:].view(16, 768), *W)  # 8-byte aligned
    assert e.value.status == -2


def test_offsets_past_32_bits():
    # H has 2.2e9 elements, dG | dU | H three times as many (12.9 GB): exact, as
    # above, on the first and last positions; dY is 0 on all others, so the
    # weights' gradients are theirs alone
    m = M()
    T, F, k = 33_000, 65_536, 5
    at = np.r_[0:k, T - k:T]
    r = np.random.default_rng(9)
    X, W, _, _ = _whole(T, 8, 3)
    W = [r.integers(-1, 2, s).astype(np.float64) for s in ((F, 768), (F, 768), (768, F))]
    dY = np.zeros((T, 768))
    dY[at] = r.integers(-1, 2, (2 * k, 768)) * (r.random((2 * k, 768)) < 0.03)
    cfg = m.config(F, T, act="relu2", y_dtype="f32", dw_dtype="f32")
    ws = m.Workspace(cfg)
    Xd, Wc = _bf16(X).cuda(), [_bf16(w).cuda() for w in W]
    y = m.fwd(cfg, ws, Xd, *Wc)
    _same(y[at], orc.forward(X[at], *W, "relu2"), "Y")
    g = m.bwd(cfg, ws, Xd, *Wc, torch.from_numpy(dY).float().cuda())
    o = orc.backward(X[at], *W, dY[at], "relu2")
    _same(g["dX"][at], o["dX"], "dX")
    assert torch.count_nonzero(g["dX"][k:T - k]) == 0
    for n in NAMES[1:]:
        _same(g[n], o[n], n)
