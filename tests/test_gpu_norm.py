"""GPU parity of the norms around a block (include/norm.h) against the float64
oracle, through the C ABI.

Tolerances (bounds.py carries them from operation to operation; u = 2^-24):
- a row's sum passes a term through at most 4 P = 16 additions in its lane, 4 + 2
  across the wavefront and 3 across the row's wavefronts, and one product with
  1/D (itself rounded): 28 u of the sum of the terms' magnitudes;
- rho: half the relative error of the mean square, and 4 u of the reciprocal root;
- sigmoid(x): exp's argument x log2(e) is rounded (|x| u), exp, sum, reciprocal and
  product a few u: (2 |x| + 8) u; its derivative has one more product and twice the
  reciprocal's error: (2 |x| + 14) u;
- sums over t: a wavefront adds its own rows one by one (at most T / 2048 + 1, or T /
  512 + 1 where a block takes a row), then four wavefronts, 512 / 16 parts and 16
  threads: T / 512 + 64.
"""
import numpy as np
import pytest
import torch

from bounds import U, V, within
from oracle import norm as orc

pytestmark = pytest.mark.gpu

EPS = 1e-6
ROW = 28
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}
TYPES = [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")]


def N():
    from sparse_hashed_gram_amd import norm
    return norm


def _dev(a, t):
    """(the tensor, its values in float64)."""
    if a is None:
        return None, None
    x = torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(TORCH[t])
    return x.cuda(), x.double().numpy()


def _norm_v(x: V, kind, eps):
    if kind == "layer":
        x = x - x.mean(ROW)
    q = (x * x).mean(ROW)
    rho = 1.0 / np.sqrt(q.v + eps)
    rho = V(rho, rho * (0.5 * q.e / (q.v + eps) + 4 * U))
    return x * rho, rho


def _affine_v(x, w, b):
    y = x if w is None else x * w
    return y if b is None else y + b


def _sig_v(g):
    s = orc.sigmoid(g)
    return V(s, (2 * np.abs(g) + 8) * U * s)


def _slope_v(g):
    s = orc.sigmoid(g) * orc.sigmoid(-g)
    return V(s, (2 * np.abs(g) + 14) * U * s)


def _through_v(xh, rho, d, kind):
    out = d - xh * (d * xh).mean(ROW)
    if kind == "layer":
        out = out - d.mean(ROW)
    return rho * out


def _steps(T):
    return T / 512 + 64


class Case:
    def __init__(self, T, D, kind, types, gate="none", scale="none", weights=True, bias=True, pre=True, post=True,
                 p="f32", seed=0, eps=EPS):
        r = np.random.default_rng([T, D, seed])
        self.T, self.D, self.kind, self.eps = T, D, kind, eps
        self.x, self.r, self.p = *types, p
        self.gate_by, self.scale_by, self.pre, self.post = gate, scale, pre, post
        n = lambda *s: r.standard_normal(s)   # noqa: E731
        self.dev, self.h = {}, {}

        def put(name, a, t):
            self.dev[name], self.h[name] = _dev(a, t)

        put("R", n(T, D) * 2 + 0.5, self.r)
        put("B", n(T, D) * 0.5 - 0.25, self.x)
        put("dX", n(T, D) / 16, self.x)
        put("dR1", n(T, D) / 16, self.r)
        put("w", 1 + 0.1 * n(D) if weights and pre else None, p)
        put("b", 0.3 * n(D) if bias and pre else None, p)
        put("post_w", 1 + 0.1 * n(D) if weights and post else None, p)
        put("post_b", 0.3 * n(D) if bias and post else None, p)
        put("gate", {"none": None, "scalar": n(1), "vector": n(D), "token": 2 * n(T, D)}[gate],
            self.x if gate == "token" else p)
        put("scale", {"none": None, "scalar": 0.9 + 0.1 * n(1), "vector": 0.9 + 0.1 * n(D)}[scale], p)

    def cfg(self, **kw):
        return N().config(self.D, self.kind, self.x, self.r, p_dtype=self.p, gate=self.gate_by, scale=self.scale_by,
                          pre=self.pre, post=self.post, eps=self.eps, **kw)

    def params(self):
        return {k: self.dev[k] for k in ("post_w", "post_b", "gate", "scale", "w", "b")}

    def oracle(self):
        return {"post": self.post, "token": self.gate_by == "token",
                **{k: self.h[k] for k in ("post_w", "post_b", "gate", "scale", "w")}}

    def gamma(self):
        return V(1.0) if self.h["gate"] is None else _sig_v(self.h["gate"]) if self.gate_by == "token" else V(self.h["gate"])


def _check_plain(c: Case):
    n, h, d = N(), c.h, c.dev
    cfg = c.cfg()
    X = n.fwd(cfg, d["R"], d["w"], d["b"])
    xh, rho = _norm_v(V(h["R"]), c.kind, c.eps)
    within(X, orc.forward(h["R"], c.kind, c.eps, h["w"], h["b"]), _affine_v(xh, h["w"], h["b"]), c.x, "X")
    ws = n.Workspace(cfg)
    ws.tensor.fill_(0xFF)   # NaN
    g = n.bwd(cfg, ws, d["R"], d["dX"], d["w"], d["b"], dR1=d["dR1"])
    o = orc.backward(h["R"], h["dX"], c.kind, c.eps, h["w"], h["dR1"])
    dX = V(h["dX"])
    within(g["dR"], o["dR"], V(h["dR1"]) + _through_v(xh, rho, _affine_v(dX, h["w"], None), c.kind), c.r, "dR")
    assert set(g) == {"dR"} | ({"dw"} if d["w"] is not None else set()) | ({"db"} if d["b"] is not None else set())
    if "dw" in g:
        within(g["dw"], o["dw"], (dX * xh).total(_steps(c.T)), "f32", "dw")
    if "db" in g:
        within(g["db"], o["db"], dX.total(_steps(c.T)), "f32", "db")


def _check_join(c: Case, dp="f32"):
    n, h, d = N(), c.h, c.dev
    cfg = c.cfg(dp_dtype=dp)
    R1, X = n.join_fwd(cfg, d["R"], d["B"], **c.params())
    o1, oX = orc.join(h["R"], h["B"], c.kind, c.eps, b=h["b"], **c.oracle())
    nh, rho = _norm_v(V(h["B"]), c.kind, c.eps) if c.post else (V(h["B"]), V(1.0))
    NN = _affine_v(nh, h["post_w"], h["post_b"])
    s = V(1.0 if h["scale"] is None else h["scale"])
    r1 = s * h["R"] + c.gamma() * NN
    within(R1, o1, r1, c.r, "R1")
    if c.pre:
        within(X, oX, _affine_v(_norm_v(r1, c.kind, c.eps)[0], h["w"], h["b"]), c.x, "X")
    else:
        assert X is None
    # backwards from R1 as it was stored
    h1 = R1.double().cpu().numpy()
    ws = n.Workspace(cfg)
    ws.tensor.fill_(0xFF)
    g = n.join_bwd(cfg, ws, d["R"], d["B"], R1, d["dX"], d["dR1"], **c.params())
    o = orc.join_backward(h["R"], h["B"], h1, h["dX"], h["dR1"], c.kind, c.eps, pre=c.pre, **c.oracle())
    k = _steps(c.T)
    want = {}
    E = V(h["dR1"])
    if c.pre:
        xh, rho1 = _norm_v(V(h1), c.kind, c.eps)
        dX = V(h["dX"])
        E = E + _through_v(xh, rho1, _affine_v(dX, h["w"], None), c.kind)
        want["dw"], want["db"] = (dX * xh).total(k), dX.total(k)
    want["dR"] = E * s
    if h["scale"] is not None:
        er = E * h["R"]
        want["dscale"] = er.all(k + 30) if c.scale_by == "scalar" else er.total(k)
    gam = c.gamma()
    dN = E * gam
    if c.gate_by == "token":
        want["dgate"] = E * NN * _slope_v(h["gate"])
    elif c.gate_by != "none":
        # summed as post_w sum(E nh) + post_b sum(E): the magnitudes of both sums count
        en = E * nh
        parts = V(np.abs(en.v), en.e)
        e0 = parts.total(k)
        v = (E * NN).total(k)
        pw = 1.0 if h["post_w"] is None else np.abs(h["post_w"])
        lim = pw * e0.e + 3 * U * pw * e0.v
        if c.post and h["post_b"] is not None:
            z = V(np.abs(E.v), E.e).total(k)
            lim = lim + np.abs(h["post_b"]) * (z.e + 3 * U * z.v)
        want["dgate"] = V(v.v, lim)
        if c.gate_by == "scalar":
            want["dgate"] = V(v.v.sum(keepdims=True).reshape(1), (lim.sum() + 30 * U * np.abs(v.v).sum()).reshape(1))
    if c.post:
        # a vector's gate multiplies the sums, a token's their terms: one rounding more or less
        want["dpost_w"], want["dpost_b"] = (dN * nh).total(k + 1), dN.total(k + 1)
        want["dB"] = _through_v(nh, rho, _affine_v(dN, h["post_w"], None), c.kind)
    else:
        want["dB"] = dN
    names = {"dR", "dB"} | {"d" + q for q in ("post_w", "post_b", "gate", "scale", "w", "b") if d[q] is not None}
    assert set(g) == names
    for q in sorted(names):
        t = {"dR": c.r, "dB": c.x}.get(q, c.x if q == "dgate" and c.gate_by == "token" else dp)
        within(g[q], o[q], want[q], t, q)
    return g


SIZES = [(1, 768), (2, 768), (5, 767), (37, 768), (130, 769), (9, 1), (9, 2), (7, 3), (33, 64), (6, 255), (6, 256), (6, 257),
         (5, 1000), (5, 1024), (4, 1025), (3, 2047), (3, 2048), (3, 2049), (2, 4095), (2, 4096)]


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("T,D", SIZES)
def test_plain(T, D, kind, types):
    # eps of 1e-2 where rows of one to three values leave the gradient nothing but eps
    _check_plain(Case(T, D, kind, types, eps=1e-2 if D < 8 else EPS))


@pytest.mark.parametrize("weights,bias", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("p", ["f32", "bf16"])
def test_plain_parameters(weights, bias, p):
    _check_plain(Case(19, 300, "layer", ("bf16", "f32"), weights=weights, bias=bias, p=p))


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("gate", ["none", "scalar", "vector", "token"])
@pytest.mark.parametrize("scale", ["none", "scalar", "vector"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_join_forms(kind, scale, gate, types):
    _check_join(Case(21, 768, kind, types, gate, scale, bias=kind == "layer"))


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("T,D", SIZES)
def test_join_sizes(T, D, types):
    _check_join(Case(T, D, "layer", types, "token", "vector", eps=1e-2 if D < 8 else EPS))
    _check_join(Case(T, D, "rms", types, "vector", "scalar", bias=False, eps=1e-2 if D < 8 else EPS))


@pytest.mark.parametrize("pre,post", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("gate", ["scalar", "vector", "token"])
def test_join_without_a_norm(pre, post, gate):
    for p in ("f32", "bf16"):
        _check_join(Case(23, 500, "rms", ("bf16", "f32"), gate, "vector", pre=pre, post=post, p=p), dp=p)


@pytest.mark.parametrize("T", [511, 2048, 2053, 9001])
def test_many_rows(T):
    _check_plain(Case(T, 96, "rms", ("bf16", "f32")))
    _check_join(Case(T, 96, "layer", ("bf16", "bf16"), "vector", "vector"))
    if T < 9000:
        _check_join(Case(T, 1100, "rms", ("bf16", "f32"), "token", "none", bias=False))


def test_parameters_of_norms_that_the_config_has_not():
    """The C ABI takes no notice of them."""
    import ctypes
    c = Case(9, 500, "rms", ("bf16", "f32"), "vector", "none", pre=False, post=False)
    n, cfg = N(), c.cfg()
    want = n.join_fwd(cfg, c.dev["R"], c.dev["B"], **c.params())[0]
    nan = torch.full((500,), float("nan"), device="cuda")
    got = torch.empty_like(want)
    p = n.NormParams(nan.data_ptr(), nan.data_ptr(), c.dev["gate"].data_ptr(), None, nan.data_ptr(), nan.data_ptr())
    assert n.lib().norm_join_fwd(ctypes.byref(cfg), c.dev["R"].data_ptr(), c.dev["B"].data_ptr(), ctypes.byref(p), 9,
                                 got.data_ptr(), None, torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(got, want)


def test_without_the_stream_gradient():
    c = Case(11, 768, "rms", ("bf16", "f32"), gate="token", bias=False)
    n, z = N(), torch.zeros(11, 768, device="cuda")
    cfg = c.cfg()
    ws = n.Workspace(cfg)
    a = n.bwd(cfg, ws, c.dev["R"], c.dev["dX"], c.dev["w"])
    b = n.bwd(cfg, ws, c.dev["R"], c.dev["dX"], c.dev["w"], dR1=z)
    R1 = n.join_fwd(cfg, c.dev["R"], c.dev["B"], **c.params())[0]
    p = n.join_bwd(cfg, ws, None, c.dev["B"], R1, c.dev["dX"], None, **c.params())
    q = n.join_bwd(cfg, ws, None, c.dev["B"], R1, c.dev["dX"], z, **c.params())
    for x, y in ((a, b), (p, q)):
        assert set(x) == set(y) and all(torch.equal(x[k], y[k]) for k in x)


def test_accumulates_and_in_place():
    c = Case(40, 768, "layer", ("bf16", "f32"), gate="scalar", scale="vector")
    n = N()
    cfg, acc = c.cfg(), c.cfg(accumulate=True)
    ws = n.Workspace(cfg)
    R1, X = n.join_fwd(cfg, c.dev["R"], c.dev["B"], **c.params())
    a = n.join_bwd(cfg, ws, c.dev["R"], c.dev["B"], R1, c.dev["dX"], c.dev["dR1"], **c.params())
    old = {k: torch.full_like(v, 3.0) for k, v in a.items() if k not in ("dR", "dB")}
    dR = c.dev["dR1"].clone()
    b = n.join_bwd(acc, ws, c.dev["R"], c.dev["B"], R1, c.dev["dX"], dR, dR=dR, grads=old, **c.params())
    for k in a:
        if k in ("dR", "dB"):
            assert torch.equal(a[k], b[k]), k
        else:
            assert b[k] is old[k] and torch.equal(b[k], a[k] + 3.0), k
    R = c.dev["R"].clone()
    S, Y = n.join_fwd(cfg, R, c.dev["B"], out_R=R, **c.params())
    assert S is R and torch.equal(R, R1) and torch.equal(X, Y)
    dR = c.dev["dR1"].clone()
    g = n.bwd(acc, ws, c.dev["R"], c.dev["dX"], c.dev["w"], c.dev["b"], dR1=dR, dR=dR, dw=old["dw"].fill_(0),
              db=old["db"].fill_(0))
    f = n.bwd(cfg, ws, c.dev["R"], c.dev["dX"], c.dev["w"], c.dev["b"], dR1=c.dev["dR1"])
    assert all(torch.equal(g[k], f[k]) for k in f)


@pytest.mark.parametrize("gate,D", [("token", 768), ("vector", 1500), ("scalar", 31)])
def test_no_positions(gate, D):
    c = Case(0, D, "rms", ("bf16", "f32"), gate=gate, scale="scalar")
    n, cfg = N(), c.cfg()
    ws = n.Workspace(cfg)
    assert n.fwd(cfg, c.dev["R"], c.dev["w"]).shape == (0, D)
    R1, X = n.join_fwd(cfg, c.dev["R"], c.dev["B"], **c.params())
    nan = {"d" + k: torch.full_like(v, float("nan")) for k, v in c.params().items()}
    g = n.join_bwd(cfg, ws, c.dev["R"], c.dev["B"], R1, c.dev["dX"], c.dev["dR1"], grads=dict(nan), **c.params())
    assert all((v == 0).all() for v in g.values())
    acc = c.cfg(accumulate=True)
    g = n.join_bwd(acc, ws, c.dev["R"], c.dev["B"], R1, c.dev["dX"], c.dev["dR1"],
                   grads={k: v.fill_(2) for k, v in nan.items()}, **c.params())
    assert all((v == 2).all() for k, v in g.items() if k not in ("dR", "dB"))


@pytest.mark.parametrize("D", [40, 768, 1030, 4096])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_huge_and_tiny_rows(kind, D):
    """Rows whose squares leave fp32's range: the norm does not depend on the scale."""
    n = N()
    cfg = n.config(D, kind, "bf16", "f32")
    base = torch.randn(5, D, generator=torch.Generator().manual_seed(D)).bfloat16().float()
    ref = n.fwd(cfg, base.cuda())
    ws = n.Workspace(cfg)
    dX = torch.randn(5, D, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    want = n.bwd(cfg, ws, base.cuda(), dX)["dR"].double()
    for e in (62, 70, 120):
        X = n.fwd(cfg, (base * 2.0 ** e).cuda())
        # eps is the only difference: 5e-7 of the value, then the rounding to bf16
        assert ((X - ref).double().abs() <= (2.0 ** -7 + 1e-6) * ref.double().abs()).all(), e
        got = n.bwd(cfg, ws, (base * 2.0 ** e).cuda(), dX)["dR"].double() * 2.0 ** e
        # the row's gradient falls as 2^-e; a hundred roundings of its largest terms
        assert ((got - want).abs() <= 100 * U * want.abs().max() + 1e-5 * want.abs()).all(), e
    tiny = n.fwd(cfg, (base * 2.0 ** -90).cuda()).double()
    if kind == "rms":
        lim = base.double().cuda() * 2.0 ** -90 * 1e3
        assert ((tiny - lim).abs() <= 2.0 ** -8 * lim.abs() + 2.0 ** -133).all()
    zero = n.fwd(cfg, torch.zeros(3, D, device="cuda"))
    assert (zero == 0).all()


@pytest.mark.parametrize("D", [768, 1100])
def test_not_finite_stays_in_its_row(D):
    n = N()
    c = Case(13, D, "layer", ("bf16", "f32"), gate="token", scale="vector")
    cfg = c.cfg()
    ws = n.Workspace(cfg)
    clean = n.join_fwd(cfg, c.dev["R"], c.dev["B"], **c.params())
    g0 = n.join_bwd(cfg, ws, c.dev["R"], c.dev["B"], clean[0], c.dev["dX"], c.dev["dR1"], **c.params())
    for v in (float("nan"), float("inf"), -float("inf")):
        B = c.dev["B"].clone()
        B[4, D - 1] = v
        R1, X = n.join_fwd(cfg, c.dev["R"], B, **c.params())
        keep = torch.arange(13, device="cuda") != 4
        assert torch.equal(R1[keep], clean[0][keep]) and torch.equal(X[keep], clean[1][keep])
        assert torch.isnan(R1[4]).all() and torch.isnan(X[4]).all()
        g = n.join_bwd(cfg, ws, c.dev["R"], B, clean[0], c.dev["dX"], c.dev["dR1"], **c.params())
        for k in ("dR", "dB", "dgate"):
            assert torch.equal(g[k][keep], g0[k][keep]), k
        assert torch.equal(g["dR"], g0["dR"]) and torch.isnan(g["dB"][4]).all()
        assert torch.equal(g["dw"], g0["dw"]) and torch.isnan(g["dpost_w"]).all()


def test_gate_far_out():
    """Gates of a sigmoid that is 0 or 1 to the last bit, infinities among them."""
    n = N()
    T, D = 4, 64
    G = torch.tensor([-float("inf"), -1e4, 1e4, float("inf")]).view(4, 1).expand(T, D).contiguous().bfloat16().cuda()
    R, B = torch.randn(T, D, device="cuda"), torch.randn(T, D, device="cuda").bfloat16()
    cfg = n.config(D, gate="token", post=False)
    R1, _ = n.join_fwd(cfg, R, B, gate=G)
    assert torch.equal(R1[:2], R[:2]) and torch.equal(R1[2:], R[2:] + B[2:].float())
    ws = n.Workspace(cfg)
    g = n.join_bwd(cfg, ws, None, B, R1, B, R, gate=G)
    assert (g["dgate"] == 0).all() and (g["dB"][:2] == 0).all() and torch.isfinite(g["dB"]).all()


def test_same_bits_every_time_other_streams_and_threads():
    import threading
    c = Case(3000, 768, "rms", ("bf16", "f32"), gate="token", scale="vector", bias=False)
    n, cfg = N(), c.cfg()
    R1, X = n.join_fwd(cfg, c.dev["R"], c.dev["B"], **c.params())
    ws = n.Workspace(cfg)
    ref = n.join_bwd(cfg, ws, c.dev["R"], c.dev["B"], R1, c.dev["dX"], c.dev["dR1"], **c.params())
    torch.cuda.synchronize()
    bad = []

    def work():
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            w = n.Workspace(cfg)
            for _ in range(3):
                a, b = n.join_fwd(cfg, c.dev["R"], c.dev["B"], **c.params())
                g = n.join_bwd(cfg, w, c.dev["R"], c.dev["B"], R1, c.dev["dX"], c.dev["dR1"], **c.params())
                s.synchronize()
                if not (torch.equal(a, R1) and torch.equal(b, X) and all(torch.equal(g[k], ref[k]) for k in ref)):
                    bad.append(1)

    th = [threading.Thread(target=work) for _ in range(3)]
    [t.start() for t in th]
    [t.join() for t in th]
    assert not bad


def test_captured():
    c = Case(300, 768, "layer", ("bf16", "f32"), gate="scalar", scale="scalar")
    n, cfg = N(), c.cfg()
    ws = n.Workspace(cfg)

    def call():
        R1, X = n.join_fwd(cfg, c.dev["R"], c.dev["B"], **c.params())
        g = n.join_bwd(cfg, ws, c.dev["R"], c.dev["B"], R1, c.dev["dX"], c.dev["dR1"], **c.params())
        h = n.bwd(cfg, ws, c.dev["R"], c.dev["dX"], c.dev["w"], c.dev["b"], dR1=g["dR"])
        return {"R1": R1, "X": X, **g, **{"n" + k: v for k, v in h.items()}}

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for k in range(3):
        c.dev["B"].copy_(torch.randn(300, 768, generator=torch.Generator().manual_seed(k)))
        graph.replay()
        want = call()
        torch.cuda.synchronize()
        assert all(torch.equal(got[q], want[q]) for q in want), k
        torch.randn(1 << 16, device="cuda").sum().item()


def test_rows_past_32_bits():
    """Element offsets past 2^32 (bf16 rows of 4,096): the last rows against the same rows alone."""
    n = N()
    T, D = (1 << 20) + 3, 4096
    cfg = n.config(D, "rms", "bf16", "bf16", gate="vector")
    R = torch.empty(T, D, dtype=torch.bfloat16, device="cuda")
    R[:8].normal_()
    R[-8:].normal_()
    R[8:-8] = 1
    B = R.clone()
    gate = torch.rand(D, device="cuda")
    R1, X = n.join_fwd(cfg, R, B, gate=gate)
    a, b = n.join_fwd(cfg, R[-8:].contiguous(), B[-8:].contiguous(), gate=gate)
    assert torch.equal(R1[-8:], a) and torch.equal(X[-8:], b)
    ws = n.Workspace(cfg)
    g = n.join_bwd(cfg, ws, None, B, R1, X, R, gate=gate)
    h = n.join_bwd(cfg, ws, None, B[-8:].contiguous(), a, b, R[-8:].contiguous(), gate=gate)
    assert torch.equal(g["dR"][-8:], h["dR"]) and torch.equal(g["dB"][-8:], h["dB"])


def test_unaligned_buffers_and_guards():
    """Buffers at odd elements, NaN on both sides of every one: the same bits, nothing written outside."""
    n = N()
    T, D = 7, 1001
    c = Case(T, D, "layer", ("bf16", "bf16"), gate="token", scale="vector", p="bf16")
    cfg = c.cfg(dp_dtype="bf16")
    R1, X = n.join_fwd(cfg, c.dev["R"], c.dev["B"], **c.params())
    ws = n.Workspace(cfg)
    ref = n.join_bwd(cfg, ws, c.dev["R"], c.dev["B"], R1, c.dev["dX"], c.dev["dR1"], **c.params())

    held = []

    def odd(t, fill=None):
        buf = torch.full((t.numel() + 64,), float("nan"), dtype=t.dtype, device="cuda")
        v = buf[31:31 + t.numel()].view(t.shape)
        v.copy_(t if fill is None else torch.full_like(t, fill))
        held.append((buf, t.numel()))
        return v

    p = {k: odd(v) for k, v in c.params().items()}
    a, b = n.join_fwd(cfg, odd(c.dev["R"]), odd(c.dev["B"]), out_R=odd(R1, 0.0), out=odd(X, 0.0), **p)
    assert torch.equal(a, R1) and torch.equal(b, X)
    g = n.join_bwd(cfg, ws, odd(c.dev["R"]), odd(c.dev["B"]), a, odd(c.dev["dX"]), odd(c.dev["dR1"]),
                   dR=odd(ref["dR"], 0.0), dB=odd(ref["dB"], 0.0),
                   grads={k: odd(v, 0.0) for k, v in ref.items() if k not in ("dR", "dB")}, **p)
    assert all(torch.equal(g[k], ref[k]) for k in ref)
    for buf, m in held:
        assert torch.isnan(buf[:31]).all() and torch.isnan(buf[31 + m:]).all()
