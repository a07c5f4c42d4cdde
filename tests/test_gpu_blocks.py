"""A model of the table, the norms, the recurrence, the feed-forward block and the
loss, run together as a training program runs them:

    E = embed_fwd(tokens)                    X = norm(E);  x, r, i of one projection of X, G of another
    B = recur(x, r, i) over the documents    R1, X1 = join(E, B, gate G)
    Y = R1 + ffn(X1)                         Z = norm(Y);  loss_fwd / loss_bwd of Z
    and back through each to E's gradient, which goes to embed_bwd_accum and the step.

Each stage is held to its operator's own bound on the inputs that it was given on the
device (the bounds are derived where each operator is tested alone).  A micro-step
captured into a graph is replayed with other tokens, documents and targets and
compared bitwise with the same calls one by one.  A serving program's prompt and its
further tokens, one by one, are compared with the whole text at once.
"""
import numpy as np
import pytest
import torch

import oracle
from bounds import V, within
from gpu_common import State, ng, to_dev
from oracle import norm as orcn
from oracle import recur as orcr
from oracle import ssm as orcs
from sparse_hashed_gram_amd import synth, workloads
from test_gpu_ffn import _bf16, _bounds, _f64, _hold, _real
from test_gpu_norm import EPS, _affine_v, _norm_v, _sig_v, _slope_v, _steps, _through_v
from test_gpu_recur import Case
from test_gpu_ssm import _check_bwd, _check_fwd

pytestmark = pytest.mark.gpu

D = 768
DOCS = 40   # places for documents in a micro-step


def _par(seed, *shape, std=1.0, mean=0.0):
    r = np.random.default_rng(seed)
    return mean + std * r.standard_normal(shape)


class Model:
    def __init__(self, T, F, C):
        from sparse_hashed_gram_amd import ffn, norm, recur, ssm
        self.N, self.M, self.S, self.n, self.r = ng(), ffn, ssm, norm, recur
        self.w, self.T, w = workloads.TINY, T, workloads.TINY
        self.cfg = self.N.config(w.vocab, w.eos_id, w.rows, "f32", max_tokens=T, mode="burst_ref")
        self.fcfg = ffn.config(F, T, act="silu", y_dtype="f32", dw_dtype="f32", accumulate=True)
        self.scfg = ssm.config(w.vocab, C, T)
        self.pcfg = norm.config(D, eps=EPS, accumulate=True)                 # the plain norms
        self.jcfg = norm.config(D, gate="token", eps=EPS, accumulate=True)
        self.rcfg = recur.config(D, T, accumulate=True)
        self.st = State(self.cfg, to_dev(synth.init_rows(w, 0, w.rows[0])), to_dev(synth.init_rows(w, 1, w.rows[1])))
        self.Wh = _real(1, F, 40)[1]
        self.W = [_bf16(a).cuda() for a in self.Wh]
        self.Uh = _bf16(_par(41, w.vocab, D, std=0.05)).float().numpy()
        self.Uw = _bf16(self.Uh).cuda()
        self.P = _bf16(_par(42, 3 * D, D, std=D ** -0.5)).cuda()
        self.Pg = _bf16(_par(43, D, D, std=D ** -0.5)).cuda()
        u = np.random.default_rng(44).uniform(0.9, 0.999, D)
        self.lam = torch.from_numpy(np.log(np.expm1(-np.log(u) / 8.0))).float().cuda()
        self.g = [torch.from_numpy(_par(45 + k, D, std=0.1, mean=1.0)).float().cuda() for k in range(4)]
        self.ws, self.fws, self.sws = self.N.Workspace(self.cfg), ffn.Workspace(self.fcfg), ssm.Workspace(self.scfg)
        self.nws, self.rws = norm.Workspace(self.jcfg), recur.Workspace(self.rcfg)
        self.dW = [torch.zeros(s, device="cuda") for s in ((F, D), (F, D), (D, F))]
        self.dU = torch.zeros((w.vocab, D), device="cuda")
        self.dg = [torch.zeros(D, device="cuda") for _ in range(4)]
        self.dlam = torch.zeros(D, device="cuda")
        self.sums = [*self.dW, self.dU, *self.dg, self.dlam]

    def step(self, tok, offsets, tgt, perm, g):
        n, q, w0, pw, w1, w2 = self.n, {}, *self.g
        E = q["E"] = self.N.embed_fwd(self.cfg, *self.st.W, tok, ws=self.ws)
        X = q["X"] = n.fwd(self.pcfg, E, w0)
        P = q["P"] = X @ self.P.t()
        G = q["G"] = X @ self.Pg.t()
        xri = P[:, :D], P[:, D:2 * D], P[:, 2 * D:]
        B, _, saved = self.r.fwd(self.rcfg, self.rws, *xri, self.lam, offsets, keep=True)
        q["B"] = B
        R1, X1 = q["R1"], q["X1"] = n.join_fwd(self.jcfg, E, B, post_w=pw, gate=G, w=w1)
        Y = q["Y"] = self.M.fwd(self.fcfg, self.fws, X1, *self.W, residual=R1)
        Z = q["Z"] = n.fwd(self.pcfg, Y, w2)
        q["cand"], q["slot"] = self.S.candidates(self.scfg, self.sws, tgt, perm)
        q["loss"], q["lse"] = self.S.loss_fwd(self.scfg, self.sws, Z, self.Uw, q["cand"], q["slot"])
        q["dZ"] = self.S.loss_bwd(self.scfg, self.sws, Z, self.Uw, q["cand"], q["slot"], q["lse"], g, self.dU)
        dZ = q["dZb"] = q["dZ"].bfloat16()
        dY = q["dY"] = n.bwd(self.pcfg, self.nws, Y, dZ, w2, dw=self.dg[3])["dR"]
        q["dX1"] = self.M.bwd(self.fcfg, self.fws, X1, *self.W, dY, None, None, *self.dW)["dX"]
        dX1 = q["dX1b"] = q["dX1"].bfloat16()
        j = n.join_bwd(self.jcfg, self.nws, None, B, R1, dX1, dY, post_w=pw, gate=G, w=w1,
                       grads={"dpost_w": self.dg[1], "dw": self.dg[2]})
        q["dR"], q["dB"], q["dG"] = j["dR"], j["dB"], j["dgate"]
        dP = q["dP"] = torch.zeros_like(P)
        self.r.bwd(self.rcfg, self.rws, *xri, self.lam, saved, j["dB"], offsets, dx=dP[:, :D], dr=dP[:, D:2 * D],
                   di=dP[:, 2 * D:], dlam=self.dlam)
        dX = q["dX"] = dP @ self.P + j["dgate"] @ self.Pg
        q["dE"] = n.bwd(self.pcfg, self.nws, E, dX, w0, dR1=j["dR"], dw=self.dg[0])["dR"]
        self.N.embed_bwd_accum(self.cfg, self.ws, tok, q["dE"])
        return q


def _inputs(w, s, T):
    """tokens, where documents begin (and end; the places that are left have none), targets, ..."""
    r = np.random.default_rng([s, T])
    tok = synth.tokens(w, s, T)
    starts = np.flatnonzero(tok == w.eos_id)
    if len(starts) == 0 or starts[0] != 0:
        starts = np.append(0, starts)
    starts = np.unique(np.append(starts, r.integers(1, T, min(10, T - 1)) if T > 1 else []))[:DOCS]
    off = np.append(starts, np.full(DOCS + 1 - len(starts), T)).astype(np.int32)
    tgt = np.append(tok[1:], tok[0]).astype(np.int32)
    g = np.where(r.random(T) < 0.9, 1.0 / T, 0.0).astype(np.float32)
    return tok, off, tgt, r.permutation(w.vocab).astype(np.int32), g


def _norm_back(m, r, dR, dw, k, R, dX, dR1):
    """One norm's backward; what it added to its weight's gradient (which was 0)."""
    w = _f64(m.g[k])
    xh, rho = _norm_v(V(R), "rms", EPS)
    o = orcn.backward(R, dX, "rms", EPS, w, dR1)
    back = _through_v(xh, rho, _affine_v(V(dX), w, None), "rms")
    within(r[dR], o["dR"], back if dR1 is None else V(dR1) + back, "f32", dR)
    within(m.dg[k], o["dw"], (V(dX) * xh).total(_steps(m.T)), "f32", dw)


@pytest.mark.parametrize("T", [1, 300, 700])
def test_stage_by_stage(T):
    w, F, C = workloads.TINY, 264, 900
    m = Model(T, F, C)
    tok, off, tgt, perm, g = _inputs(w, 3, T)
    r = m.step(to_dev(tok), to_dev(off), to_dev(tgt), to_dev(perm), to_dev(g))
    h = {k: _f64(v) for k, v in r.items()}
    w0, pw, w1, w2 = (_f64(x) for x in m.g)
    rb, nb, rt, nt, _ = oracle.ngram_rows(tok, w.vocab, w.eos_id, w.rows)
    W0 = [x.cpu().numpy() for x in m.st.W]
    assert np.array_equal(h["E"], oracle.forward(*W0, rb, nb, rt, nt).astype(np.float64))
    within(r["X"], orcn.forward(h["E"], "rms", EPS, w0), _affine_v(_norm_v(V(h["E"]), "rms", EPS)[0], w0, None), "bf16", "X")
    c = Case.__new__(Case)
    c.T, c.D, c.t, c.c, c.off, c.n, c.hh0, c.hdhT = T, D, "bf16", 8.0, off, DOCS, None, None
    c.hx, c.hr, c.hi = (h["P"][:, k * D:(k + 1) * D] for k in range(3))
    c.hdy, c.hlam = h["dB"], _f64(m.lam)
    b, inside = c.bounds()
    assert inside.all()
    within(r["B"], orcr.forward(c.hx, c.hr, c.hi, c.hlam, 8.0, off)[0], b["y"], "bf16", "B")
    o1, oX = orcn.join(h["E"], h["B"], "rms", EPS, post_w=pw, gate=h["G"], token=True, w=w1)
    nh, rho = _norm_v(V(h["B"]), "rms", EPS)
    r1 = h["E"] + _sig_v(h["G"]) * _affine_v(nh, pw, None)
    within(r["R1"], o1, r1, "f32", "R1")
    within(r["X1"], oX, _affine_v(_norm_v(r1, "rms", EPS)[0], w1, None), "bf16", "X1")
    o = _bounds(h["X1"], m.Wh, h["dY"], "silu", None, True)
    _hold(r["Y"], o["Y"][0] + h["R1"], o["Y"][1] + 2.0 ** -23 * np.abs(h["R1"]), False, "Y")
    within(r["Z"], orcn.forward(h["Y"], "rms", EPS, w2), _affine_v(_norm_v(V(h["Y"]), "rms", EPS)[0], w2, None), "bf16", "Z")
    cand_o, slot_o, _, ok = orcs.candidates(tgt, perm, w.vocab, C)
    assert ok
    np.testing.assert_array_equal(r["cand"].cpu().numpy(), cand_o)
    np.testing.assert_array_equal(r["slot"].cpu().numpy(), slot_o)
    Z = r["Z"].float().cpu().numpy()
    _check_fwd(Z, m.Uh, cand_o, slot_o, r["loss"], r["lse"], C)
    _check_bwd(Z, m.Uh, cand_o, slot_o, g, r["dZ"], m.dU, np.zeros((w.vocab, D), np.float32), C)
    _norm_back(m, r, "dY", "dw2", 3, h["Y"], h["dZb"], None)
    _hold(r["dX1"], *o["dX"], False, "dX1")
    for k, name in enumerate(("dWg", "dWu", "dWd")):
        _hold(m.dW[k], *o[name], False, name)
    j = orcn.join_backward(h["E"], h["B"], h["R1"], h["dX1b"], h["dY"], "rms", EPS, post_w=pw, gate=h["G"], token=True, w=w1)
    xh, rho1 = _norm_v(V(h["R1"]), "rms", EPS)
    dE = V(h["dY"]) + _through_v(xh, rho1, _affine_v(V(h["dX1b"]), w1, None), "rms")
    dN = dE * _sig_v(h["G"])
    within(r["dR"], j["dR"], dE, "f32", "dR")
    within(r["dG"], j["dgate"], dE * _affine_v(nh, pw, None) * _slope_v(h["G"]), "bf16", "dG")
    within(r["dB"], j["dB"], _through_v(nh, rho, _affine_v(dN, pw, None), "rms"), "bf16", "dB")
    within(m.dg[1], j["dpost_w"], (dN * nh).total(_steps(T) + 1), "f32", "dpost_w")
    within(m.dg[2], j["dw"], (V(h["dX1b"]) * xh).total(_steps(T)), "f32", "dw1")
    q = orcr.backward(c.hx, c.hr, c.hi, c.hlam, 8.0, c.hdy, off)
    for k, name in enumerate(("dx", "dr", "di")):
        within(r["dP"][:, k * D:(k + 1) * D], q[name], b[name], "bf16", name)
    within(m.dlam, q["dlam"], b["dlam"], "f32", "dlam")
    _norm_back(m, r, "dE", "dw0", 0, h["E"], h["dX"], h["dR"])
    assert m.N.device_status(m.cfg, m.ws) == 0 and m.S.device_status(m.scfg, m.sws) == 0


@pytest.mark.parametrize("T", [37, 600])
def test_captured_equals_eager(T):
    w, F, C = workloads.TINY, 264, 900
    a, b = Model(T, F, C), Model(T, F, C)      # a: captured, b: call by call
    bufs = [torch.zeros(n, dtype=t, device="cuda") for n, t in
            ((T, torch.int32), (DOCS + 1, torch.int32), (T, torch.int32), (w.vocab, torch.int32), (T, torch.float32))]

    def load(s):
        x = [to_dev(v) for v in _inputs(w, s, T)]
        for dst, src in zip(bufs, x):
            dst.copy_(src)
        return x

    def run(m, x):
        for v in m.sums:
            v.zero_()
        return m.step(*x)

    x = load(0)
    run(a, x)
    a.st.step(a.ws, 1, w.lr, w.beta2, w.eps)    # the first use of everything lies before the capture
    run(b, x)
    b.st.step(b.ws, 1, w.lr, w.beta2, w.eps)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = run(a, bufs)
    for k in range(1, 4):
        x = load(k)
        g.replay()
        a.st.step(a.ws, k + 1, w.lr, w.beta2, w.eps)
        ref = run(b, x)
        b.st.step(b.ws, k + 1, w.lr, w.beta2, w.eps)
        torch.cuda.synchronize()
        for q in ref:
            assert torch.equal(got[q], ref[q]), (k, q)
        for p, q in zip(a.sums + list(a.st.W) + list(a.st.st), b.sums + list(b.st.W) + list(b.st.st)):
            assert torch.equal(p, q), k
        torch.randn(1 << 16, device="cuda").sum().item()   # other work between the replays


def test_serving_continues_a_prompt():
    """A prompt, then its tokens one at a time: embedding, norm, recurrence and join of each are those of the
    whole text at once, up to the order of the recurrence's sums."""
    m = Model(64, 264, 900)
    n, q, T, cut = m.n, m.r, 60, 41
    tok = synth.tokens(m.w, 9, T).astype(np.int32)
    tok[0] = m.w.eos_id
    tok[1:][tok[1:] == m.w.eos_id] = 5
    tok = to_dev(tok)
    rws = q.Workspace(m.rcfg, backward=False)
    E = m.N.embed_fwd(m.cfg, *m.st.W, tok, ws=m.ws)

    def block(E, recur):
        X = n.fwd(m.pcfg, E, m.g[0])
        P, G = (X.float() @ m.P.float().t()).bfloat16(), (X.float() @ m.Pg.float().t()).bfloat16()
        B = recur(*(P[:, k * D:(k + 1) * D] for k in range(3)))
        return n.join_fwd(m.jcfg, E, B, post_w=m.g[1], gate=G, w=m.g[2])

    whole, _ = block(E, lambda x, r, i: q.fwd(m.rcfg, rws, x, r, i, m.lam)[0])
    state = []

    def prompt(x, r, i):
        y, s, _ = q.fwd(m.rcfg, rws, x, r, i, m.lam, final=True)
        state.append(s)
        return y

    parts = [block(E[:cut], prompt)[0]]
    for t in range(cut, T):
        parts.append(block(E[t:t + 1], lambda x, r, i: q.step(m.rcfg, x, r, i, m.lam, state[0]))[0])
    got = torch.cat(parts)
    # B is rounded to bf16 in both; where the sums' order puts it on the other side of a border it
    # differs by a step, 2^-7 of its value, and so does the gated norm of it
    lim = 2.0 ** -6 * (whole - E).abs() + 2.0 ** -8 * (whole - E).abs().amax(1, keepdim=True)
    assert ((got - whole).abs() <= lim).all()
