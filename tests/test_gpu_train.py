"""The dropped embedding, the feed-forward block, the sampled-softmax loss and
the sparse step run together, as a training program runs them:

    E = embed_fwd_drop(tokens)          Y = E + drop(ffn(bf16 E))
    loss_fwd / loss_bwd of bf16 Y       dY = dX of the loss
    dE = dY + dX of ffn.bwd(dY)         drop.bwd(dE) -> embed_bwd_accum, then the step

for the micro-steps of one window, each with masks of its own.  Each stage is
held to its operator's own bound on the inputs that it was given on the device
(the bounds are derived where each operator is tested alone), so an output left
out, mixed up or overwritten by a neighbour's call shows at its stage.  A window
captured into one graph is replayed with other tokens, targets and masks and
compared bitwise with the same window run call by call.
"""
import numpy as np
import pytest
import torch

import oracle
from gpu_common import State, check_step_against_oracle, ng, oracle_snapshots, to_dev, window_oracle
from oracle import drop as orcd
from oracle import ssm as orcs
from sparse_hashed_gram_amd import synth, workloads
from test_gpu_ffn import _bf16, _bounds, _f64, _hold, _real
from test_gpu_ssm import _check_bwd, _check_fwd

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
P_E, P_F, SEED = 0.1, 0.2, 77
NAMES = ("dWg", "dWu", "dWd")


class Model:
    def __init__(self, T, F, C):
        from sparse_hashed_gram_amd import drop, ffn, ssm
        self.N, self.D, self.M, self.S = ng(), drop, ffn, ssm
        self.w, self.T = workloads.TINY, T
        w = self.w
        self.cfg = self.N.config(w.vocab, w.eos_id, w.rows, "f32", max_tokens=T, mode="burst_ref")
        self.fcfg = ffn.config(F, T, act="gelu", y_dtype="f32", dw_dtype="f32", accumulate=True)
        self.scfg = ssm.config(w.vocab, C, T)
        self.st = State(self.cfg, to_dev(synth.init_rows(w, 0, w.rows[0])), to_dev(synth.init_rows(w, 1, w.rows[1])))
        self.Wh = _real(1, F, 40)[1]
        self.W = [_bf16(a).cuda() for a in self.Wh]
        self.Uh = _bf16(np.random.default_rng(41).standard_normal((w.vocab, 768)) * 0.05).float().numpy()
        self.Uw = _bf16(self.Uh).cuda()
        self.ws, self.fws, self.sws = self.N.Workspace(self.cfg), ffn.Workspace(self.fcfg), ssm.Workspace(self.scfg)
        self.dW = [torch.zeros(s, device="cuda") for s in ((F, 768), (F, 768), (768, F))]
        self.dU = torch.zeros((w.vocab, 768), device="cuda")

    def step(self, tok, tgt, perm, g, spec_e, spec_f):
        """One micro-step, all its results."""
        r = {}
        E = r["E"] = self.N.embed_fwd_drop(self.cfg, *self.st.W, tok, spec_e, ws=self.ws)
        X = r["X"] = E.bfloat16()
        Y = r["Y"] = self.M.fwd(self.fcfg, self.fws, X, *self.W, residual=E, drop=spec_f)
        Z = r["Z"] = Y.bfloat16()
        r["cand"], r["slot"] = self.S.candidates(self.scfg, self.sws, tgt, perm)
        r["loss"], r["lse"] = self.S.loss_fwd(self.scfg, self.sws, Z, self.Uw, r["cand"], r["slot"])
        dY = r["dY"] = self.S.loss_bwd(self.scfg, self.sws, Z, self.Uw, r["cand"], r["slot"], r["lse"], g, self.dU)
        r["dX"] = self.M.bwd(self.fcfg, self.fws, X, *self.W, dY, spec_f, None, *self.dW)["dX"]
        r["dE"] = self.D.bwd(spec_e, dY + r["dX"])
        self.N.embed_bwd_accum(self.cfg, self.ws, tok, r["dE"])
        return r


def _inputs(w, s, T):
    r = np.random.default_rng([s, T])
    tok = synth.tokens(w, s, T)
    tgt = np.append(tok[1:], tok[0]).astype(np.int32)   # the next token
    g = np.where(r.random(T) < 0.9, 1.0 / T, 0.0).astype(np.float32)   # some positions without a loss
    return tok, tgt, r.permutation(w.vocab).astype(np.int32), g


@pytest.mark.parametrize("T", [1, 300])
def test_window_stage_by_stage(T):
    w, F, C = workloads.TINY, 264, 400
    m = Model(T, F, C)
    factor = lambda p, o: orcd.keep(T, 768, p, SEED, o) * (65536 / (65536 - orcd.threshold(p)))   # noqa: E731
    toks, dEs, seen = [], [], []
    want = [(np.zeros(s), np.zeros(s)) for s in ((F, 768), (F, 768), (768, F))]
    dU0 = np.zeros((w.vocab, 768), np.float32)
    W0 = [x.cpu().numpy() for x in m.st.W]
    for s in range(w.accum_steps):
        tok, tgt, perm, g = _inputs(w, s, T)
        spec_e, spec_f = m.D.spec(P_E, SEED, 2 * s), m.D.spec(P_F, SEED, 2 * s + 1)
        r = m.step(to_dev(tok), to_dev(tgt), to_dev(perm), to_dev(g), spec_e, spec_f)
        fe, ff = factor(P_E, 2 * s), factor(P_F, 2 * s + 1)
        rb, nb, rt, nt, _ = oracle.ngram_rows(tok, w.vocab, w.eos_id, w.rows)
        e = oracle.forward(*W0, rb, nb, rt, nt).astype(np.float64) * fe
        assert np.all(np.abs(_f64(r["E"]) - e) <= 2 * U * np.abs(e))
        X, dY = _f64(r["X"]), _f64(r["dY"])
        o = _bounds(X, m.Wh, dY, "gelu", ff, True)
        E = _f64(r["E"])
        _hold(r["Y"], o["Y"][0] + E, o["Y"][1] + 2 * U * np.abs(E), False, "Y")
        cand_o, slot_o, _, ok = orcs.candidates(tgt, perm, w.vocab, C)
        assert ok
        np.testing.assert_array_equal(r["cand"].cpu().numpy(), cand_o)
        np.testing.assert_array_equal(r["slot"].cpu().numpy(), slot_o)
        Z = r["Z"].float().cpu().numpy()
        _check_fwd(Z, m.Uh, cand_o, slot_o, r["loss"], r["lse"], C)
        _check_bwd(Z, m.Uh, cand_o, slot_o, g, r["dY"], m.dU, dU0, C)
        dU0 = m.dU.cpu().numpy().copy()
        _hold(r["dX"], *o["dX"], False, "dX")
        for i, k in enumerate(NAMES):   # each micro-step's sum is rounded to fp32 as it is added
            v, b = want[i][0] + o[k][0], want[i][1] + o[k][1] + 2 * U * np.abs(o[k][0])
            want[i] = (v, b + 2 * U * (np.abs(v) + b))
        d = (dY + _f64(r["dX"])) * fe
        assert np.all(np.abs(_f64(r["dE"]) - d) <= 2.01 * 2 * U * np.abs(d))   # the sum's and the scale's rounding
        toks.append(tok)
        dEs.append(r["dE"].cpu().numpy())
        seen.append(r)
    for i, k in enumerate(NAMES):
        assert np.all(np.abs(_f64(m.dW[i]) - want[i][0]) <= want[i][1]), k
    assert not torch.equal(seen[0]["E"] == 0, seen[1]["E"] == 0)
    snaps = oracle_snapshots(m.st, window_oracle(m.cfg, toks, dEs), np.random.default_rng(T))
    m.st.step(m.ws, 1, w.lr, w.beta2, w.eps)
    check_step_against_oracle(m.st, snaps, 1, w.lr, w.beta2, w.eps, "f32")
    assert m.N.device_status(m.cfg, m.ws) == 0 and m.S.device_status(m.scfg, m.sws) == 0


@pytest.mark.parametrize("T", [37, 600])
def test_captured_window_equals_eager(T):
    w, F, C = workloads.TINY, 520, 900
    A = w.accum_steps
    a, b = Model(T, F, C), Model(T, F, C)      # a: captured, b: call by call
    rng = torch.zeros(2 * A, 2, dtype=torch.int64, device="cuda")
    bufs = [[torch.zeros(n, dtype=t, device="cuda") for n, t in
             ((T, torch.int32), (T, torch.int32), (w.vocab, torch.int32), (T, torch.float32))] for _ in range(A)]
    params = a.N.step_params(1, w.lr, w.beta2, w.eps)

    def load(win):
        out = []
        for s in range(A):
            x = [to_dev(v) for v in _inputs(w, 100 * win + s, T)]
            for dst, src in zip(bufs[s], x):
                dst.copy_(src)
            for i in range(2):
                a.D.rng_state(SEED + win, 2 * s + i, out=rng[2 * s + i])
            out.append(x)
        return out

    def window():
        for x in a.dW + [a.dU]:
            x.zero_()
        rs = [a.step(*bufs[s], a.D.spec(P_E, rng=rng[2 * s]), a.D.spec(P_F, rng=rng[2 * s + 1])) for s in range(A)]
        a.N.sparse_step_dev(a.cfg, a.ws, *a.st.W, *a.st.st, params)
        return rs

    load(0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = window()
    for win in range(3):
        x = load(win)
        a.N.step_params(win + 1, w.lr, w.beta2, w.eps, out=params)
        g.replay()
        for y in b.dW + [b.dU]:
            y.zero_()
        ref = [b.step(*x[s], b.D.spec(P_E, SEED + win, 2 * s), b.D.spec(P_F, SEED + win, 2 * s + 1)) for s in range(A)]
        b.st.step(b.ws, win + 1, w.lr, w.beta2, w.eps)
        torch.cuda.synchronize()
        for s in range(A):
            for k in ref[s]:
                assert torch.equal(got[s][k], ref[s][k]), (win, s, k)
        for p, q in zip(a.dW + [a.dU] + list(a.st.W) + list(a.st.st), b.dW + [b.dU] + list(b.st.W) + list(b.st.st)):
            assert torch.equal(p, q), win
        torch.randn(1 << 16, device="cuda").sum().item()   # other work between the replays
    for m in (a, b):
        assert m.N.device_status(m.cfg, m.ws) == 0 and m.S.device_status(m.scfg, m.sws) == 0
