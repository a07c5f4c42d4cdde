"""Cases that measure the norms around a block (alone, and joined with the block's gate and the residual stream) and the gated linear
recurrence (training over packed sequences, prefill, and the step of single tokens).

Every case runs in two ways on the same inputs: ``own = False`` computes the operator from elementary torch operations in 32 bits,
``own = True`` makes the calls a training or serving program makes of ``sparse_hashed_gram_amd``.

Norm of a row x: (x - mu) / sqrt(mean((x - mu)^2) + eps) w + b, with mu = 0 ("rms") or the row's mean ("layer").
Join: R1 = s R + gamma norm(B), X = norm(R1), gamma a vector or the sigmoid of a gate for each element.
Recurrence, each channel by itself: a = exp(-c softplus(lam) sigmoid(r)), h_t = a h_{t-1} + sqrt(1 - a^2) sigmoid(i) x.
"""
import math

import torch

own = False

EPS = 1e-6
C = 8.0
_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one token of a serving loop, in front of its block
        {"name": "norm_fwd_1x768", "op": "norm", "dir": "fwd", "T": 1, "D": 768, "kind": "rms", "x": "bf16", "r": "f32"},
        # a training micro-batch's gradient on its way past the norm, joined with the residual stream's
        {"name": "norm_bwd_49152x768", "op": "norm", "dir": "bwd", "T": 49152, "D": 768, "kind": "rms", "x": "bf16", "r": "f32"},
        # the end of one block and the start of the next, a short document
        {"name": "join_fwd_37x768_bf16", "op": "join", "dir": "fwd", "T": 37, "D": 768, "kind": "rms", "x": "bf16", "r": "bf16", "gate": "vector", "scale": True},
        # the recurrence's block: its output normalised and gated element by element, fp32 residual stream
        {"name": "join_fwd_49152x768_token", "op": "join", "dir": "fwd", "T": 49152, "D": 768, "kind": "rms", "x": "bf16", "r": "f32", "gate": "token", "scale": False},
        # rows of an odd width, norms with mean and bias, everything in fp32
        {"name": "join_bwd_4099x1001_layer", "op": "join", "dir": "bwd", "T": 4099, "D": 1001, "kind": "layer", "x": "f32", "r": "f32", "gate": "vector", "scale": True},
        # that block's training micro-batch backwards
        {"name": "join_bwd_49152x768_token", "op": "join", "dir": "bwd", "T": 49152, "D": 768, "kind": "rms", "x": "bf16", "r": "f32", "gate": "token", "scale": False},
        # a prompt's ragged batch in a serving program: states go in and come out
        {"name": "recur_fwd_1000x770", "op": "recur", "dir": "fwd", "T": 1000, "D": 770, "type": "bf16", "docs": 90, "h0": True},
        # one long sequence, its state kept
        {"name": "recur_fwd_131072x768_one", "op": "recur", "dir": "fwd", "T": 131072, "D": 768, "type": "bf16", "docs": 0, "h0": False},
        # forward and backward of the small fp32 configuration's micro-step
        {"name": "recur_train_2048x768_f32", "op": "recur", "dir": "train", "T": 2048, "D": 768, "type": "f32", "docs": 512, "h0": False},
        # forward and backward of a training micro-batch of packed documents
        {"name": "recur_train_49152x768", "op": "recur", "dir": "train", "T": 49152, "D": 768, "type": "bf16", "docs": 512, "h0": False},
        # one token of one sequence
        {"name": "recur_step_1x768", "op": "step", "n": 1, "D": 768, "type": "bf16", "pool": 0},
        # a serving batch whose sequences lie anywhere in a pool of states, some places of the batch unused
        {"name": "recur_step_500x2048_pool", "op": "step", "n": 500, "D": 2048, "type": "bf16", "pool": 1024},
    ]


def _spread(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "join", "recur", "step"])
    D = rng.choice([768, _spread(rng, 16, 4096)])
    if op == "step":
        n = _spread(rng, 1, 1024)
        return {"op": op, "n": n, "D": D, "type": rng.choice(["f32", "bf16"]), "pool": rng.choice([0, _spread(rng, n, 2048)])}
    T = _spread(rng, 1, max(1, min(65536, 49152 * 768 // D)))
    if op == "recur":
        return {"op": op, "dir": rng.choice(["fwd", "train"]), "T": T, "D": D, "type": rng.choice(["f32", "bf16"]),
                "docs": rng.choice([0, _spread(rng, 1, 2048)]), "h0": rng.random() < 0.5}
    x, r = rng.choice([("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
    case = {"op": op, "dir": rng.choice(["fwd", "bwd"]), "T": T, "D": D, "kind": rng.choice(["rms", "layer"]), "x": x, "r": r}
    return case if op == "norm" else {**case, "gate": rng.choice(["none", "vector", "token"]), "scale": rng.random() < 0.5}


def work(case):
    op, D = case["op"], case["D"]
    if op == "step":
        e = 4 if case["type"] == "f32" else 2
        return {"bytes": case["n"] * D * (4 * e + 8), "flops": 25 * case["n"] * D}
    n = case["T"] * D
    if op == "recur":
        e = 4 if case["type"] == "f32" else 2
        # training: x, r, i in and y out, then dy in and three gradients out (its inputs were read once)
        return {"bytes": n * e * (4 if case["dir"] == "fwd" else 8), "flops": (25 if case["dir"] == "fwd" else 75) * n}
    e, f = (4 if case[k] == "f32" else 2 for k in ("x", "r"))
    if op == "norm":
        return {"bytes": n * (f + e) if case["dir"] == "fwd" else n * (3 * f + e), "flops": (6 if case["dir"] == "fwd" else 14) * n}
    token = case["gate"] == "token"
    if case["dir"] == "fwd":
        return {"bytes": n * (2 * f + 2 * e + (e if token else 0)), "flops": 14 * n}
    return {"bytes": n * (3 * f + 3 * e + (2 * e if token else 0) + (f if case["scale"] else 0)), "flops": 40 * n}


def _sequences(T, mean, gen):
    """The places where packed documents of `mean` positions on average (at most four times that) begin, and the end; the last
    entries are unused (documents of no position), as a program with a fixed number of entries has them."""
    most = 2 * (T // mean) + 4
    length = (torch.empty(most, device="cuda").exponential_(generator=gen) * mean).clamp(1, 4 * mean).long()
    ends = length.cumsum(0).clamp(max=T)
    ends[-1] = T
    return torch.cat([ends.new_zeros(1), ends]).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    D = case["D"]

    def normal(*shape, dtype=torch.float32, std=1.0, mean=0.0):
        return torch.randn(*shape, device="cuda", generator=gen).mul_(std).add_(mean).to(dtype)

    s = {"case": case}
    if case["op"] in ("recur", "step"):
        t = _TYPES[case["type"]]
        n = case["n"] if case["op"] == "step" else case["T"]
        for k in ("x", "r", "i"):
            s[k] = normal(n, D, dtype=t)
        # the slowest decay of a channel lies between 0.9 and 0.999 a position
        decay = torch.rand(D, dtype=torch.float64, device="cuda", generator=gen) * 0.099 + 0.9
        s["lam"] = torch.log(torch.expm1(-torch.log(decay) / C)).float()
        if case["op"] == "step":
            s["state"] = normal(case["pool"] or n, D)
            s["slots"] = None
            if case["pool"]:
                slots = torch.randperm(case["pool"], device="cuda", generator=gen)[:n].to(torch.int32)
                unused = torch.rand(n, device="cuda", generator=gen) < 0.05
                s["slots"] = torch.where(unused, torch.full_like(slots, -1), slots)
            return s
        s["offsets"] = _sequences(n, case["docs"], gen) if case["docs"] else None
        sequences = s["offsets"].numel() - 1 if case["docs"] else 1
        s["h0"] = normal(sequences, D) if case["h0"] else None
        if case["dir"] == "train":
            s["dy"] = normal(n, D, dtype=t, std=1.0 / 64)
        return s
    T, x, r = case["T"], _TYPES[case["x"]], _TYPES[case["r"]]
    # a residual stream: some channels many times the others
    wide = 1.0 + 8.0 * (torch.rand(D, device="cuda", generator=gen) < 0.02)
    s["R"] = (normal(T, D) * wide).to(r)
    s["w"] = normal(D, std=0.1, mean=1.0)
    s["b"] = normal(D, std=0.1) if case["kind"] == "layer" else None
    if case["op"] == "join":
        s["B"] = normal(T, D, dtype=x, std=0.5)
        s["post_w"] = normal(D, std=0.1, mean=1.0)
        s["post_b"] = normal(D, std=0.1) if case["kind"] == "layer" else None
        s["gate"] = {"none": lambda: None, "vector": lambda: normal(D, std=0.2, mean=0.5), "token": lambda: normal(T, D, dtype=x)}[case["gate"]]()
        s["scale"] = normal(D, std=0.05, mean=0.9) if case["scale"] else None
    if case["dir"] == "bwd":
        s["dX"] = normal(T, D, dtype=x, std=1.0 / 64)
        s["dR1"] = normal(T, D, dtype=r, std=1.0 / 64)
        if case["op"] == "join":   # what the forward left in the residual stream
            s["R1"] = _join(s)[0].to(r)
    return s


# ---------------------------------------------------------------- the framework's calls

_kept = {}   # the configuration and workspace of the last case, as a training program keeps its own


def _plan(key, make):
    if key not in _kept:
        _kept.clear()
        _kept[key] = make()
    return _kept[key]


def _own_norm(s):
    from sparse_hashed_gram_amd import norm
    c = s["case"]

    def make():
        gate, scale = (c["gate"], "vector" if c["scale"] else "none") if c["op"] == "join" else ("none", "none")
        cfg = norm.config(c["D"], kind=c["kind"], x_dtype=c["x"], r_dtype=c["r"], gate=gate, scale=scale, eps=EPS)
        return cfg, norm.Workspace(cfg) if c["dir"] == "bwd" else None

    cfg, ws = _plan(tuple(sorted(c.items())), make)
    if c["op"] == "norm":
        if c["dir"] == "fwd":
            return norm.fwd(cfg, s["R"], s["w"], s["b"])
        return norm.bwd(cfg, ws, s["R"], s["dX"], s["w"], s["b"], dR1=s["dR1"])
    p = {k: s[k] for k in ("post_w", "post_b", "gate", "scale", "w", "b")}
    if c["dir"] == "fwd":
        return norm.join_fwd(cfg, s["R"], s["B"], **p)
    return norm.join_bwd(cfg, ws, s["R"] if c["scale"] else None, s["B"], s["R1"], s["dX"], s["dR1"], **p)


def _own_recur(s):
    from sparse_hashed_gram_amd import recur
    c = s["case"]

    def make():
        cfg = recur.config(c["D"], max_tokens=c["T"], dtype=c["type"], c=C)
        return cfg, recur.Workspace(cfg)

    cfg, ws = _plan(tuple(sorted(c.items())), make)
    x, r, i, lam = s["x"], s["r"], s["i"], s["lam"]
    if c["dir"] == "fwd":
        return recur.fwd(cfg, ws, x, r, i, lam, offsets=s["offsets"], h0=s["h0"], final=True)[:2]
    y, _, saved = recur.fwd(cfg, ws, x, r, i, lam, offsets=s["offsets"], h0=s["h0"], keep=True)
    return {"y": y, **recur.bwd(cfg, ws, x, r, i, lam, saved, s["dy"], offsets=s["offsets"], h0=s["h0"])}


def _own_step(s):
    from sparse_hashed_gram_amd import recur
    c = s["case"]
    cfg = _plan(tuple(sorted(c.items())), lambda: recur.config(c["D"], max_tokens=c["n"], dtype=c["type"], c=C))
    return recur.step(cfg, s["x"], s["r"], s["i"], s["lam"], s["state"], slots=s["slots"]), s["state"]


def run(s):
    op = s["case"]["op"]
    if own:
        return _own_recur(s) if op == "recur" else _own_step(s) if op == "step" else _own_norm(s)
    return _plain_recur(s) if op == "recur" else _plain_step(s) if op == "step" else _plain_norm(s)


# ---------------------------------------------------------------- the plain forms

def _normed(v, kind):
    """(the normalised rows, 1 / deviation)."""
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    rho = torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)
    return v * rho, rho


def _affine(v, w, b):
    return v * w if b is None else v * w + b


def _unnormed(d, xh, rho, kind):
    """The gradient in front of a norm from the one behind it."""
    back = d - xh * (d * xh).mean(1, keepdim=True)
    if kind == "layer":
        back = back - d.mean(1, keepdim=True)
    return back * rho


def _gamma(s):
    gate, kind = s["gate"], s["case"]["gate"]
    return 1.0 if kind == "none" else gate if kind == "vector" else 1.0 / (1.0 + torch.exp(-gate.float()))


def _join(s):
    """R1 and X in 32 bits."""
    kind = s["case"]["kind"]
    N = _affine(_normed(s["B"].float(), kind)[0], s["post_w"], s["post_b"])
    R = s["R"].float() if s["scale"] is None else s["R"].float() * s["scale"]
    R1 = R + _gamma(s) * N
    return R1, _affine(_normed(R1, kind)[0], s["w"], s["b"])


def _plain_norm(s):
    c = s["case"]
    kind, x, r = c["kind"], _TYPES[c["x"]], _TYPES[c["r"]]
    if c["dir"] == "fwd":
        if c["op"] == "norm":
            return _affine(_normed(s["R"].float(), kind)[0], s["w"], s["b"]).to(x)
        R1, X = _join(s)
        return R1.to(r), X.to(x)
    dX = s["dX"].float()
    xh, rho = _normed(s["R" if c["op"] == "norm" else "R1"].float(), kind)
    back = s["dR1"].float() + _unnormed(dX * s["w"], xh, rho, kind)
    out = {"dw": (dX * xh).sum(0)}
    if s["b"] is not None:
        out["db"] = dX.sum(0)
    if c["op"] == "norm":
        return {"dR": back.to(r), **out}
    nh, rho = _normed(s["B"].float(), kind)
    gamma = _gamma(s)
    dN = back * gamma
    out["dpost_w"] = (dN * nh).sum(0)
    if s["post_b"] is not None:
        out["dpost_b"] = dN.sum(0)
    if c["gate"] == "vector":
        out["dgate"] = (back * _affine(nh, s["post_w"], s["post_b"])).sum(0)
    elif c["gate"] == "token":
        out["dgate"] = (back * _affine(nh, s["post_w"], s["post_b"]) * gamma * (1.0 - gamma)).to(x)
    out["dB"] = _unnormed(dN * s["post_w"], nh, rho, kind).to(x)
    if s["scale"] is None:
        return {"dR": back.to(r), **out}
    return {"dR": (back * s["scale"]).to(r), "dscale": (back * s["R"].float()).sum(0), **out}


def _gates(x, r, i, lam):
    """(a, m, sigmoid(i), sigmoid(r), softplus(lam)) in 32 bits, m = sqrt(1 - a^2)."""
    sp = torch.clamp(lam, min=0.0) + torch.log1p(torch.exp(-lam.abs()))
    rho, g = (1.0 / (1.0 + torch.exp(-v.float())) for v in (r, i))
    z = -C * sp * rho
    return torch.exp(z), torch.sqrt(-torch.expm1(2.0 * z)), g, rho, sp


def _scan(a, u):
    """h_t = a_t h_{t-1} + u_t down the rows, by doubling."""
    d = 1
    while d < u.shape[0]:
        u = torch.cat([u[:d], u[d:] + a[d:] * u[:-d]])
        a = torch.cat([a[:d], a[d:] * a[:-d]])
        d *= 2
    return u


def _where(s):
    """(truth values [T, 1]: a sequence begins here; the sequence of each position; the offsets)."""
    T = s["x"].shape[0]
    off = torch.tensor([0, T], device="cuda") if s["offsets"] is None else s["offsets"].long()
    t = torch.arange(T, device="cuda")
    seq = torch.searchsorted(off, t, right=True) - 1
    return (off[seq] == t)[:, None], seq, off


def _plain_recur(s):
    c = s["case"]
    typ = _TYPES[c["type"]]
    x = s["x"].float()
    a, m, g, rho, sp = _gates(x, s["r"], s["i"], s["lam"])
    begins, seq, off = _where(s)
    cut = torch.where(begins, torch.zeros_like(a), a)
    u = m * g * x
    first = 0.0 if s["h0"] is None else s["h0"][seq]
    h = _scan(cut, u if s["h0"] is None else torch.where(begins, u + a * first, u))
    if c["dir"] == "fwd":
        some = (off[1:] > off[:-1])[:, None]
        last = h[(off[1:] - 1).clamp(min=0)]
        return h.to(typ), torch.where(some, last, torch.zeros_like(last) if s["h0"] is None else s["h0"])
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    before = torch.where(begins, torch.zeros_like(h) if s["h0"] is None else first, before)
    onward = torch.cat([cut[1:], torch.zeros_like(cut[:1])])
    G = _scan(onward.flip(0), s["dy"].float().flip(0)).flip(0)
    dz = G * a * before - G * g * x * a * a / m
    dsp = (-C * rho * dz).sum(0)
    out = {"y": h.to(typ), "dx": (G * m * g).to(typ), "di": (G * m * x * g * (1.0 - g)).to(typ),
           "dr": (-C * sp * dz * rho * (1.0 - rho)).to(typ), "dlam": dsp / (1.0 + torch.exp(-s["lam"]))}
    if s["h0"] is not None:
        some = (off[1:] > off[:-1])[:, None]
        at = off[:-1].clamp(max=x.shape[0] - 1)
        out["dh0"] = torch.where(some, (a * G)[at], torch.zeros_like(s["h0"]))
    return out


def _plain_step(s):
    x = s["x"].float()
    a, m, g, _, _ = _gates(x, s["r"], s["i"], s["lam"])
    if s["slots"] is None:
        s["state"].copy_(a * s["state"] + m * g * x)
        return s["state"].to(s["x"].dtype), s["state"]
    used = s["slots"] >= 0
    at = s["slots"].long().clamp(min=0)
    h = a * s["state"][at] + m * g * x
    # an unused place writes to a row behind the pool
    behind = torch.cat([s["state"], torch.zeros_like(h[:1])])
    behind.index_copy_(0, torch.where(used, at, torch.full_like(at, s["state"].shape[0])), h)
    s["state"].copy_(behind[:-1])
    return torch.where(used[:, None], h, torch.zeros_like(h)).to(s["x"].dtype), s["state"]


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_norm(v, kind, w, b):
    """(the norm, d -> the gradient in front of it, the normalised rows)."""
    D = v.shape[1]
    mu = v.sum(1, keepdim=True) / D if kind == "layer" else torch.zeros_like(v[:, :1])
    dev = torch.sqrt((v - mu).square().sum(1, keepdim=True) / D + EPS)
    xh = (v - mu) / dev
    out = xh * w.double()

    def back(d):
        e = d * w.double()
        along = (e * xh).sum(1, keepdim=True) / D
        flat = e.sum(1, keepdim=True) / D if kind == "layer" else torch.zeros_like(along)
        return (e - flat - xh * along) / dev

    return (out if b is None else out + b.double()), back, xh


def _exact_scan(a, u):
    """The recurrence over pieces of 256 rows side by side, then over the pieces."""
    T, D = u.shape
    L = 256
    n = (T + L - 1) // L
    A = torch.ones(n * L, D, dtype=torch.float64, device="cuda")
    H = torch.zeros(n * L, D, dtype=torch.float64, device="cuda")
    A[:T], H[:T] = a, u
    A, H = A.view(n, L, D), H.view(n, L, D)
    for k in range(1, L):
        H[:, k] += A[:, k] * H[:, k - 1]
        A[:, k] *= A[:, k - 1]
    for k in range(1, n):
        H[k] += A[k] * H[k - 1, L - 1]
    return H.view(n * L, D)[:T]


def _exact_recur(case, s):
    sig = torch.sigmoid
    x, r, i, lam = (s[k].double() for k in ("x", "r", "i", "lam"))
    sp = torch.log1p(torch.exp(lam))
    a = torch.exp(-C * sp * sig(r))
    m = torch.sqrt(-torch.expm1(-2.0 * C * sp * sig(r)))
    g = sig(i)
    if case["op"] == "step":
        state = s["state"].double()
        at = range(case["n"]) if s["slots"] is None else s["slots"].tolist()
        rows = torch.tensor([k for k, slot in enumerate(at) if slot >= 0], dtype=torch.long, device="cuda")
        to = torch.tensor([slot for slot in at if slot >= 0], dtype=torch.long, device="cuda")
        y = torch.zeros_like(x)
        y[rows] = a[rows] * state[to] + (m * g * x)[rows]
        state[to] = y[rows]
        return y, state
    T, D = x.shape
    off = [0, T] if s["offsets"] is None else s["offsets"].tolist()
    full = [k for k in range(len(off) - 1) if off[k + 1] > off[k]]
    at = torch.tensor([off[k] for k in full], device="cuda")
    end = torch.tensor([off[k + 1] - 1 for k in full], device="cuda")
    of = torch.tensor(full, device="cuda")
    start = torch.zeros(len(off) - 1, D, dtype=torch.float64, device="cuda") if s["h0"] is None else s["h0"].double()
    u = m * g * x
    w, v = a.clone(), u.clone()
    v[at] += a[at] * start[of]
    w[at] = 0.0
    h = _exact_scan(w, v)
    final = start.clone()
    final[of] = h[end]
    if case["dir"] == "fwd":
        return h, final
    prev = torch.zeros_like(h)
    prev[1:] = h[:-1]
    prev[at] = start[of]
    w[:-1] = w[1:].clone()
    w[-1] = 0.0
    G = torch.flip(_exact_scan(torch.flip(w, [0]), torch.flip(s["dy"].double(), [0])), [0])
    dz = G * (a * prev - g * x * a.square() / m)
    out = {"y": h, "dx": G * m * g, "di": G * u * (1.0 - g), "dr": dz * -C * sp * sig(r) * sig(-r),
           "dlam": (dz * -C * sig(r)).sum(0) * sig(lam)}
    if s["h0"] is not None:
        out["dh0"] = torch.zeros_like(start)
        out["dh0"][of] = a[at] * G[at]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("recur", "step"):
        return _exact_recur(case, s)
    kind = case["kind"]
    R, b = s["R"].double(), s["b"]
    if case["op"] == "join":
        N, back_N, nh = _exact_norm(s["B"].double(), kind, s["post_w"], s["post_b"])
        gamma = {"none": lambda: torch.ones_like(N), "vector": lambda: s["gate"].double().expand_as(N),
                 "token": lambda: torch.sigmoid(s["gate"].double())}[case["gate"]]()
        scale = torch.ones_like(R[0]) if s["scale"] is None else s["scale"].double()
    if case["dir"] == "fwd":
        if case["op"] == "norm":
            return _exact_norm(R, kind, s["w"], b)[0]
        R1 = scale * R + gamma * N
        return R1, _exact_norm(R1, kind, s["w"], b)[0]
    dX = s["dX"].double()
    _, back, xh = _exact_norm(R if case["op"] == "norm" else s["R1"].double(), kind, s["w"], b)
    D1 = s["dR1"].double() + back(dX)
    out = {"dw": torch.einsum("td,td->d", dX, xh)}
    if b is not None:
        out["db"] = dX.sum(0)
    if case["op"] == "norm":
        return {"dR": D1, **out}
    out["dR"] = D1 * scale
    out["dB"] = back_N(D1 * gamma)
    out["dpost_w"] = (D1 * gamma * nh).sum(0)
    if s["post_b"] is not None:
        out["dpost_b"] = (D1 * gamma).sum(0)
    if case["gate"] == "vector":
        out["dgate"] = (D1 * N).sum(0)
    if case["gate"] == "token":
        out["dgate"] = D1 * N * gamma * torch.sigmoid(-s["gate"].double())
    if s["scale"] is not None:
        out["dscale"] = (D1 * R).sum(0)
    return out
