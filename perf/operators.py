"""Cases that measure the counter-based dropout, the n-gram embedding with dropout and the gated feed-forward block.

Every case runs in two ways on the same inputs: ``own = False`` computes the operator from elementary torch operations in 32 bits,
``own = True`` makes the calls a training or serving program makes of ``sparse_hashed_gram_amd``.

Dropout: element j of row r belongs to group r ceil(cols / 8) + j // 8; Philox4x32-10 (Salmon et al. 2011) of (group, offset) under
the seed gives the group 128 bits, 16 for each of its 8 elements, low half of word 0 first.  An element is kept iff its 16 bits are
at least round(65536 p), and a kept one is scaled by 65536 / (65536 - round(65536 p)).
"""
import functools
import math

import numpy as np
import torch

own = False

D = 768
VOCAB, EOS = 50304, 50256
_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
_MOST_TF = 49152 * 2048   # positions x hidden units of the largest feed-forward case


def listed():
    return [
        # one short document's activations, a launch-bound call
        {"name": "drop_fwd_37x768_bf16", "op": "drop", "dir": "fwd", "rows": 37, "cols": 768, "x": "bf16", "y": "bf16", "res": False, "p": 0.1},
        # a training micro-batch's branch output, dropped and added to the fp32 residual stream
        {"name": "drop_fwd_49152x768_res", "op": "drop", "dir": "fwd", "rows": 49152, "cols": 768, "x": "bf16", "y": "f32", "res": True, "p": 0.1},
        # the gradient of the largest micro-step's embedding output on its way to the tables
        {"name": "drop_bwd_393216x768_bf16", "op": "drop", "dir": "bwd", "rows": 393216, "cols": 768, "x": "bf16", "y": "bf16", "res": False, "p": 0.1},
        # rows of an odd width: groups end inside a row, rows start unaligned
        {"name": "drop_fwd_4099x1001_f32", "op": "drop", "dir": "fwd", "rows": 4099, "cols": 1001, "x": "f32", "y": "f32", "res": False, "p": 0.25},
        # the small fp32 tables' micro-step
        {"name": "embed_2048_f32", "op": "embed", "T": 2048, "rows": 4096, "dtype": "f32", "p": 0.1},
        # one shard's micro-step out of 16 GB of bf16 tables
        {"name": "embed_49152_bf16", "op": "embed", "T": 49152, "rows": 5287500, "dtype": "bf16", "p": 0.1},
        # one token of a serving loop
        {"name": "ffn_fwd_1x2048", "op": "ffn_fwd", "T": 1, "F": 2048, "act": "silu", "res": True, "p": 0.0},
        # a ragged batch, hidden units that end inside a tile
        {"name": "ffn_fwd_3001x2056_gelu", "op": "ffn_fwd", "T": 3001, "F": 2056, "act": "gelu", "res": False, "p": 0.0},
        # a training micro-batch with residual dropout
        {"name": "ffn_fwd_49152x2048_drop", "op": "ffn_fwd", "T": 49152, "F": 2048, "act": "silu", "res": True, "p": 0.1},
        # a short ragged batch's backward, a narrow block
        {"name": "ffn_bwd_257x1000_relu2", "op": "ffn_bwd", "T": 257, "F": 1000, "act": "relu2", "p": 0.0},
        # an accumulation step of a smaller batch
        {"name": "ffn_bwd_8192x2304_gelu", "op": "ffn_bwd", "T": 8192, "F": 2304, "act": "gelu", "p": 0.1},
        # the training micro-batch's backward
        {"name": "ffn_bwd_49152x2048_drop", "op": "ffn_bwd", "T": 49152, "F": 2048, "act": "silu", "p": 0.1},
    ]


def _spread(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["drop", "embed", "ffn_fwd", "ffn_bwd"])
    p = rng.choice([0.05, 0.1, 0.2, 0.5])
    if op == "drop":
        rows = _spread(rng, 1, 393216)
        cols = rng.choice([768, _spread(rng, 1, 4096)])
        rows = max(1, min(rows, 393216 * 384 // cols))
        fwd = rng.random() < 0.5
        x = rng.choice(["f32", "bf16"])
        y = rng.choice(["f32", "bf16"]) if fwd else x
        return {"op": op, "dir": "fwd" if fwd else "bwd", "rows": rows, "cols": cols, "x": x, "y": y, "res": fwd and rng.random() < 0.5, "p": p}
    if op == "embed":
        dtype = rng.choice(["f32", "bf16"])
        return {"op": op, "T": _spread(rng, 1, 98304), "rows": _spread(rng, 97, 5287500 if dtype == "bf16" else 1048576), "dtype": dtype, "p": p}
    T = _spread(rng, 1, 49152)
    F = 8 * _spread(rng, 16, max(16, min(1024, _MOST_TF // T // 8)))
    case = {"op": op, "T": T, "F": F, "act": rng.choice(["silu", "gelu", "relu2"]), "p": p if rng.random() < 0.5 else 0.0}
    return {**case, "res": rng.random() < 0.5} if op == "ffn_fwd" else case


def work(case):
    if case["op"] == "drop":
        n = case["rows"] * case["cols"]
        el = {"f32": 4, "bf16": 2}
        return {"bytes": n * (el[case["x"]] + el[case["y"]] * (2 if case["res"] else 1)), "flops": n}
    if case["op"] == "embed":
        el = 4 if case["dtype"] == "f32" else 2
        # rows that occur more than once are read once: at most the tables
        rows = min(2 * case["T"], 2 * case["rows"])
        return {"bytes": case["T"] * (D * el + 4) + rows * D * el, "flops": 2 * case["T"] * D}
    T, F = case["T"], case["F"]
    if case["op"] == "ffn_fwd":
        return {"bytes": 2 * (T * D * (3 if case["res"] else 2) + 3 * D * F), "flops": 6 * T * D * F}
    return {"bytes": 2 * (3 * T * D + 6 * D * F), "flops": 16 * T * D * F}   # both projections again, dH, dX, three weights


def _zipf_tokens(T, gen):
    """Zipf(1.1) ids with documents of 512 positions on average, each opened by the end-of-sequence id."""
    cdf = torch.arange(1, VOCAB + 1, dtype=torch.float64, device="cuda").pow(-1.1).cumsum(0)
    u = torch.rand(T, dtype=torch.float64, device="cuda", generator=gen)
    tok = torch.searchsorted(cdf / cdf[-1], u).clamp(max=VOCAB - 1).to(torch.int32)
    opens = torch.rand(T, device="cuda", generator=gen) < 1.0 / 512
    opens[:1] = True
    return torch.where(opens, torch.full_like(tok, EOS), tok)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))

    def normal(*shape, dtype=torch.bfloat16, std=1.0):
        return torch.randn(*shape, dtype=dtype, device="cuda", generator=gen).mul_(std)

    # the generator's state of this step: the run's seed and the step's own offset
    s = {"case": case, "seed": (int(seed) * 0x9E3779B97F4A7C15 + 0x1234567) % (1 << 64), "offset": int(seed) % 1000003 + (1 << 33)}
    if case["op"] == "drop":
        s["x"] = normal(case["rows"], case["cols"], dtype=_TYPES[case["x"]])
        s["res"] = normal(case["rows"], case["cols"], dtype=_TYPES[case["y"]]) if case["res"] else None
    elif case["op"] == "embed":
        dt = _TYPES[case["dtype"]]
        s["W"] = [normal(case["rows"], D, dtype=dt, std=0.02) for _ in range(2)]
        s["tok"] = _zipf_tokens(case["T"], gen)
    else:
        T, F = case["T"], case["F"]
        s["X"] = normal(T, D)
        s["Wg"], s["Wu"] = normal(F, D, std=D ** -0.5), normal(F, D, std=D ** -0.5)
        s["Wd"] = normal(D, F, std=F ** -0.5)
        if case["op"] == "ffn_bwd":
            s["dY"] = normal(T, D, std=1.0 / 64)
        else:
            s["res"] = normal(T, D) if case["res"] else None
    return s


# ---------------------------------------------------------------- the framework's calls

_kept = {}   # one workspace of each configuration, as a training program keeps it


def _spec(s):
    from sparse_hashed_gram_amd import drop
    return drop.spec(s["case"]["p"], s["seed"], s["offset"])


def _own_drop(s):
    from sparse_hashed_gram_amd import drop
    c = s["case"]
    if c["dir"] == "bwd":
        return drop.bwd(_spec(s), s["x"])
    return drop.fwd(_spec(s), s["x"], residual=s["res"], out_dtype=_TYPES[c["y"]])


def _own_embed(s):
    from sparse_hashed_gram_amd import ngram
    c = s["case"]
    cfg = ngram.config(VOCAB, EOS, (c["rows"], c["rows"]), c["dtype"], max_tokens=c["T"])
    return ngram.embed_fwd_drop(cfg, s["W"][0], s["W"][1], s["tok"], _spec(s))


def _own_ffn(s):
    from sparse_hashed_gram_amd import ffn
    c = s["case"]
    key = (c["op"], c["T"], c["F"], c["act"])
    if key not in _kept:
        _kept.clear()
        cfg = ffn.config(c["F"], max_tokens=c["T"], act=c["act"])
        _kept[key] = cfg, ffn.Workspace(cfg)
    cfg, ws = _kept[key]
    drop = _spec(s) if c["p"] else None
    if c["op"] == "ffn_fwd":
        return ffn.fwd(cfg, ws, s["X"], s["Wg"], s["Wu"], s["Wd"], residual=s["res"], drop=drop)
    return ffn.bwd(cfg, ws, s["X"], s["Wg"], s["Wu"], s["Wd"], s["dY"], drop=drop)


def run(s):
    op = s["case"]["op"]
    if own:
        return _own_drop(s) if op == "drop" else _own_embed(s) if op == "embed" else _own_ffn(s)
    return _plain_drop(s) if op == "drop" else _plain_embed(s) if op == "embed" else _plain_ffn(s)


# ---------------------------------------------------------------- the plain forms

_M32 = 0xFFFFFFFF


def _threshold(p):
    return int(np.rint(np.float32(p) * np.float32(65536)))


def _philox_round(c, k):
    a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57   # 64-bit products; the shift's copies of the sign are masked off
    return (((b >> 32) & _M32) ^ c[1] ^ k[0], b & _M32, ((a >> 32) & _M32) ^ c[3] ^ k[1], a & _M32)


def _keep(rows, cols, p, seed, offset):
    """Truth values [rows, cols]: the elements that stay."""
    per = -(-cols // 8)
    g = torch.arange(rows * per, dtype=torch.int64, device="cuda")
    keys = [((seed + r * 0x9E3779B9) & _M32, ((seed >> 32) + r * 0xBB67AE85) & _M32) for r in range(10)]
    word = lambda v: torch.full_like(g, v & _M32)   # noqa: E731
    w = functools.reduce(_philox_round, keys, (g & _M32, g >> 32, word(offset), word(offset >> 32)))
    bits = torch.stack([h for x in w for h in (x & 0xFFFF, x >> 16)], 1)
    return (bits >= _threshold(p)).view(rows, 8 * per)[:, :cols]


def _scale(p):
    return 65536.0 / (65536 - _threshold(p))


def _dropped(v, s):
    """v (32 bits), dropped and scaled."""
    keep = _keep(v.shape[0], v.shape[1], s["case"]["p"], s["seed"], s["offset"])
    return torch.where(keep, v * _scale(s["case"]["p"]), torch.zeros_like(v))


def _plain_drop(s):
    v = _dropped(s["x"].float(), s)
    return (v if s["res"] is None else s["res"].float() + v).to(_TYPES[s["case"]["y"]])


def _mix64(z):
    """SplitMix64's finaliser on wrapping 64-bit words."""
    z = (z ^ ((z >> 30) & ((1 << 34) - 1))) * (0xBF58476D1CE4E5B9 - (1 << 64))
    z = (z ^ ((z >> 27) & ((1 << 37) - 1))) * (0x94D049BB133111EB - (1 << 64))
    return z ^ ((z >> 31) & ((1 << 33) - 1))


def _ngram_rows(tok, R):
    """(row, sign) of both channels: the n-gram ends at each position and does not reach over the start of its document."""
    t = tok.to(torch.int64)
    none = torch.full_like(t, VOCAB)
    opens = t == EOS
    t1, t2 = torch.cat([none[:1], t[:-1]]), torch.cat([none[:2], t[:-2]])[: t.numel()]
    p1 = torch.where(opens, none, t1)
    p2 = torch.where(opens | (t1 == EOS), none, t2)
    B = VOCAB + 1
    found = []
    for key, seed in ((p1 * B + t, 1), ((p2 * B + p1) * B + t, 2)):
        z = _mix64((key ^ seed) + (0x9E3779B97F4A7C15 - (1 << 64)))
        found.append(((((z >> 32) & _M32) * R) >> 32, 1.0 - 2.0 * (z & 1).float()))
    return found


def _plain_embed(s):
    c = s["case"]
    (rb, sb), (rt, st) = _ngram_rows(s["tok"], c["rows"])
    v = s["W"][0][rb].float() * sb[:, None] + s["W"][1][rt].float() * st[:, None]
    return _dropped(v, s).to(_TYPES[c["dtype"]])


_G1, _G3 = math.sqrt(2.0 / math.pi), 0.044715


def _act(g, kind):
    """(a(g), a'(g))."""
    if kind == "silu":
        e = 1.0 / (1.0 + torch.exp(-g))
        return g * e, e * (1.0 + g * (1.0 - e))
    if kind == "gelu":
        th = torch.tanh(_G1 * (g + _G3 * g * g * g))
        return 0.5 * g * (1.0 + th), 0.5 * (1.0 + th) + 0.5 * g * (1.0 - th * th) * _G1 * (1.0 + 3.0 * _G3 * g * g)
    r = torch.clamp(g, min=0.0)
    return r * r, 2.0 * r


def _plain_ffn(s):
    c = s["case"]
    X, Wg, Wu, Wd = (s[k].float() for k in ("X", "Wg", "Wu", "Wd"))
    a, da = _act(X @ Wg.t(), c["act"])
    U = X @ Wu.t()
    H = a * U
    if c["op"] == "ffn_fwd":
        v = H @ Wd.t()
        v = _dropped(v, s) if c["p"] else v
        return (v if s["res"] is None else s["res"].float() + v).to(torch.bfloat16)
    dY = _dropped(s["dY"].float(), s) if c["p"] else s["dY"].float()
    dH = dY @ Wd
    dU, dG = dH * a, dH * U * da
    out = {"dX": dG @ Wg + dU @ Wu, "dWg": dG.t() @ X, "dWu": dU.t() @ X, "dWd": dY.t() @ H}
    return {k: v.to(torch.bfloat16) for k, v in out.items()}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_factor(rows, cols, p, seed, offset):
    """[rows, cols] in 64 bits: 0 for a dropped element, 1 / (kept share) for another.  Products of 32-bit words by 16-bit halves."""
    per = (cols + 7) // 8
    n = rows * per

    def times(m, x):
        lo, hi = m * (x & 0xFFFF), m * (x >> 16)      # below 2^48 each
        s = lo + ((hi & 0xFFFF) << 16)                 # below 2^49
        return (hi >> 16) + (s >> 32), s & _M32        # upper and lower word

    g = torch.arange(n, dtype=torch.int64, device="cuda")
    x = [g % (1 << 32), g // (1 << 32), torch.zeros_like(g) + offset % (1 << 32), torch.zeros_like(g) + offset // (1 << 32)]
    k0, k1 = seed % (1 << 32), seed // (1 << 32)
    for _ in range(10):
        h0, l0 = times(0xD2511F53, x[0])
        h1, l1 = times(0xCD9E8D57, x[2])
        x = [h1 ^ x[1] ^ k0, l1, h0 ^ x[3] ^ k1, l0]
        k0, k1 = (k0 + 0x9E3779B9) % (1 << 32), (k1 + 0xBB67AE85) % (1 << 32)
    thr = _threshold(p)
    out = torch.zeros(rows, per, 8, dtype=torch.float64, device="cuda")
    for j in range(8):
        half = x[j // 2] // (1 << (16 * (j % 2))) % 65536
        out[:, :, j] = (half >= thr).view(rows, per).double() * (65536.0 / (65536.0 - thr))
    return out.view(rows, 8 * per)[:, :cols]


def _exact_rows(tok, R):
    t = tok.cpu().numpy().astype(np.uint64)
    n = len(t)
    B = np.uint64(VOCAB + 1)
    p1 = np.full(n, VOCAB, np.uint64)
    p2 = np.full(n, VOCAB, np.uint64)
    starts = t == EOS
    p1[1:] = np.where(starts[1:], np.uint64(VOCAB), t[:-1])
    p2[2:] = np.where(starts[2:] | starts[1:-1], np.uint64(VOCAB), t[:-2])
    rows = []
    with np.errstate(over="ignore"):
        for key, seed in ((p1 * B + t, 1), ((p2 * B + p1) * B + t, 2)):
            z = (key ^ np.uint64(seed)) + np.uint64(0x9E3779B97F4A7C15)
            z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
            z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
            z ^= z >> np.uint64(31)
            row = ((z >> np.uint64(32)) * np.uint64(R)) >> np.uint64(32)
            rows.append((torch.from_numpy(row.astype(np.int64)).cuda(), torch.from_numpy(np.where(z & np.uint64(1), -1.0, 1.0)).cuda()))
    return rows


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    factor = lambda r, c: _exact_factor(r, c, case["p"], s["seed"], s["offset"])   # noqa: E731
    if op == "drop":
        v = s["x"].double() * factor(case["rows"], case["cols"])
        return v if s["res"] is None else v + s["res"].double()
    if op == "embed":
        (rb, sb), (rt, st) = _exact_rows(s["tok"], case["rows"])
        return (s["W"][0][rb].double() * sb[:, None] + s["W"][1][rt].double() * st[:, None]) * factor(case["T"], D)
    X, Wg, Wu, Wd = (s[k].double() for k in ("X", "Wg", "Wu", "Wd"))
    g, u = X @ Wg.t(), X @ Wu.t()
    if case["act"] == "silu":
        sg = torch.sigmoid(g)
        a, da = g * sg, sg + g * sg * (1.0 - sg)
    elif case["act"] == "gelu":
        c0 = math.sqrt(2.0 / math.pi)
        th = torch.tanh(c0 * (g + 0.044715 * g.pow(3)))
        a, da = g * (1.0 + th) / 2, (1.0 + th) / 2 + g / 2 * (1.0 - th.square()) * c0 * (1.0 + 3 * 0.044715 * g.square())
    else:
        a, da = g.relu().square(), 2.0 * g.relu()
    if op == "ffn_fwd":
        v = (a * u) @ Wd.t()
        v = v * factor(case["T"], D) if case["p"] else v
        return v if s["res"] is None else v + s["res"].double()
    dY = s["dY"].double() * factor(case["T"], D) if case["p"] else s["dY"].double()
    dH = dY @ Wd
    dU, dG = dH * a, dH * u * da
    return {"dX": dG @ Wg + dU @ Wu, "dWg": dG.t() @ X, "dWu": dU.t() @ X, "dWd": dY.t() @ (a * u)}
