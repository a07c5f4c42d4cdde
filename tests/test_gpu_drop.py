"""GPU parity of counter-based dropout (include/drop.h) and of the n-gram
forward with dropout, against the numpy oracle.

The mask is integer work: exact (a dropped element gives res, or 0, bit for
bit).  A kept one is fl(fl(x c) + res), rounded to the output: c is off by
u = 2^-24 relative from its exact value, the product and the sum by u each, the
last rounding by u (fp32: none of its own) or 2^-8 (bf16), so
|y - exact| <= 2 u |x c| (1 + u) + u |y|, and for bf16 2^-8 (|y| + that) more.
"""
import numpy as np
import pytest
import torch

from oracle import drop as orc

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def D():
    from sparse_hashed_gram_amd import drop
    return drop


def N():
    from sparse_hashed_gram_amd import ngram
    return ngram


def _values(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(DT[dtype])


def _f64(t):
    return t.detach().float().cpu().double().numpy()


def _limit(o, xc, out):
    e = 2 * U * (1 + U) * np.abs(xc) + U * np.abs(o)
    return e + (2.0 ** -8 * (np.abs(o) + e) if out == "bf16" else 0.0) + 2.0 ** -149


def _check(y, x, res, p, seed, off, out):
    k = orc.keep(x.shape[0], x.shape[1], p, seed, off)
    o = orc.dropout(_f64(x), p, seed, off, None if res is None else _f64(res))
    xc = orc.dropout(_f64(x), p, seed, off)
    err = np.abs(_f64(y) - o)
    assert np.all(err <= _limit(o, xc, out))
    rest = np.zeros_like(o) if res is None else _f64(res)
    assert np.array_equal(_f64(y)[~k], rest[~k])   # dropped: exactly what was there


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7), (1, 8), (3, 9), (5, 768), (37, 768), (129, 1001), (300, 26), (2, 4097)])
@pytest.mark.parametrize("xt,yt,with_res", [("f32", "f32", False), ("bf16", "bf16", True), ("bf16", "f32", True),
                                            ("f32", "bf16", False), ("bf16", "bf16", False), ("f32", "f32", True)])
def test_forward(rows, cols, xt, yt, with_res):
    seed, off = 0xFEDCBA9876543210 ^ rows, (5 << 32) + cols
    x = _values((rows, cols), xt, 1)
    res = _values((rows, cols), yt, 2) if with_res else None
    y = D().fwd(D().spec(0.3, seed, off), x.cuda(), residual=None if res is None else res.cuda(), out_dtype=DT[yt])
    assert y.dtype == DT[yt] and y.shape == x.shape
    _check(y, x, res, 0.3, seed, off, yt)


@pytest.mark.parametrize("xt,yt", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
def test_backward_is_the_same_mask(xt, yt):
    dy = _values((65, 771), xt, 3)
    dx = D().bwd(D().spec(0.5, 9, 8), dy.cuda(), out_dtype=DT[yt])
    _check(dx, dy, None, 0.5, 9, 8, yt)


@pytest.mark.parametrize("p", [0.0, 2.0 ** -18, 1.0, 1 - 2.0 ** -18, 0.999])
def test_ends_of_p(p):
    x = _values((33, 96), "f32", 4)
    y = D().fwd(D().spec(p, 1, 2), x.cuda())
    _check(y, x, None, p, 1, 2, "f32")
    if orc.threshold(p) == 0:
        assert torch.equal(y.cpu(), x)
    if orc.threshold(p) == 65536:
        assert torch.count_nonzero(y) == 0


def test_nan_and_inf_stay_out_of_dropped_places():
    x = torch.full((64, 40), float("nan"))
    x[::2] = float("inf")
    k = torch.from_numpy(orc.keep(64, 40, 0.5, 3, 4))
    for dt in (torch.float32, torch.bfloat16):
        res = torch.ones(64, 40, dtype=dt)
        y = D().fwd(D().spec(0.5, 3, 4), x.to(dt).cuda(), residual=res.cuda()).float().cpu()
        assert torch.all(y[~k] == 1)
        assert torch.all(torch.isnan(y[1::2][k[1::2]])) and torch.all(torch.isinf(y[::2][k[::2]]))


def test_in_place_shapes_and_unaligned_rows():
    d = D()
    s = d.spec(0.25, 5, 6)
    x = _values((2, 31, 769), "bf16", 5)
    want = d.fwd(s, x.cuda())
    assert torch.equal(want.reshape(62, 769), d.fwd(s, x.reshape(62, 769).cuda()))   # rows of the last dimension
    y = x.cuda()
    assert d.fwd(s, y, out=y) is y and torch.equal(y, want)
    r = _values((2, 31, 769), "bf16", 6).cuda()
    want_r = d.fwd(s, x.cuda(), residual=r)
    assert torch.equal(d.fwd(s, x.cuda(), residual=r, out=r), want_r) and torch.equal(r, want_r)
    # a contiguous slice that starts at an odd element
    flat = torch.zeros(1 + 62 * 769 + 5, dtype=torch.bfloat16, device="cuda")
    v = flat[1:1 + 62 * 769].view(62, 769)
    v.copy_(x.reshape(62, 769))
    out = torch.full_like(flat, 7.0)
    d.fwd(s, v, out=out[1:1 + 62 * 769].view(62, 769))
    assert torch.equal(out[1:1 + 62 * 769].view(62, 769), want.reshape(62, 769))
    assert out[0] == 7 and torch.all(out[1 + 62 * 769:] == 7)     # nothing beside the tensor
    assert d.fwd(s, x.cuda()[:0]).shape == (0, 31, 769)
    assert d.fwd(s, x.cuda()[:, :, :0]).shape == (2, 31, 0)


def test_refusals_on_the_gpu():
    d = D()
    s, x = d.spec(0.5, 1, 2), torch.zeros(8, 8, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        d.fwd(s, x.t()[:, :4])
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        d.fwd(s, x.half())
    with pytest.raises(TypeError, match="residual"):
        d.fwd(s, x, residual=x.bfloat16(), out=torch.empty_like(x))
    with pytest.raises(ValueError, match="shape"):
        d.fwd(s, x, residual=torch.zeros(4, 8, device="cuda"))
    with pytest.raises(ValueError, match="shape"):
        d.bwd(s, x, out=torch.zeros(8, 9, device="cuda"))
    with pytest.raises(ValueError, match="residual must be a GPU"):
        d.fwd(s, x, residual=torch.zeros(8, 8))
    with pytest.raises(d.DropError) as e:
        d.fwd(d.spec(1.5, 1, 2), x)
    assert e.value.status == -5
    big = torch.zeros(100, device="cuda")
    with pytest.raises(d.DropError) as e:
        d.fwd(s, big[:64], out=big[4:68])
    assert e.value.status == -5
    with pytest.raises(ValueError, match="rng must be a GPU"):
        d.spec(0.5, rng=torch.zeros(2, dtype=torch.int64))


def test_device_rng_and_graph_replays():
    d = D()
    x = _values((50, 768), "bf16", 7)
    xd, res = x.cuda(), torch.zeros(50, 768, device="cuda")
    rng = d.rng_state(123, 456)
    s = d.spec(0.4, 99, 99, rng=rng)           # seed and offset are rng's
    assert torch.equal(d.fwd(s, xd), d.fwd(d.spec(0.4, 123, 456), xd))
    out = torch.empty(50, 768, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        d.fwd(s, xd, residual=res, out=out)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        d.fwd(s, xd, residual=res, out=out)
    for seed, off in [(1, 2), ((1 << 64) - 1, 1 << 40), (1, 3)]:
        d.rng_state(seed, off, out=rng)
        g.replay()
        torch.cuda.synchronize()
        eager = d.fwd(d.spec(0.4, seed, off), xd, residual=res)
        assert torch.equal(out, eager)
        _check(out, x, torch.zeros(50, 768), 0.4, seed, off, "f32")


@pytest.mark.parametrize("rows,cols", [((1 << 32) + 300, 1), ((1 << 29) + 77, 9)])
def test_offsets_past_32_bits(rows, cols):
    # over 2^32 groups, and over 2^32 elements in fewer: the first, middle and last rows
    d = D()
    x = torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")
    d.fwd(d.spec(0.5, 21, 22), x, out=x)
    for lo in (0, (1 << 32) // cols - 100, rows - 200):
        k = orc.keep_rows(np.arange(lo, lo + 200), cols, 0.5, 21, 22)
        assert np.array_equal(_f64(x[lo:lo + 200]), np.where(k, 2.0, 0.0)), lo


# ------------------------------------------------------------ the embedding

def _tables(n, dtype, rows):
    return [_values((rows[c], 768), dtype, 30 + c).cuda() for c in range(n)]


@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 500, 2048])
@pytest.mark.parametrize("dtype,out_f32,direct", [("f32", False, False), ("bf16", False, False), ("bf16", True, False),
                                                  ("f32", False, True), ("bf16", False, True), ("bf16", True, True)])
def test_embedding_with_dropout(T, dtype, out_f32, direct):
    n, d = N(), D()
    rows = (300, 1) if direct else (211, 389)
    cfg = n.config(300, 7, rows, dtype, max_tokens=T, out_f32=out_f32, direct=direct)
    W = _tables(2, dtype, rows)
    tok = torch.from_numpy(np.random.default_rng(T).integers(0, 300, T).astype(np.int32)).cuda()
    s = d.spec(0.2, 77, 1 << 33)
    got = n.embed_fwd_drop(cfg, W[0], None if direct else W[1], tok, s)
    assert got.dtype == cfg.out_torch_dtype
    # the exact fp32 sum (the plain forward with an fp32 output), dropped by the numpy oracle
    full = n.embed_fwd(n.config(300, 7, rows, dtype, max_tokens=T, out_f32=True, direct=direct), W[0],
                       None if direct else W[1], tok) if not direct else W[0][tok.long()].float()
    _check(got, full.cpu(), None, 0.2, 77, 1 << 33, "f32" if got.dtype == torch.float32 else "bf16")
    # and, bit for bit, the two calls one after the other
    assert torch.equal(got, d.fwd(s, full, out_dtype=got.dtype))


def test_embedding_longer_than_one_launch_of_blocks():
    # more positions than the grid's blocks hold at once (8 each, 2^23 blocks)
    n, d = N(), D()
    T = (1 << 26) + 77
    cfg = n.config(300, 7, (300, 1), "bf16", max_tokens=T, direct=True)
    W = _tables(1, "bf16", (300,))[0]
    tok = torch.randint(0, 300, (T,), dtype=torch.int32, device="cuda")
    got = n.embed_fwd_drop(cfg, W, None, tok, d.spec(0.5, 8, 9))
    for lo in (0, (1 << 26) - 40, T - 50):
        k = torch.from_numpy(orc.keep_rows(np.arange(lo, lo + 50), 768, 0.5, 8, 9)).cuda()
        want = torch.where(k, 2.0 * W[tok[lo:lo + 50].long()].float(), 0.0)
        assert torch.equal(got[lo:lo + 50].float(), want), lo


def test_embedding_without_dropout_is_the_plain_forward():
    n, d = N(), D()
    cfg = n.config(300, 7, (211, 389), "bf16", max_tokens=200)
    W = _tables(2, "bf16", (211, 389))
    tok = torch.randint(0, 300, (200,), dtype=torch.int32, device="cuda")
    assert torch.equal(n.embed_fwd_drop(cfg, W[0], W[1], tok, d.spec(0.0)), n.embed_fwd(cfg, W[0], W[1], tok))
    assert n.embed_fwd_drop(cfg, W[0], W[1], tok[:0], d.spec(0.5)).shape == (0, 768)


def test_embedding_bad_token_flag_and_bad_shapes():
    n, d = N(), D()
    cfg = n.config(300, 7, (211, 389), "f32", max_tokens=64)
    ws = n.Workspace(cfg)
    W = _tables(2, "f32", (211, 389))
    tok = torch.zeros(64, dtype=torch.int32, device="cuda")
    n.embed_fwd_drop(cfg, W[0], W[1], tok, d.spec(0.5), ws=ws)
    assert n.device_status(cfg, ws) == 0
    tok[40] = 300
    n.embed_fwd_drop(cfg, W[0], W[1], tok, d.spec(0.5), ws=ws)
    assert n.device_status(cfg, ws) == n.FLAG_BAD_TOKEN
    with pytest.raises(ValueError, match="table 0"):
        n.embed_fwd_drop(cfg, W[1], W[0], tok, d.spec(0.5))
    with pytest.raises(ValueError, match="out must have shape"):
        n.embed_fwd_drop(cfg, W[0], W[1], tok, d.spec(0.5), out=torch.zeros(63, 768, device="cuda"))


def test_window_with_dropped_gradients():
    # forward dropped, dY dropped in place, window and step: the tables move by
    # what the plain path gives for the masked gradient
    n, d = N(), D()
    T, rows = 200, (211, 389)
    tok = torch.randint(0, 300, (T,), dtype=torch.int32, device="cuda")
    dY = torch.randn(T, 768, device="cuda")
    s = d.spec(0.3, 4, 5)
    masked = (torch.from_numpy(orc.keep(T, 768, 0.3, 4, 5)).cuda() * (dY * float(orc.scale(0.3)))).contiguous()
    got = []
    for grad in (d.bwd(s, dY.clone()), masked):
        cfg = n.config(300, 7, rows, "f32", max_tokens=T)
        ws, W = n.Workspace(cfg), _tables(2, "f32", rows)
        st = [n.new_state(r) for r in rows]
        n.embed_bwd_accum(cfg, ws, tok, grad)
        n.sparse_step(cfg, ws, W[0], W[1], st[0], st[1], 1, 0.01, 0.95, 1e-8)
        got.append(W)
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert not torch.equal(got[0][0], _tables(2, "f32", rows)[0])


def test_other_stream():
    d = D()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        x = torch.full((4000, 768), 1.0, device="cuda")
        for _ in range(20):
            x = x * 1.0
        y = d.fwd(d.spec(0.5, 6, 7), x)
    side.synchronize()
    k = torch.from_numpy(orc.keep(4000, 768, 0.5, 6, 7)).cuda()
    assert torch.equal(y, torch.where(k, 2.0, 0.0))
