"""CPU checks of the dropout C ABI (include/drop.h) and of
ngram_embed_fwd_drop: exports, layout, and refusals before any HIP call."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "drop.h")
P = 1 << 12       # fake device addresses: never dereferenced on these paths
Q = 1 << 30


@pytest.fixture(scope="module")
def D():
    from sparse_hashed_gram_amd import drop
    return drop


def test_exports_layout_version(D):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(drop_[a-z_]+)\s*\(", src)))
    assert names == ["drop_abi_version", "drop_bwd", "drop_fwd", "drop_status_string"]
    for n in names:
        assert hasattr(D.lib(), n)
    assert D.lib().drop_abi_version() == 1
    assert ctypes.sizeof(D.DropSpec) == 32 and D.DropSpec.rng.offset == 24
    for s in (0, -1, -2, -4, -5, -6):
        assert D.status_string(s) not in ("", "unknown status")
    assert D.status_string(-99) == "unknown status"


@pytest.mark.parametrize("p,reserved", [(-0.1, 0), (1.0000001, 0), (float("nan"), 0), (float("inf"), 0), (0.1, 1)])
def test_bad_spec(D, p, reserved):
    s = D.DropSpec(p, reserved, 1, 2, None)
    assert D.lib().drop_fwd(s, P, 0, None, Q, 0, 4, 4, None) == -5
    assert D.lib().drop_bwd(s, P, 0, Q, 0, 4, 4, None) == -5


def test_host_rejections_enqueue_nothing(D):
    L = D.lib()
    s = D.spec(0.5, 1, 2)
    f = L.drop_fwd
    assert f(None, P, 0, None, Q, 0, 4, 4, None) == -1
    assert f(s, None, 0, None, Q, 0, 4, 4, None) == -1
    assert f(s, P, 0, None, None, 0, 4, 4, None) == -1
    assert f(s, P + 2, 0, None, Q, 0, 4, 4, None) == -2          # fp32 at a 2-byte address
    assert f(s, P + 1, 1, None, Q, 1, 4, 4, None) == -2
    assert f(s, P, 1, Q + 2, 2 * Q, 0, 4, 4, None) == -2
    assert f(s, P, 2, None, Q, 0, 4, 4, None) == -5
    assert f(s, P, 0, None, Q, -1, 4, 4, None) == -5
    assert f(s, P, 0, None, Q, 0, -1, 4, None) == -4
    assert f(s, P, 0, None, Q, 0, 4, -1, None) == -4
    assert f(s, P, 0, None, Q, 0, 1, 1 << 31, None) == -4
    assert f(s, P, 0, None, Q, 0, (1 << 40) // 3 + 1, 3, None) == -4
    assert f(s, P, 0, None, P + 16, 0, 4, 4, None) == -5         # y over part of x
    assert f(s, P, 1, None, P, 0, 4, 4, None) == -5              # in place needs one dtype
    assert f(s, P, 1, Q, Q + 4, 0, 4, 4, None) == -5             # y over part of res
    assert f(s, None, 0, None, None, 0, 0, 4, None) == 0         # nothing to do
    assert f(s, None, 0, None, None, 0, 4, 0, None) == 0
    r = D.DropSpec(0.5, 0, 1, 2, P + 8)
    assert f(r, P, 0, None, Q, 0, 4, 4, None) == -2              # rng not 16-byte aligned


def test_binding_refuses(D):
    s = D.spec(0.5, 1, 2)
    with pytest.raises(ValueError, match="GPU tensor"):
        D.fwd(s, torch.zeros(3, 4))
    with pytest.raises(ValueError, match="64-bit"):
        D.spec(0.5, -1, 0)
    with pytest.raises(ValueError, match="64-bit"):
        D.spec(0.5, 0, 1 << 64)
    with pytest.raises(ValueError, match="rng"):
        D.spec(0.5, rng=torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="dimension"):
        D.fwd(s, torch.zeros(()))


def test_embed_fwd_drop_rejects_as_embed_fwd_does(D):
    from sparse_hashed_gram_amd import ngram as N
    L, c = N.lib(), N.config(50304, 50256, (4096, 4096), "f32", max_tokens=64)
    s = D.spec(0.1, 1, 2)
    f = L.ngram_embed_fwd_drop
    assert f(c, P, P, P, 65, s, Q, None, None) == -4
    assert f(c, None, P, P, 10, s, Q, None, None) == -1
    assert f(c, P, None, P, 10, s, Q, None, None) == -1
    assert f(c, P, P, None, 10, s, Q, None, None) == -1
    assert f(c, P, P, P, 10, None, Q, None, None) == -1
    assert f(c, P, P, P, 10, s, None, None, None) == -1
    assert f(c, P + 4, P, P, 10, s, Q, None, None) == -2
    assert f(c, P, P, P, 10, D.DropSpec(2.0, 0, 0, 0, None), Q, None, None) == -5
    assert f(c, P, P, P, 10, D.DropSpec(0.5, 0, 0, 0, P + 4), Q, None, None) == -2
    assert f(c, P, P, None, 0, s, None, None, None) == 0
    c.dim = 512
    assert f(c, P, P, P, 10, s, Q, None, None) == -3


def test_generator_state_inside_the_results_is_refused(D):
    # a block could write over the state before another has read it
    from sparse_hashed_gram_amd import ngram as N
    n = 10 * 768 * 4
    for at in (Q, Q + n - 16):
        r = D.DropSpec(0.5, 0, 1, 2, at)
        assert D.lib().drop_fwd(r, P, 0, None, Q, 0, 10, 768, None) == -5
        assert D.lib().drop_bwd(r, P, 0, Q, 0, 10, 768, None) == -5
        c = N.config(50304, 50256, (4096, 4096), "f32", max_tokens=64)
        assert N.lib().ngram_embed_fwd_drop(c, P, P, P, 10, r, Q, None, None) == -5
