"""The workspaces' sizes that include/norm.h and include/recur.h state."""
import pytest


@pytest.mark.parametrize("D", [1, 2, 4, 5, 64, 768, 769, 1001, 4096])
def test_norm(D):
    from sparse_hashed_gram_amd import norm
    want = -(-10248 * (-(-D // 4) * 4) // 256) * 256
    for kw in ({}, {"kind": "layer", "x_dtype": "f32"}, {"gate": "token", "scale": "vector", "dp_dtype": "bf16"}):
        assert norm.workspace_bytes(norm.config(D, **kw)) == want


@pytest.mark.parametrize("tokens", [1, 32, 33, 128, 129, 256, 257, 2048, 49152, 1 << 24])
@pytest.mark.parametrize("D", [1, 16, 64, 65, 127, 128, 129, 768, 769, 16384])
def test_recur(D, tokens):
    from sparse_hashed_gram_amd import recur
    E = -(-D // 128) * 128
    for dtype in ("f32", "bf16"):
        cfg = recur.config(D, tokens, dtype)
        for backward, piece, single in ((False, 64, 256), (True, 32, 128)):
            n = 1 if tokens <= single else -(-tokens // piece)
            want = 256 * -(-D // 64) + 8 * E * (n + n // 16 + 1) + (-(-4 * D * n // 256) * 256 if backward else 0)
            assert recur.workspace_bytes(cfg, backward) == want
        if D % 128 == 0 and tokens >= 1 << 16:   # "of wide rows"
            for backward, share in ((False, 1 / 7), (True, 2 / 5)):
                assert abs(recur.workspace_bytes(cfg, backward) / (D * tokens) / share - 1) < 0.1
