"""Refusals of ngram_embed_fwd_drop that concern its workspace, before any HIP call."""


def test_generator_state_in_the_workspace_header_is_refused():
    # a block that meets a bad token sets a flag there, which another would read as the seed
    from sparse_hashed_gram_amd import drop, ngram as N
    P, Q, WS = 1 << 12, 1 << 30, 1 << 40      # fake device addresses: never dereferenced
    c = N.config(50304, 50256, (4096, 4096), "f32", max_tokens=64)
    for at in (WS, WS + 16, WS + 48):
        s = drop.DropSpec(0.5, 0, 1, 2, at)
        assert N.lib().ngram_embed_fwd_drop(c, P, P, P, 10, s, Q, WS, None) == -5
