"""CPU check of which kernels a call over the 8-bit cache launches: with both, the workspace holds
partial results of either."""
from test_cache_abi import I, L, Z, lib  # noqa: F401


def test_batches_of_uneven_sequences_have_room_for_both_kernels(lib):
    both, one = lib.attn_varlen_cache8_fwd_workspace_size, lib.attn_varlen_cache_fwd_workspace_size
    both.restype = one.restype = Z

    def more(B, P, Hq, Hkv, d, T):
        a = I(B), I(P), I(Hq), I(Hkv), I(d), L(T)
        return both(*a) - one(*a)

    for d in (64, 128, 160):
        rows = 2 * 160 * 8 * (16 + 4 * d)   # of every CTA, both ends of its share
        # by the average all sequences have few rows, but one of them may have nearly all
        for B, Hq, Hkv, T in ((256, 32, 8, 1024), (256, 32, 8, 257), (256, 32, 8, 200), (2, 16, 1, 1), (2, 4, 1, 8)):
            assert more(B, 0, Hq, Hkv, d, T) == rows, (B, Hq, Hkv, T)
        # one token each; more rows on average; prefixes
        for B, P, Hq, Hkv, T in ((256, 0, 32, 8, 256), (1, 0, 16, 1, 1), (256, 0, 32, 8, 1025), (3, 0, 48, 1, 2), (256, 1, 32, 8, 1024)):
            assert more(B, P, Hq, Hkv, d, T) == 0, (B, P, Hq, Hkv, T)
    assert both(I(-1), I(0), I(1), I(1), I(64), L(1)) == 0 and both(I(1), I(0), I(3), I(2), I(64), L(1)) == 0 and both(I(1), I(0), I(1), I(1), I(96), L(1)) == 0
