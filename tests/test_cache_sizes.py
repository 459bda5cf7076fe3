"""Sizes of the decoding entry points whose products leave 64 bits (no GPU needed: refused before any launch)."""

import pytest

import lsh_attention_hash_b200 as lsh

SHAPE = 2
F32, BF16 = 0, 1
A = 0x10000  # aligned, never dereferenced
BIG = [(1 << 22, 1 << 21, 1 << 21), (1 << 30, 1 << 30, 1 << 4), (1 << 30, 1 << 30, 16 + 1), (3 << 29, 1 << 30, 1 << 30),
       (2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1), (1 << 16, 1 << 15, 1)]


@pytest.mark.parametrize("B,H,T", BIG)
def test_products_of_sizes(B, H, T):
    lib = lsh.load_library()
    assert lib.lsh_cache_write(A, A, BF16, B, H, T, 128, None, 0, A, None, A, 4, 64, 64, A, 8, None, None) == SHAPE
    assert lib.lsh_cache_read(A, 8, B, H, T, 128, A, None, A, 4, 64, 64, A, A, BF16, None, None) == SHAPE
    assert lib.lsh_cache_select(A, 8, A, B, H, H, T, 4, A, None, A, 4, 64, 2, 1, 2, A, A, None) == SHAPE
    assert lib.lsh_cache_attend(A, BF16, B, H, H, T, 128, A, 8, A, None, A, 4, 64, 64, None, 0, 3, 1, 0.0, A, BF16, A,
                                A, 1 << 40, None) == SHAPE
    # sizes that no call takes need nothing
    assert lib.lsh_cache_attend_workspace_bytes(BF16, B, H, H, T, 128, 1024, 64, 0) == 0
    assert lib.lsh_cache_attend_workspace_bytes(F32, B, H, H, T, 128, 1024, 64, 3) == 0


def test_products_with_lists_tables_and_rounds():
    lib = lsh.load_library()

    def select(**kw):
        a = dict(B=4, Hq=8, H=8, T=4, nr=4, maxp=4, page=64, ns=2)
        a.update(kw)
        return lib.lsh_cache_select(A, 8, A, a["B"], a["Hq"], a["H"], a["T"], a["nr"], A, None, A, a["maxp"], a["page"],
                                    a["ns"], 1, 2, A, A, None)

    assert select(B=1 << 20, H=1 << 10, Hq=1 << 10, T=1) == SHAPE                 # lists of 2
    assert select(B=1 << 10, H=1 << 10, Hq=1 << 10, T=1, maxp=1 << 11) == SHAPE  # scores
    assert select(B=1 << 15, H=1 << 10, Hq=1 << 10, T=1, nr=64, ns=1) == SHAPE   # buckets
    need = lib.lsh_cache_attend_workspace_bytes
    assert need(BF16, 1, 8, 8, 1, 128, 1 << 14, 64, 1 << 24) > 0
    assert need(BF16, 1, 8, 8, 1, 128, 1 << 14, 64, (1 << 24) + 1) == 0          # a list of more than 2^30 positions
    assert need(BF16, 1 << 10, 8, 8, 1, 128, 1 << 14, 16, 1 << 20) == 0
