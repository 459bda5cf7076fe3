"""Refusals of the decoding entry points before any launch (no GPU needed)."""

import pytest
import torch

import lsh_attention_hash_b200 as lsh

OK, INVALID, SHAPE, DTYPE, ALIGN, WORKSPACE, UNSUPPORTED = 0, 1, 2, 3, 4, 5, 8
F32, BF16 = 0, 1
A = 0x10000  # aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    return lsh.load_library()


def _caller(fn, names, args):
    def call(**kw):
        a = list(args)
        for k, val in kw.items():
            a[names.index(k)] = val
        return fn(*a)
    return call


def test_block_bytes(lib):
    f = lib.lsh_cache_block_bytes
    for page in (16, 32, 64, 128, 256):
        for D in (64, 128, 256):
            for group in (32, 64):
                # codes of K and V, scale and zero words of both, K lengths
                assert f(page, D, group) == page * (D + 8 * (D // group) + 4)
    for bad in ((48, 128, 64), (8, 128, 64), (512, 128, 64), (64, 96, 32), (64, 128, 128), (64, 128, 48), (0, 128, 64)):
        assert f(*bad) == 0


def test_write_refusals(lib):
    names = ["k", "v", "dtype", "B", "H", "T", "D", "bk", "nr", "ctx", "new", "table", "maxp", "page", "group",
             "cache", "n_pages", "tags", "stream"]
    call = _caller(lib.lsh_cache_write, names,
                   [A, A, BF16, 2, 3, 0, 128, None, 0, A, None, A, 4, 64, 64, A, 8, None, None])
    assert call() == OK  # no rows: no launch
    assert call(dtype=2) == DTYPE
    assert call(B=-1) == SHAPE
    assert call(T=-1) == SHAPE
    assert call(D=60) == SHAPE
    assert call(D=512) == SHAPE
    assert call(D=96, group=32) == UNSUPPORTED
    assert call(group=128) == UNSUPPORTED
    assert call(group=48) == SHAPE
    assert call(group=0) == SHAPE
    assert call(page=8) == SHAPE
    assert call(page=48) == SHAPE
    assert call(page=512) == SHAPE
    assert call(maxp=1 << 25) == SHAPE          # positions beyond 2^30
    assert call(B=1 << 12, H=1 << 10, T=1 << 10) == SHAPE
    assert call(bk=A) == INVALID                # buckets without tags
    assert call(tags=A) == INVALID
    assert call(bk=A, tags=A, nr=0) == SHAPE
    assert call(bk=A, tags=A, nr=65) == SHAPE
    for p in ("k", "v", "ctx", "table", "cache"):
        assert call(**{p: None}) == INVALID
        assert call(**{p: A + 4}) == ALIGN
    assert call(new=A + 4) == ALIGN
    assert call(bk=A + 8, tags=A, nr=2) == ALIGN
    assert call(bk=A, tags=A, nr=2) == OK
    assert call(B=0, T=5) == OK


def test_read_refusals(lib):
    names = ["cache", "n_pages", "B", "H", "T", "D", "ctx", "new", "table", "maxp", "page", "group", "k", "v",
             "dtype", "inv", "stream"]
    call = _caller(lib.lsh_cache_read, names, [A, 8, 2, 3, 0, 128, A, None, A, 4, 64, 64, A, A, BF16, None, None])
    assert call() == OK
    assert call(dtype=9) == DTYPE
    assert call(n_pages=-1) == SHAPE
    assert call(T=1 << 30) == SHAPE
    assert call(page=24) == SHAPE
    assert call(D=192, group=64) == UNSUPPORTED
    for p in ("cache", "ctx", "table", "k", "v"):
        assert call(**{p: None}) == INVALID
        assert call(**{p: A + 8}) == ALIGN
    assert call(inv=A + 4) == ALIGN
    assert call(new=A + 4) == ALIGN


def test_select_refusals(lib):
    names = ["tags", "n_pages", "qb", "B", "Hq", "H", "T", "nr", "ctx", "new", "table", "maxp", "page", "ns", "nl",
             "mask", "sel", "scores", "stream"]
    call = _caller(lib.lsh_cache_select, names,
                   [A, 8, A, 2, 6, 3, 0, 4, A, None, A, 4, 64, 2, 1, 2, A, A, None])
    assert call() == OK
    assert call(Hq=7) == SHAPE
    assert call(Hq=0) == SHAPE
    assert call(T=-1) == SHAPE
    assert call(nr=0) == SHAPE
    assert call(nr=65) == SHAPE
    assert call(ns=0) == SHAPE
    assert call(nl=3) == SHAPE                   # more local pages than are selected
    assert call(nl=-1) == SHAPE
    assert call(ns=1 << 26) == SHAPE
    assert call(T=1 << 20, maxp=1 << 12) == SHAPE
    assert call(mask=1) == INVALID               # only the causal bit
    assert call(mask=-1) == INVALID
    for p in ("tags", "qb", "ctx", "table", "sel", "scores"):
        assert call(**{p: None}) == INVALID
        assert call(**{p: A + 4}) == ALIGN
    assert call(new=A + 4) == ALIGN
    assert call(Hq=387, T=1) == UNSUPPORTED      # 129 query heads per cached head
    assert call(T=1, maxp=49153, page=16) == UNSUPPORTED


def test_attend_refusals(lib):
    names = ["q", "dtype", "B", "Hq", "H", "T", "D", "cache", "n_pages", "ctx", "new", "table", "maxp", "page",
             "group", "sel", "ns", "mask", "unit", "scale", "out", "out_dtype", "lse", "ws", "ws_bytes", "stream"]
    call = _caller(lib.lsh_cache_attend, names,
                   [A, BF16, 2, 6, 3, 0, 128, A, 8, A, None, A, 4, 64, 64, None, 0, 3, 1, 0.0, A, BF16, A, None, 0,
                    None])
    assert call() == OK
    assert call(dtype=4) == DTYPE
    assert call(out_dtype=4) == DTYPE
    assert call(Hq=5) == SHAPE
    assert call(H=0) == SHAPE
    assert call(D=100) == SHAPE
    assert call(D=96, group=32) == UNSUPPORTED
    assert call(page=20) == SHAPE
    assert call(ns=2) == INVALID                 # a list length without a list
    assert call(sel=A) == INVALID                # a list without a length
    assert call(sel=A, ns=1 << 26) == SHAPE
    assert call(mask=4) == INVALID
    assert call(mask=-1) == INVALID
    assert call(unit=2) == INVALID
    for p in ("q", "cache", "ctx", "table", "out", "lse"):
        assert call(**{p: None}) == INVALID
        assert call(**{p: A + 4}) == ALIGN
    assert call(new=A + 4) == ALIGN
    assert call(sel=A + 4, ns=2) == ALIGN
    need = lib.lsh_cache_attend_workspace_bytes(BF16, 2, 6, 3, 1, 128, 1024, 64, 0)
    assert need > 0
    assert call(T=1, maxp=1024) == WORKSPACE
    assert call(T=1, maxp=1024, ws=A, ws_bytes=need - 1) == WORKSPACE
    assert call(T=1, maxp=1024, ws=A + 4, ws_bytes=need) == ALIGN
    # sizes that no call takes need nothing
    assert lib.lsh_cache_attend_workspace_bytes(BF16, 2, 5, 3, 1, 128, 1024, 64, 0) == 0
    assert lib.lsh_cache_attend_workspace_bytes(7, 2, 6, 3, 1, 128, 1024, 64, 0) == 0


def test_binding_refuses_host_tensors_and_wrong_forms():
    k = torch.zeros(1, 2, 3, 64)
    cache = torch.zeros(4, 2, lsh.lsh_cache_block_bytes(64, 64, 64), dtype=torch.uint8)
    table, ctx = torch.zeros(1, 4, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    for call in (lambda: lsh.lsh_cache_write(k, k, cache, table, ctx),
                 lambda: lsh.lsh_cache_read(cache, table, ctx, 3, 64),
                 lambda: lsh.lsh_cache_attend(k, cache, table, ctx),
                 lambda: lsh.lsh_cache_select(torch.zeros(4, 2, 1, 64, dtype=torch.int16), table, table, ctx, 1)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        lsh.alloc_cache(4, 2, 96, device="cpu")
    cache, tags = lsh.alloc_cache(4, 2, 128, page=32, group=32, n_rounds=3, device="cpu")
    assert cache.shape == (4, 2, 32 * (128 + 32 + 4)) and tags.shape == (4, 2, 3, 32)
