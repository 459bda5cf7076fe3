"""Calls of the decoding operators that their documentation allows and that ordinary use meets rarely: first calls of
a process, several threads, empty problems, pointers between others."""

import os
import subprocess
import sys
import threading

import pytest
import torch

import lsh_attention_hash_b200 as lsh
from tests.test_gpu_cache import DEV, Cache, _check_attend, _status

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _wide_select(pages):
    """The choice of 2 of ``pages`` pages of 64 tokens, 4 rounds (scored by the scoring kernel): page 5 has hits."""
    tags = torch.zeros(2, 1, 4, 64, dtype=torch.int16, device=DEV)
    tags[1] = 9
    table = torch.zeros(1, pages, dtype=torch.int32, device=DEV)
    table[0, 5] = 1
    qb = torch.full((1, 1, 4, 1), 9, dtype=torch.int32, device=DEV)
    ctx = torch.tensor([pages * 64], dtype=torch.int32, device=DEV)
    return lambda: lsh.lsh_cache_select(tags, qb, table, ctx, 2)[0]


FIRST = """
import sys
sys.path.insert(0, {root!r})
from tests.test_gpu_cache_calls import _wide_select
for pages in {pages!r}:
    assert _wide_select(pages)().flatten().tolist() == [5, pages - 1], pages
print("fine")
"""


@pytest.mark.parametrize("pages", [(12160,), (12220,), (12221,), (12288,), (12289,), (49152, 12230, 100)])
def test_select_of_any_width_as_the_first_call(pages):
    """Scores of 12288 pages are 48 KB of shared memory, to which the kernel's own variables come."""
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=ROOT, pages=pages)], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout == "fine\n", r.stderr[-2000:]


def test_selects_of_several_threads():
    """Calls with tables of different widths at once: none lowers what another one's launch needs."""
    widths = [12300, 49152, 20000, 40000]
    calls, wrong = [_wide_select(w) for w in widths], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(300):
                    got = calls[i]()
                if got.flatten().tolist() != [5, widths[i] - 1]:
                    wrong.append((i, got))
        except Exception as e:  # (reported by the test's thread)
            wrong.append((i, e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(widths))]
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and _status() == 0


@pytest.mark.parametrize("which", ["attend", "select", "select wide"])
def test_a_refused_launch_is_reported_once(which):
    """A launch that CUDA refuses (on the legacy stream while a blocking stream captures) is that call's error and
    not also the next one's."""
    import ctypes

    rt = ctypes.CDLL("libcudart.so.12")
    c = Cache(90, B=1, H=1, ctx=(40,), n_rounds=2)
    q, k = c.rand(1, 1, 1, 128).to(DEV), c.k[:, :, -1:].contiguous().to(DEV)
    out, lse = torch.empty_like(q), torch.empty(1, 1, 1, device=DEV)
    pages = 1200 if which == "select wide" else c.max_pages  # (wide: its scoring kernel is refused, then its choice)
    table = torch.zeros(1, pages, dtype=torch.int32, device=DEV)
    qb = torch.zeros(1, 1, 2, 1, dtype=torch.int32, device=DEV)
    sel, scores = (torch.empty(1, 1, 1, n, dtype=torch.int32, device=DEV) for n in (1, pages))

    def call():
        if which == "attend":
            lsh.lsh_cache_attend(q, c.cache, c.table, c.ctx_len, out=out, lse=lse, **c.form)
        else:
            lsh.lsh_cache_select(c.tags, qb, table, c.ctx_len, 1, selected=sel, scores=scores)

    call()
    torch.cuda.synchronize()
    s, graph = ctypes.c_void_p(), ctypes.c_void_p()
    assert torch.cuda.current_stream().cuda_stream == 0
    assert rt.cudaStreamCreate(ctypes.byref(s)) == 0
    assert rt.cudaStreamBeginCapture(s, 2) == 0  # relaxed
    try:
        with pytest.raises(lsh.LSHError, match="LSH_ERR_CUDA"):
            call()
    finally:
        rt.cudaStreamEndCapture(s, ctypes.byref(graph))  # (the capture is void)
        rt.cudaGetLastError()
        rt.cudaStreamDestroy(s)
    lsh.lsh_cache_write(k, k, c.cache, c.table, c.ctx_len, **c.form)
    call()
    torch.cuda.synchronize()
    assert _status() == 0


def test_an_empty_list_of_pages_is_refused():
    """A list without places is not "every page"; a list of -1 answers as no key does."""
    c = Cache(91, B=1, H=2, ctx=(40,))
    q = c.rand(1, 2, 1, 128).to(DEV)
    with pytest.raises(ValueError, match="at least one page"):
        lsh.lsh_cache_attend(q, c.cache, c.table, c.ctx_len,
                             selected=torch.empty(1, 2, 1, 0, dtype=torch.int32, device=DEV), **c.form)
    none = torch.full((1, 2, 1, 1), -1, dtype=torch.int32, device=DEV)
    out, lse = lsh.lsh_cache_attend(q, c.cache, c.table, c.ctx_len, selected=none, **c.form)
    assert (out == 0).all() and torch.isneginf(lse).all() and _status() == 0


def _empty(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device=DEV)


@pytest.mark.parametrize("B,H,T", [(2, 2, 0), (0, 2, 3), (2, 0, 3), (0, 0, 0)])
def test_calls_without_rows(B, H, T):
    """No rows: empty answers of the right shapes, and nothing is written."""
    cache, tags = lsh.alloc_cache(4, H, 128, n_rounds=3, device=DEV)
    cache.fill_(7)
    tags.fill_(7)
    table, ctx = torch.zeros(B, 2, dtype=torch.int32, device=DEV), torch.full((B,), 5, dtype=torch.int32, device=DEV)
    rows, bk = _empty(B, H, T, 128), _empty(B, H, 3, T, dtype=torch.int32)
    lsh.lsh_cache_write(rows, rows, cache, table, ctx, buckets=bk, tags=tags, new_len=ctx)
    k, v, inv = lsh.lsh_cache_read(cache, table, ctx, T, 128)
    assert k.shape == v.shape == (B, H, T, 128) and inv.shape == (B, H, T)
    sel, scores = lsh.lsh_cache_select(tags, bk, table, ctx, 2)
    assert sel.shape == (B, H, T, 2) and scores.shape == (B, H, T, 2)
    for s in (None, sel):
        out, lse = lsh.lsh_cache_attend(rows, cache, table, ctx, selected=s)
        assert out.shape == rows.shape and lse.shape == (B, H, T)
    R = torch.randn(3, 128, 8, device=DEV).bfloat16()
    for n_select in (0, 2):
        out, lse = lsh.lsh_attention_decode(rows, rows, R, 16, cache, tags, table, ctx, n_select=n_select, check=True)
        assert out.shape == rows.shape and lse.shape == (B, H, T)
    assert (cache == 7).all() and (tags == 7).all() and _status() == 0


@pytest.mark.parametrize("n_pages,max_pages", [(4, 0), (0, 0), (0, 2)])
def test_calls_without_pages(n_pages, max_pages):
    """Sequences without a token over tables, or a cache, of no pages: rows are padding."""
    cache, tags = lsh.alloc_cache(n_pages, 2, 64, n_rounds=2, device=DEV)
    cache.fill_(7)
    table = torch.full((2, max_pages), -1, dtype=torch.int32, device=DEV)
    ctx = torch.zeros(2, dtype=torch.int32, device=DEV)
    rows, bk = torch.randn(2, 2, 3, 64, device=DEV).bfloat16(), torch.zeros(2, 2, 2, 3, dtype=torch.int32, device=DEV)
    lsh.lsh_cache_write(rows, rows, cache, table, ctx, buckets=bk, tags=tags)
    k, v, inv = lsh.lsh_cache_read(cache, table, ctx, 3, 64)
    assert (k == 0).all() and (v == 0).all() and (inv == 0).all()
    sel, scores = lsh.lsh_cache_select(tags, bk, table, ctx, 2)
    assert (sel == -1).all() and scores.shape == (2, 2, 3, max_pages) and (scores == -1).all()
    for s in (None, sel):
        out, lse = lsh.lsh_cache_attend(rows, cache, table, ctx, selected=s)
        assert (out == 0).all() and torch.isneginf(lse).all()
    R = torch.randn(2, 64, 8, device=DEV).bfloat16()
    out, lse = lsh.lsh_attention_decode(rows, rows, R, 16, cache, tags, table, ctx, n_select=1, check=True)
    assert (out == 0).all() and torch.isneginf(lse).all()
    assert (cache == 7).all() and _status() == 0
    # tokens that no table has room for, or whose pages the cache lacks, are the caller's error
    out, lse = lsh.lsh_cache_attend(rows, cache, table, ctx + 3)
    assert (out == 0).all() and torch.isneginf(lse).all() and _status() == 1


def test_slices_of_lengths_and_tables():
    """Lengths and tables that start between 16-byte boundaries, as slices of a batch do, in eager calls and in a
    captured one that follows their contents."""
    c = Cache(92, B=3, H=2, ctx=(50, 90, 130), n_rounds=2)
    wide = torch.full((4, 5), -1, dtype=torch.int32, device=DEV)  # odd width: row 1 starts 20 bytes in
    wide[1:, :c.max_pages] = c.table
    ctx = torch.cat([torch.zeros(1, dtype=torch.int32, device=DEV), c.ctx_len])
    new = torch.tensor([0, 2, 1, 0], dtype=torch.int32, device=DEV)
    assert wide[1:].data_ptr() % 16 and ctx[1:].data_ptr() % 16
    k, v = c.rand(3, 2, 2, 128).to(DEV), c.rand(3, 2, 2, 128).to(DEV)
    bk = torch.randint(0, 16, (3, 2, 2, 2), generator=c.g, dtype=torch.int32).to(DEV)

    def step(cache, tags, table, ctx, new):
        lsh.lsh_cache_write(k, v, cache, table, ctx, new_len=new, buckets=bk, tags=tags, **c.form)
        got = list(lsh.lsh_cache_read(cache, table, ctx, 2, 128, new_len=new, **c.form))
        got += lsh.lsh_cache_select(tags, bk, table, ctx, 2, new_len=new)  # got[3]: the selection
        got += lsh.lsh_cache_attend(k, cache, table, ctx, new_len=new, selected=got[3], **c.form)
        got += lsh.lsh_cache_attend(k, cache, table, ctx, new_len=new, **c.form)
        return got + [cache, tags]

    def same(a, b):
        return all(torch.equal(x, y) for x, y in zip(a, b))

    def plain():
        return step(c.cache.clone(), c.tags.clone(), wide[1:].clone(), ctx[1:].clone(), new[1:].clone())

    assert same(step(c.cache.clone(), c.tags.clone(), wide[1:], ctx[1:], new[1:]), plain())
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    cache, tags = c.cache.clone(), c.tags.clone()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        got = step(cache, tags, wide[1:], ctx[1:], new[1:])
    for i in range(3):
        ctx[1:] -= 1
        new[1:] = torch.tensor([1, 2 - i, i], dtype=torch.int32)
        cache.copy_(c.cache)
        tags.copy_(c.tags)
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, plain())
    assert _status() == 0


@pytest.mark.parametrize("T,ctx,causal,self_mask", [(64, 64, True, True), (257, 300, True, True), (257, 300, False, True),
                                                   (257, 300, True, False), (1000, 1100, True, True)])
@pytest.mark.parametrize("dtype,D", [(torch.bfloat16, 128), (torch.float32, 64), (torch.bfloat16, 256)])
def test_prompt_rows_over_the_cache(T, ctx, causal, self_mask, dtype, D):
    """Prompts of hundreds of rows, also over earlier tokens, with a shorter prompt in the batch."""
    c = Cache(93, dtype=dtype, B=2, H=1, D=D, group=64, page=32, ctx=(ctx, ctx // 2))
    new = [T, T // 3]
    q = c.rand(2, 1, T, D, dtype=dtype).to(DEV)
    nl = torch.tensor(new, dtype=torch.int32, device=DEV)
    out, lse = lsh.lsh_cache_attend(q, c.cache, c.table, c.ctx_len, new_len=nl, causal=causal, self_mask=self_mask,
                                    **c.form)
    _check_attend(c, q, out, lse, new, causal=causal, self_mask=self_mask)
    assert _status() == 0
