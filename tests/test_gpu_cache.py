"""The decoding operators on the GPU against the float64 oracle: 4-bit storage, attention over it, page choice.

Storage is exact: every stored value is compared bit for bit.  Attention's bounds are derived in
``_bounds`` from the roundings that the kernels state, never from what they gave.
"""

import numpy as np
import pytest
import torch

import lsh_attention_hash_b200 as lsh
from oracle import cache_oracle as co

pytestmark = pytest.mark.gpu
DEV = "cuda"
INVALID = 1


def np64(t):
    return t.detach().cpu().double().numpy()


class Cache:
    """A cache with random page order, filled with a sequence of rows per batch entry, and its oracle."""

    def __init__(self, seed, dtype=torch.bfloat16, B=2, H=2, D=128, group=64, page=64, ctx=(100, 37), n_rounds=0,
                 n_buckets=16, spare=3, fill=None, rows=None):
        self.g = torch.Generator().manual_seed(seed)
        self.B, self.H, self.D, self.group, self.page = B, H, D, group, page
        self.ctx = list(ctx)
        self.max_pages = max(1, -(-max(max(ctx), 1) // page))
        n = B * self.max_pages + spare
        self.table = torch.randperm(n, generator=self.g)[:B * self.max_pages].to(torch.int32).reshape(
            B, self.max_pages).to(DEV)
        self.cache, self.tags = lsh.alloc_cache(n, H, D, page=page, group=group, n_rounds=n_rounds, device=DEV)
        self.cache.fill_(0xFF if fill is None else fill)  # 0xFF: scales of places never written are NaN
        if self.tags is not None:
            self.tags.fill_(3)
        L = max(max(ctx), 1)
        self.k, self.v = rows if rows is not None else (self.rand(B, H, L, D, dtype=dtype) for _ in range(2))
        self.buckets = torch.randint(0, n_buckets, (B, H, n_rounds, L), generator=self.g, dtype=torch.int32) \
            if n_rounds else None
        self.ctx_len = torch.tensor(self.ctx, dtype=torch.int32, device=DEV)
        self.form = {"page": page, "group": group}
        lsh.lsh_cache_write(self.k.to(DEV), self.v.to(DEV), self.cache, self.table, self.ctx_len,
                            new_len=self.ctx_len, tags=self.tags,
                            buckets=None if self.buckets is None else self.buckets.to(DEV), **self.form)

    def rand(self, *shape, dtype=torch.bfloat16):
        x = torch.randn(*shape, generator=self.g)
        return (x * torch.exp(0.3 * torch.randn(shape[-1], generator=self.g))
                + 0.3 * torch.randn(shape[-1], generator=self.g)).to(dtype)

    def stored(self, b, h):
        n = self.ctx[b]
        k = np64(self.k[b, h, :n])
        return co.oracle_stored(k, self.group), co.oracle_stored(np64(self.v[b, h, :n]), self.group), co.oracle_key_inv(k)


def _status():
    return lsh.lsh_get_device_status()


# ---------------------------------------------------------------------------------------------------
# Storage

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,group,page", [(64, 32, 16), (64, 64, 128), (128, 32, 64), (128, 64, 64), (256, 64, 32),
                                          (256, 32, 256)])
def test_write_then_read_is_exact(dtype, D, group, page):
    c = Cache(1, dtype=dtype, B=3, H=2, D=D, group=group, page=page, ctx=(133, 0, 17))
    for out_dtype in (torch.float32, torch.bfloat16):
        k, v, inv = lsh.lsh_cache_read(c.cache, c.table, c.ctx_len, 140, D, new_len=c.ctx_len, out_dtype=out_dtype,
                                       **c.form)
        for b in range(3):
            n = c.ctx[b]
            assert (k[b, :, n:] == 0).all() and (v[b, :, n:] == 0).all() and (inv[b, :, n:] == 0).all()
            for h in range(2):
                K, V, iv = c.stored(b, h)
                # one rounding of the exact value to the output type
                for got, want in ((k, K), (v, V)):
                    w = want.astype(np.float32) if out_dtype == torch.float32 else co.round_bf16(want)
                    assert np.array_equal(np64(got[b, h, :n]), w.astype(np.float64))
                # sum of D squares in float: D/8 + 5 roundings of 2^-24, square root and quotient
                assert np.allclose(np64(inv[b, h, :n]), iv, rtol=(D / 8 + 8) * 2.0 ** -24, atol=0)
    assert _status() == 0


def test_read_of_the_last_rows():
    c = Cache(2, ctx=(100, 37))
    k, v, _ = lsh.lsh_cache_read(c.cache, c.table, c.ctx_len, 5, 128, **c.form)
    K, V, _ = c.stored(1, 1)
    assert np.array_equal(np64(k[1, 1]), co.round_bf16(K[32:]))
    assert np.array_equal(np64(v[1, 1]), co.round_bf16(V[32:]))
    # more rows than the sequence has: the first are padding
    k, _, inv = lsh.lsh_cache_read(c.cache, c.table, c.ctx_len, 40, 128, **c.form)
    assert (k[1, :, :3] == 0).all() and (inv[1, :, :3] == 0).all()
    assert np.array_equal(np64(k[1, 1, 3:]), co.round_bf16(K))


def _special_rows():
    """fp32 rows of 64 dims whose two groups of 32 hit the quantiser's borders."""
    t = np.arange(32, dtype=np.float64)
    rows = [
        np.zeros(32), np.full(32, -0.0), np.full(32, 3.3), np.full(32, -1e-30), np.full(32, 1e38),
        t, -t, t / 15, t * 0.5,                                   # scale a power of two: every half is a tie
        np.where(t % 2 == 0, 7.5, -7.5) * (t > 3) + 0.0,          # borders at zero
        np.concatenate([[-7.5, 7.5], 1e-10 * (t[:30] - 15)]),     # next to the border at zero, both sides
        np.concatenate([[0.0, 15.0], np.float32(t[:30] * 0.5) + np.float32(2.0 ** -20)]),
        np.concatenate([[0.0, 15.0], np.nextafter(np.float32(t[:30] * 0.5), np.float32(-1))]),
        np.concatenate([[0.0, 15.0], np.nextafter(np.float32(t[:30] * 0.5), np.float32(99))]),
        np.concatenate([[1000.0, 1000.5], 1000.0 + t[:30] / 64]),
        np.concatenate([[0.0, 15 * (1 + 2.0 ** -8)], t[:30] / 3]),      # scale on the middle of two bf16
        np.concatenate([[0.0, 15 * (1 + 3 * 2.0 ** -8)], t[:30] / 3]),
        np.concatenate([[0.0, float(np.nextafter(np.float32(15 * (1 + 2.0 ** -8)), np.float32(99)))], t[:30] / 3]),
        np.concatenate([[0.0, float(np.nextafter(np.float32(15 * (1 + 2.0 ** -8)), np.float32(0)))], t[:30] / 3]),
        t * 2.0 ** -101, t * 2.0 ** -130, t * 2.0 ** -98,
        np.concatenate([[3e38, -3e38], t[:30]]), np.concatenate([[3.3e38, 0.0], t[:30]]),
        np.concatenate([[-3.4e38, 0.0], t[:30]]), np.concatenate([[np.inf, 0.0], t[:30]]),
        np.concatenate([[-np.inf, 0.0], t[:30]]), np.concatenate([[np.nan, 0.0], t[:30]]),
    ]
    x = np.stack(rows).astype(np.float32)
    return np.concatenate([x, x[::-1]], 1)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantiser_borders(dtype):
    x = torch.from_numpy(_special_rows()).to(dtype)[None, None]
    n = x.shape[2]
    c = Cache(3, dtype=dtype, B=1, H=1, D=64, group=32, page=16, ctx=(n,), rows=(x, x.flip(2).contiguous()))
    k, v, inv = lsh.lsh_cache_read(c.cache, c.table, c.ctx_len, n, 64, out_dtype=torch.float32, **c.form)
    K, V, _ = c.stored(0, 0)
    for got, want in ((k, K), (v, V)):
        w = torch.from_numpy(want.astype(np.float32))
        got = got[0, 0].cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(w))
        assert torch.equal(got[~torch.isnan(w)], w[~torch.isnan(w)])


@pytest.mark.parametrize("scale", [1.0, 1e-20, 1e20])
def test_quantiser_many_groups(scale):
    """A few million fp32 and bf16 values on fine and coarse grids: every code as the oracle's."""
    g = torch.Generator().manual_seed(11)
    x = torch.randn(1, 1, 6000, 128, generator=g)
    y = (torch.randn(1, 1, 6000, 128, generator=g) * 8).round() / 8  # many exact ties
    for a, dt in ((x * scale, torch.float32), (y * scale, torch.float32), (x * scale, torch.bfloat16),
                  (y, torch.bfloat16)):
        a = a.to(dt)
        b = a.flip(3).contiguous()
        c = Cache(4, dtype=dt, B=1, H=1, D=128, group=32, page=64, ctx=(6000,), rows=(a, b))
        k, v, _ = lsh.lsh_cache_read(c.cache, c.table, c.ctx_len, 6000, 128, out_dtype=torch.float32, **c.form)
        K, V, _ = c.stored(0, 0)
        assert np.array_equal(k[0, 0].cpu().numpy(), K.astype(np.float32))
        assert np.array_equal(v[0, 0].cpu().numpy(), V.astype(np.float32))


def test_write_changes_only_its_rows():
    """Appending leaves every other byte of the cache and the tags alone; padding rows write nothing."""
    for D, group, page in ((128, 64, 64), (64, 32, 16)):
        c = Cache(5, B=3, H=2, D=D, group=group, page=page, ctx=(90, 40, 21), n_rounds=3)
        before, tags_before = c.cache.clone(), c.tags.clone()
        ctx = torch.tensor([90, 40, 21], dtype=torch.int32, device=DEV)
        new = torch.tensor([5, 0, 2], dtype=torch.int32, device=DEV)
        k, v = c.rand(3, 2, 5, D).to(DEV), c.rand(3, 2, 5, D).to(DEV)
        bk = torch.full((3, 2, 3, 5), 60000, dtype=torch.int32, device=DEV)
        lsh.lsh_cache_write(k, v, c.cache, c.table, ctx, new_len=new, buckets=bk, tags=c.tags, **c.form)
        for b, n in ((0, 5), (1, 0), (2, 2)):
            if n:
                c.k[b, :, c.ctx[b] - n:c.ctx[b]] = k[b, :, :n].cpu()
                c.v[b, :, c.ctx[b] - n:c.ctx[b]] = v[b, :, :n].cpu()
        # the same rows written in one go give the same bytes
        whole = torch.full_like(c.cache, 0xFF)
        lsh.lsh_cache_write(c.k.to(DEV), c.v.to(DEV), whole, c.table, c.ctx_len, new_len=c.ctx_len, **c.form)
        assert torch.equal(whole, c.cache)
        assert not torch.equal(before, c.cache)
        changed = (c.tags != tags_before).sum().item()
        assert changed == 7 * 2 * 3
        assert (c.tags[c.tags != tags_before].to(torch.int32) & 0xFFFF == 60000).all()
    assert _status() == 0


def test_write_bad_pages_and_lengths_are_skipped():
    c = Cache(6, B=2, H=2, ctx=(100, 70), page=64)
    assert _status() == 0
    before = c.cache.clone()
    k, v = c.rand(2, 2, 100, 128).to(DEV), c.rand(2, 2, 100, 128).to(DEV)
    for bad in (-1, c.cache.shape[0], 1 << 30):
        table = c.table.clone()
        table[0] = bad
        lsh.lsh_cache_write(k, v, c.cache, table, torch.tensor([100, 0], dtype=torch.int32, device=DEV), **c.form)
        assert _status() == INVALID
    for length in (-1, 129, 1 << 30):
        ctx = torch.tensor([length, 0], dtype=torch.int32, device=DEV)
        lsh.lsh_cache_write(k, v, c.cache, c.table, ctx, **c.form)
        assert _status() == INVALID
        kk, _, _ = lsh.lsh_cache_read(c.cache, c.table, ctx, 4, 128, **c.form)
        assert (kk == 0).all() and _status() == INVALID
        out, lse = lsh.lsh_cache_attend(k[:, :, :2].contiguous(), c.cache, c.table, ctx, **c.form)
        assert (out == 0).all() and torch.isneginf(lse).all() and _status() == INVALID
    assert torch.equal(before, c.cache)
    # a missing page is left out of the attention, the others count
    table = c.table.clone()
    table[0, 0] = -5
    q = c.rand(2, 2, 1, 128).to(DEV)
    out, lse = lsh.lsh_cache_attend(q, c.cache, table, c.ctx_len, **c.form)
    assert _status() == INVALID
    K, V, inv = c.stored(0, 1)
    want, _, _, _ = co.oracle_cache_attend_row(np64(q[0, 1, 0]), K, V, inv, 99, 100, [1], 64, True, True, True, None)
    assert np.abs(np64(out[0, 1, 0]) - want).max() < 0.05  # both sides of the same softmax, not another's


# ---------------------------------------------------------------------------------------------------
# Attention

def _bounds(q, K, zK, V, zV, sV, w, key_scale, f32_in, f32_out, want):
    """Bound of the output's error per dim, and of the lse's, from the roundings that the kernel states.

    Logit of key j: the code part sum_d q_d (K - z)_jd takes q rounded to half a step, step = max|q| /
    8355711; the integer sums are exact; what float does to the code part and to z's part is
    within 2^-20 of their sizes.  Weights p s go in as fixed-point numbers of the largest of their stage:
    half a step, 1 / 65535 (fp32: 1 / 8388607) of it, times codes of at most 15; the largest of any stage is
    at most the largest of all.  exp2 and the other float steps are within 2^-18 of the sizes.
    """
    step = np.abs(q).max() / 8355711
    code = np.abs(K - zK)
    dz = ((0.5 * step * code.sum(1) + 2.0 ** -20 * ((code + np.abs(zK)) @ np.abs(q))) * key_scale).max() + 2.0 ** -20
    unit = (w[:, None] * sV).max(0) / (8388607 if f32_in else 65535)
    out = w.size * 7.5 * unit + (2 * dz + 2.0 ** -18) * (w @ (np.abs(V - zV) + np.abs(zV)))
    return out + np.abs(want) * (2.0 ** -24 if f32_out else 2.0 ** -8), dz + 2.0 ** -18


def _check_attend(c, q, out, lse, new, selected=None, self_mask=True, causal=True, unit_keys=True, scale=None):
    B, Hq, T, D = q.shape
    G = Hq // c.H
    f32_in, f32_out = q.dtype == torch.float32, out.dtype == torch.float32
    sc = scale if scale else 1 / np.sqrt(D)
    for b in range(B):
        for hq in range(Hq):
            h = hq // G
            K, V, inv = c.stored(b, h)
            if c.ctx[b]:
                _, _, zk = co.oracle_quantise(np64(c.k[b, h, :c.ctx[b]]), c.group)
                _, sv, zv = co.oracle_quantise(np64(c.v[b, h, :c.ctx[b]]), c.group)
                zK, zV, sV = (np.repeat(x, c.group, axis=1) for x in (zk, zv, sv))
            for t in range(T):
                pos = c.ctx[b] - new[b] + t
                got, gl = np64(out[b, hq, t]), float(lse[b, hq, t])
                if t >= new[b] or pos < 0:
                    assert (got == 0).all() and gl == -np.inf, (b, hq, t)
                    continue
                pages = None if selected is None else selected[b, h, t].tolist()
                want, wl, w, keys = co.oracle_cache_attend_row(np64(q[b, hq, t]), K, V, inv, pos, c.ctx[b], pages,
                                                               c.page, self_mask, causal, unit_keys, scale)
                if keys.size == 0:
                    assert (got == 0).all() and gl == -np.inf, (b, hq, t)
                    continue
                ks = sc * (inv[keys] if unit_keys else np.ones(keys.size))
                bound, lb = _bounds(np64(q[b, hq, t]), K[keys], zK[keys], V[keys], zV[keys], sV[keys], w, ks, f32_in,
                                    f32_out, want)
                assert (np.abs(got - want) <= bound).all(), (b, hq, t, np.abs(got - want).max(), bound.min())
                assert abs(gl - wl) <= lb + 2.0 ** -22 * abs(wl), (b, hq, t, gl, wl)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,group,page", [(64, 32, 16), (64, 64, 128), (128, 32, 32), (128, 64, 64), (256, 64, 64),
                                          (256, 32, 256)])
def test_attend_forms(dtype, D, group, page):
    c = Cache(20, dtype=dtype, B=2, H=2, D=D, group=group, page=page, ctx=(301, 45))
    q = c.rand(2, 2, 1, D, dtype=dtype).to(DEV)
    for out_dtype in (torch.bfloat16, torch.float32):
        out, lse = lsh.lsh_cache_attend(q, c.cache, c.table, c.ctx_len, out_dtype=out_dtype, **c.form)
        assert out.dtype == out_dtype
        _check_attend(c, q, out, lse, [1, 1])
    assert _status() == 0


@pytest.mark.parametrize("n", [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513, 1025])
def test_attend_lengths(n):
    c = Cache(21 + n, B=2, H=1, ctx=(n, max(0, n - 1)))
    q = c.rand(2, 1, 1, 128).to(DEV)
    out, lse = lsh.lsh_cache_attend(q, c.cache, c.table, c.ctx_len, **c.form)
    _check_attend(c, q, out, lse, [1, 1])
    assert _status() == 0


@pytest.mark.parametrize("self_mask", [False, True])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("unit_keys", [False, True])
def test_attend_masks(self_mask, causal, unit_keys):
    c = Cache(22, B=3, H=2, page=32, ctx=(70, 3, 33))
    new = [3, 3, 1]
    q = c.rand(3, 4, 3, 128).to(DEV)
    nl = torch.tensor(new, dtype=torch.int32, device=DEV)
    kw = dict(self_mask=self_mask, causal=causal, unit_keys=unit_keys)
    out, lse = lsh.lsh_cache_attend(q, c.cache, c.table, c.ctx_len, new_len=nl, **kw, **c.form)
    _check_attend(c, q, out, lse, new, **kw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("G,T", [(1, 1), (2, 1), (8, 1), (9, 1), (16, 1), (17, 1), (1, 5), (3, 7), (4, 4), (7, 5)])
def test_attend_shared_heads_and_several_tokens(dtype, G, T):
    D = 64 if G > 8 else 128
    c = Cache(23, dtype=dtype, B=2, H=2, D=D, group=32, page=16, ctx=(150, T))
    q = c.rand(2, 2 * G, T, D, dtype=dtype).to(DEV)
    out, lse = lsh.lsh_cache_attend(q, c.cache, c.table, c.ctx_len, scale=0.3, **c.form)
    _check_attend(c, q, out, lse, [T, T], scale=0.3)


def test_attend_more_rows_than_tokens():
    """Rows whose position would be negative are padding."""
    c = Cache(24, B=2, H=1, ctx=(40, 2))
    q = c.rand(2, 1, 5, 128).to(DEV)
    out, lse = lsh.lsh_cache_attend(q, c.cache, c.table, c.ctx_len, **c.form)
    _check_attend(c, q, out, lse, [5, 5])
    assert torch.isneginf(lse[1, 0, :3]).all()


@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("T", [1, 3])
def test_attend_selected_pages(page, T):
    n = 5 * page + 3
    c = Cache(25, B=2, H=2, D=64, group=64, page=page, ctx=(n, page + 1))
    q = c.rand(2, 6, T, 64).to(DEV)
    g = torch.Generator().manual_seed(1)
    sel = torch.randint(-2, 8, (2, 2, T, 7), generator=g, dtype=torch.int32)  # unordered, twice, outside
    sel[0, 0, 0] = -1                                                        # nothing at all
    sel[0, 1, 0] = torch.tensor([5, -1, -1, -1, -1, -1, -1])                  # its own page only
    sel[1, 0, 0] = torch.tensor([2 ** 31 - 1, 1 << 26, -2 ** 31, 0, 0, 1, 1])
    for kw in (dict(), dict(self_mask=False), dict(causal=False)):
        out, lse = lsh.lsh_cache_attend(q, c.cache, c.table, c.ctx_len, selected=sel.to(DEV), **kw, **c.form)
        _check_attend(c, q, out, lse, [T, T], selected=sel, **kw)
    assert _status() == 0


@pytest.mark.parametrize("causal", [False, True])
def test_attend_self_alone_on_its_page(causal):
    """The self rule over selected pages: a page that holds only the token itself."""
    c = Cache(26, B=1, H=1, page=64, ctx=(129,))
    q = c.rand(1, 1, 1, 128).to(DEV)
    for lst in ([2], [2, 2], [2, 9], [2, 0], [0, 2], [1]):
        sel = torch.tensor(lst, dtype=torch.int32).reshape(1, 1, 1, -1)
        out, lse = lsh.lsh_cache_attend(q, c.cache, c.table, c.ctx_len, selected=sel.to(DEV), causal=causal, **c.form)
        _check_attend(c, q, out, lse, [1], selected=sel, causal=causal)


def test_attend_ignores_what_is_masked():
    """NaN rows behind a query's position, and in pages it does not list, change nothing before them."""
    g = torch.Generator().manual_seed(9)
    k, v = torch.randn(1, 2, 96, 128, generator=g), torch.randn(1, 2, 96, 128, generator=g)
    kn, vn = k.clone(), v.clone()
    kn[:, :, 93:] = float("nan")
    vn[:, :, 93:] = float("inf")
    a = Cache(27, B=1, H=2, page=32, ctx=(96,), rows=(k.bfloat16(), v.bfloat16()))
    b = Cache(27, B=1, H=2, page=32, ctx=(96,), rows=(kn.bfloat16(), vn.bfloat16()))
    q = a.rand(1, 2, 6, 128).to(DEV)
    for dt in (torch.bfloat16, torch.float32):
        oa, la = lsh.lsh_cache_attend(q.to(dt), a.cache, a.table, a.ctx_len, **a.form)
        ob, lb = lsh.lsh_cache_attend(q.to(dt), b.cache, b.table, b.ctx_len, **b.form)
        # rows 0..3 are positions 90..93: row 3's own key is NaN, but masked
        assert torch.equal(oa[:, :, :4], ob[:, :, :4]) and torch.equal(la[:, :, :4], lb[:, :, :4])
        assert torch.isnan(ob[:, :, 4:]).all() and torch.isnan(lb[:, :, 4:]).all()
    sel = torch.tensor([0, 1, -1], dtype=torch.int32, device=DEV).expand(1, 2, 6, 3).contiguous()
    oa, _ = lsh.lsh_cache_attend(q, a.cache, a.table, a.ctx_len, selected=sel, causal=False, **a.form)
    ob, _ = lsh.lsh_cache_attend(q, b.cache, b.table, b.ctx_len, selected=sel, causal=False, **b.form)
    assert torch.equal(oa, ob)


def test_attend_extreme_logits():
    """Logits far above and below each other, rising along the sequence, and infinite queries."""
    g = torch.Generator().manual_seed(10)
    k = torch.randn(1, 1, 700, 128, generator=g) * torch.linspace(0.01, 30, 700)[None, None, :, None]
    v = torch.randn(1, 1, 700, 128, generator=g)
    c = Cache(28, B=1, H=1, dtype=torch.float32, ctx=(700,), rows=(k, v))
    q = (5 * torch.randn(1, 1, 2, 128, generator=g)).to(DEV)
    out, lse = lsh.lsh_cache_attend(q, c.cache, c.table, c.ctx_len, unit_keys=False, **c.form)
    _check_attend(c, q, out, lse, [2], unit_keys=False)
    # all logits equal and huge in size
    z = torch.zeros(1, 1, 1, 128, device=DEV)
    out, lse = lsh.lsh_cache_attend(z, c.cache, c.table, c.ctx_len, unit_keys=False, **c.form)
    _check_attend(c, z, out, lse, [1], unit_keys=False)
    out, lse = lsh.lsh_cache_attend(z + float("inf"), c.cache, c.table, c.ctx_len, **c.form)
    assert torch.isnan(out).all()


@pytest.mark.parametrize("shape", [(1, 2, 128, 64, 64, 20001, 1), (2, 1, 64, 32, 16, 9000, 1),
                                   (1, 1, 256, 64, 128, 5000, 2), (1, 2, 128, 64, 64, 12345, 17)])
def test_attend_many_splits(shape):
    B, H, D, group, page, n, G = shape
    c = Cache(29, B=B, H=H, D=D, group=group, page=page, ctx=(n,) + (n // 3,) * (B - 1))
    q = c.rand(B, H * G, 1, D).to(DEV)
    out, lse = lsh.lsh_cache_attend(q, c.cache, c.table, c.ctx_len, **c.form)
    _check_attend(c, q, out, lse, [1] * B)
    again, _ = lsh.lsh_cache_attend(q, c.cache, c.table, c.ctx_len, **c.form)
    assert torch.equal(out, again)  # no atomics: the same sums in the same order


@pytest.mark.parametrize("G", [1, 9, 16, 17, 40])
@pytest.mark.parametrize("D,group", [(128, 64), (64, 32)])
def test_attend_wide_table_short_sequence(G, D, group):
    """A table with room for far more than the sequence holds (entries behind it are garbage); that also takes
    the kernel for much work, with up to 16 columns at a time."""
    c = Cache(30, B=2, H=2, D=D, group=group, ctx=(77, 130))
    wide = torch.full((2, 4096), 1 << 30, dtype=torch.int32, device=DEV)
    wide[:, :c.max_pages] = c.table
    q = c.rand(2, 2 * G, 1, D).to(DEV)
    out, lse = lsh.lsh_cache_attend(q, c.cache, wide, c.ctx_len, **c.form)
    assert _status() == 0
    _check_attend(c, q, out, lse, [1, 1])


def test_cache_offsets_beyond_32_bits():
    """Pages whose bytes lie past 2^32 of the cache."""
    block = lsh.lsh_cache_block_bytes(64, 128, 64)
    n_pages = (1 << 32) // (2 * block) + 40
    cache, tags = lsh.alloc_cache(n_pages, 2, 128, n_rounds=2, device=DEV)
    small = Cache(31, B=1, H=2, ctx=(150,), n_rounds=2)
    table = torch.tensor([[n_pages - 1, n_pages - 9, n_pages - 4]], dtype=torch.int32, device=DEV)
    lsh.lsh_cache_write(small.k.to(DEV), small.v.to(DEV), cache, table, small.ctx_len, buckets=small.buckets.to(DEV),
                        tags=tags)
    k, v, _ = lsh.lsh_cache_read(cache, table, small.ctx_len, 150, 128, out_dtype=torch.float32)
    K, V, _ = small.stored(0, 1)
    assert np.array_equal(k[0, 1].cpu().numpy(), K.astype(np.float32))
    q = small.rand(1, 2, 1, 128).to(DEV)
    out, lse = lsh.lsh_cache_attend(q, cache, table, small.ctx_len)
    _check_attend(small, q, out, lse, [1])
    a, sa = lsh.lsh_cache_select(tags, small.buckets[..., -1:].contiguous().to(DEV), table, small.ctx_len, 2)
    b, sb = lsh.lsh_cache_select(small.tags, small.buckets[..., -1:].contiguous().to(DEV), small.table, small.ctx_len, 2)
    assert torch.equal(a, b) and torch.equal(sa, sb)


# ---------------------------------------------------------------------------------------------------
# Selection

@pytest.mark.parametrize("page,n_rounds,G,T,n_select,n_local,causal,n_buckets", [
    (64, 4, 1, 1, 4, 1, True, 16), (16, 1, 1, 1, 3, 0, True, 2), (16, 8, 3, 2, 5, 5, True, 16),
    (32, 3, 2, 4, 7, 2, False, 65536), (128, 2, 1, 1, 1, 1, True, 4), (256, 64, 1, 1, 2, 0, True, 16),
    (16, 2, 1, 3, 200, 3, True, 16), (64, 8, 1, 1, 1, 0, False, 1024)])
def test_select(page, n_rounds, G, T, n_select, n_local, causal, n_buckets):
    ctx = (9 * page + 5, T, 3 * page, 0)
    c = Cache(40, B=4, H=2, D=64, group=64, page=page, ctx=ctx, n_rounds=n_rounds, n_buckets=n_buckets)
    qb = torch.randint(0, n_buckets, (4, 2 * G, n_rounds, T), generator=c.g, dtype=torch.int32)
    new = [T, T, max(0, T - 1), 0]
    nl = torch.tensor(new, dtype=torch.int32, device=DEV)
    sel, scores = lsh.lsh_cache_select(c.tags, qb.to(DEV), c.table, c.ctx_len, n_select, new_len=nl, n_local=n_local,
                                       causal=causal)
    for b in range(4):
        for h in range(2):
            for t in range(T):
                pos = ctx[b] - new[b] + t if t < new[b] else -1
                tags = c.buckets[b, h, :, :ctx[b]].numpy()
                want, ws = co.oracle_cache_select(tags, qb[b, h * G:(h + 1) * G, :, t].numpy(), pos, ctx[b], page,
                                                  c.max_pages, n_select, n_local, causal)
                assert scores[b, h, t].tolist() == ws, (b, h, t)
                assert sel[b, h, t].tolist() == want, (b, h, t)
    assert _status() == 0


@pytest.mark.parametrize("n_pages", [511, 512, 513, 1500, 20000])
def test_select_many_pages(n_pages):
    """Pages far beyond one per thread, most scores equal."""
    page, n = 16, n_pages * 16 - 3
    tags = torch.zeros(n_pages, 1, 1, page, dtype=torch.int16)
    g = torch.Generator().manual_seed(n_pages)
    hit = torch.randint(0, n_pages, (n_pages // 10,), generator=g)
    tags[hit, 0, 0, 0] = 7
    tags[hit[:5], 0, 0, 1] = 7
    table = torch.randperm(n_pages, generator=g).to(torch.int32)[None]
    logical = tags[table[0].long(), 0]
    qb = torch.full((1, 1, 1, 1), 7, dtype=torch.int32)
    ctx = torch.tensor([n], dtype=torch.int32, device=DEV)
    for n_select, n_local in ((1, 0), (5, 2), (n_pages // 10, 1), (n_pages - 1, 1), (n_pages // 2, 0)):
        sel, _ = lsh.lsh_cache_select(tags.to(DEV), qb.to(DEV), table.to(DEV), ctx, n_select, n_local=n_local)
        want, _ = co.oracle_cache_select(logical.reshape(1, -1)[:, :n].numpy(), qb[0, :, :, 0].numpy(), n - 1, n, page,
                                         n_pages, n_select, n_local, True)
        assert sel[0, 0, 0].tolist() == want


def test_select_buckets_out_of_range_match_nothing():
    c = Cache(41, B=1, H=1, D=64, ctx=(100,), n_rounds=2)
    qb = torch.tensor([-1, 65536 + 3], dtype=torch.int32, device=DEV).reshape(1, 1, 2, 1)
    _, scores = lsh.lsh_cache_select(c.tags, qb, c.table, c.ctx_len, 1)
    assert scores.flatten().tolist() == [0, 0]
    bk = torch.full((1, 1, 2, 1), 65536, dtype=torch.int32, device=DEV)
    assert _status() == 0
    row = c.rand(1, 1, 1, 64).to(DEV)
    lsh.lsh_cache_write(row, row, c.cache, c.table, c.ctx_len, buckets=bk, tags=c.tags, **c.form)
    assert _status() == INVALID


# ---------------------------------------------------------------------------------------------------
# Together, streams, graphs

def _stepwise(dtype, n_select, steps=20, B=2, H=2, D=64, page=16, n_buckets=16, n_rounds=2):
    """Prompt, then tokens one by one; every step against the oracle."""
    g = torch.Generator().manual_seed(50)
    L0 = 37
    L = L0 + steps
    qk, v = torch.randn(B, H, L, D, generator=g).to(dtype), torch.randn(B, H, L, D, generator=g).to(dtype)
    R = torch.randn(n_rounds, D, n_buckets // 2, generator=g).to(dtype).to(DEV)
    c = Cache(51, dtype=dtype, B=B, H=H, D=D, group=32, page=page, ctx=(L,) * B, n_rounds=n_rounds, rows=(qk, v))
    c.cache.fill_(0xFF)
    ctx = torch.full((B,), L0, dtype=torch.int32, device=DEV)
    out, lse = lsh.lsh_attention_decode(qk[:, :, :L0].contiguous().to(DEV), v[:, :, :L0].contiguous().to(DEV), R,
                                        n_buckets, c.cache, c.tags, c.table, ctx, n_select=n_select, check=True,
                                        **c.form)
    c.ctx = [L0] * B
    allb = lsh.lsh_hash(qk.to(DEV), R, n_buckets)[0].cpu()

    def selected(t0, t1):
        if not n_select:
            return None
        s = torch.empty(B, H, t1 - t0, n_select, dtype=torch.int32)
        for b in range(B):
            for h in range(H):
                for t in range(t0, t1):
                    s[b, h, t - t0] = torch.tensor(co.oracle_cache_select(
                        allb[b, h, :, :t1].numpy(), allb[b, h, :, t][None].numpy(), t, t1, page, c.max_pages, n_select,
                        1, True)[0])
        return s

    _check_attend(c, qk[:, :, :L0].to(DEV), out, lse, [L0] * B, selected=selected(0, L0))
    for i in range(steps):
        ctx += 1
        t = L0 + i
        row, vrow = qk[:, :, t:t + 1].contiguous().to(DEV), v[:, :, t:t + 1].contiguous().to(DEV)
        out, lse = lsh.lsh_attention_decode(row, vrow, R, n_buckets, c.cache, c.tags, c.table, ctx, n_select=n_select,
                                            check=True, **c.form)
        c.ctx = [t + 1] * B
        _check_attend(c, row, out, lse, [1] * B, selected=selected(t, t + 1))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n_select", [0, 2])
def test_decoding_step_by_step(dtype, n_select):
    _stepwise(dtype, n_select)


def test_decode_matches_full_causal_lsh_when_one_chunk_covers_all():
    """With one chunk over the whole sequence, causal LSH attention is full attention over the same keys:
    decoding differs by the 4-bit storage alone."""
    g = torch.Generator().manual_seed(60)
    qk, v = torch.randn(1, 2, 64, 128, generator=g), torch.randn(1, 2, 64, 128, generator=g)
    R = torch.randn(1, 128, 8, generator=g)
    full = lsh.lsh_attention(qk.to(DEV), v.to(DEV), R.to(DEV), 16, 64, causal=True)
    cache, tags = lsh.alloc_cache(2, 2, 128, group=32, device=DEV)
    table = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    ctx = torch.tensor([64], dtype=torch.int32, device=DEV)
    out, _ = lsh.lsh_attention_decode(qk.to(DEV), v.to(DEV), None, 16, cache, None, table, ctx, group=32)
    # values are off by half a step of 1/15 of a group's range (about 4), logits by far less than 1
    err = np.abs(np64(out) - np64(full))
    assert err.max() < 0.5 * 5.0 / 15 + 0.25 and err.mean() < 0.1


def test_own_stream_and_graph_replay():
    c = Cache(61, B=2, H=2, ctx=(200, 90), n_rounds=2)
    q = c.rand(2, 2, 1, 128).to(DEV)
    base = lsh.lsh_cache_attend(q, c.cache, c.table, c.ctx_len, **c.form)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    other = lsh.lsh_cache_attend(q, c.cache, c.table, c.ctx_len, stream=s, **c.form)
    s.synchronize()
    assert torch.equal(base[0], other[0])
    # a captured step follows the contents of its tensors, also the lengths
    ctx = c.ctx_len.clone()
    row, vrow = c.rand(2, 2, 1, 128).to(DEV), c.rand(2, 2, 1, 128).to(DEV)
    R = torch.randn(2, 128, 8, device=DEV).bfloat16()
    wide = torch.cat([c.table, torch.tensor([[c.cache.shape[0] - 1], [c.cache.shape[0] - 2]], device=DEV,
                                            dtype=torch.int32)], 1)
    free = sorted(set(range(c.cache.shape[0])) - set(c.table.flatten().tolist()))
    wide[:, -1] = torch.tensor(free[:2], dtype=torch.int32)

    def step():
        return lsh.lsh_attention_decode(row, vrow, R, 16, c.cache, c.tags, wide, ctx, n_select=2, **c.form)

    graph = torch.cuda.CUDAGraph()
    pool = torch.cuda.Stream()
    with torch.cuda.stream(pool):
        step()
        pool.synchronize()
        with torch.cuda.graph(graph, stream=pool):
            got = step()
    torch.cuda.synchronize()
    for i in range(5):
        ctx += 1
        row.copy_(c.rand(2, 2, 1, 128))
        vrow.copy_(c.rand(2, 2, 1, 128))
        cache, tags = c.cache.clone(), c.tags.clone()
        graph.replay()
        torch.cuda.synchronize()
        want = lsh.lsh_attention_decode(row, vrow, R, 16, cache, tags, wide, ctx, n_select=2, **c.form)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(cache, c.cache) and torch.equal(tags, c.tags)
    assert _status() == 0


def test_two_graphs_with_own_workspaces_at_once():
    c = Cache(62, B=1, H=2, ctx=(9000,))
    need = lsh.lsh_cache_attend_workspace_bytes(torch.bfloat16, 1, 2, 2, 1, 128, c.max_pages, 64)
    assert need > 0
    qs = [c.rand(1, 2, 1, 128).to(DEV) for _ in range(2)]
    want = [lsh.lsh_cache_attend(q, c.cache, c.table, c.ctx_len, **c.form)[0] for q in qs]
    graphs, outs, streams = [], [], []
    for q in qs:
        ws = torch.empty(need, dtype=torch.uint8, device=DEV)
        out, lse = torch.empty_like(q), torch.empty(1, 2, 1, device=DEV)
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            lsh.lsh_cache_attend(q, c.cache, c.table, c.ctx_len, workspace=ws, out=out, lse=lse, **c.form)
        graphs.append(gr)
        outs.append((out, ws, lse))
        streams.append(s)
    for _ in range(20):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o[0], w)


def test_joins_with_exact_recent_rows():
    """lse joins the cached part with other key sets through lsh_combine_rounds."""
    c = Cache(63, B=1, H=2, ctx=(160,), page=32)
    q = c.rand(1, 2, 1, 128).to(DEV)
    parts = []
    for pages in ([0, 1, 2], [3, 4]):
        sel = torch.tensor(pages, dtype=torch.int32, device=DEV).expand(1, 2, 1, len(pages)).contiguous()
        parts.append(lsh.lsh_cache_attend(q, c.cache, c.table, c.ctx_len, selected=sel, out_dtype=torch.float32,
                                          **c.form))
    o = torch.stack([p[0] for p in parts], 2)
    l = torch.stack([p[1] for p in parts], 2)
    out, lse = lsh.lsh_combine_rounds(o, l)
    whole, wl = lsh.lsh_cache_attend(q, c.cache, c.table, c.ctx_len, out_dtype=torch.float32, **c.form)
    assert torch.allclose(lse, wl, atol=1e-4) and (out - whole).abs().max() < 2.0 ** -7


# ---------------------------------------------------------------------------------------------------
# Sizes and layouts beyond the ordinary

def test_write_on_16_byte_boundaries():
    """Rows and outputs that start on a 16-byte but not on a 32-byte boundary give the same bytes."""
    c = Cache(70, B=1, H=2, ctx=(75,))
    n = c.k.numel()
    for dt in (torch.bfloat16, torch.float32):
        off = 16 // torch.empty(0, dtype=dt).element_size()
        big = torch.empty(2, n + 2 * off, dtype=dt, device=DEV)
        k, v = (big[i, off:off + n].view(c.k.shape) for i in range(2))
        k.copy_(c.k)
        v.copy_(c.v)
        assert (k.data_ptr() | v.data_ptr()) % 32 == 16 or dt == torch.float32
        other = torch.full_like(c.cache, 0xFF)
        lsh.lsh_cache_write(k, v, other, c.table, c.ctx_len, **c.form)
        assert torch.equal(other, c.cache)
        lsh.lsh_cache_read(c.cache, c.table, c.ctx_len, 75, 128, out_dtype=dt, k=k, v=v, **c.form)
        kk, vv, _ = lsh.lsh_cache_read(c.cache, c.table, c.ctx_len, 75, 128, out_dtype=dt, **c.form)
        assert torch.equal(k, kk) and torch.equal(v, vv)


@pytest.mark.parametrize("B", [33, 70])
def test_many_sequences(B):
    """More sequences than a warp scans at a time, many of them empty, all lengths."""
    g = torch.Generator().manual_seed(B)
    ctx = [int(x) for x in torch.randint(0, 400, (B,), generator=g)]
    ctx[0], ctx[5], ctx[31], ctx[32] = 0, 2000, 0, 1
    c = Cache(71, B=B, H=1, D=64, page=16, ctx=ctx)
    q = c.rand(B, 2, 1, 64).to(DEV)
    out, lse = lsh.lsh_cache_attend(q, c.cache, c.table, c.ctx_len, **c.form)
    _check_attend(c, q, out, lse, [1] * B)
    sel = torch.randint(0, 125, (B, 1, 1, 70), generator=g, dtype=torch.int32)
    out, lse = lsh.lsh_cache_attend(q, c.cache, c.table, c.ctx_len, selected=sel.to(DEV), **c.form)
    _check_attend(c, q, out, lse, [1] * B, selected=sel)


def test_long_pieces_of_small_pages():
    """A CTA's stretch of the keys longer than the pages it looks up at a time (256 of 16 tokens)."""
    n, H, D = 500000, 8, 64
    g = torch.Generator(device=DEV).manual_seed(72)
    k = torch.randn(1, H, n, D, generator=g, device=DEV).bfloat16()
    v = torch.randn(1, H, n, D, generator=g, device=DEV).bfloat16()
    q = torch.randn(1, H, 1, D, generator=g, device=DEV).bfloat16()
    ctx = torch.tensor([n], dtype=torch.int32, device=DEV)
    got = []
    for page in (16, 256):
        pages = -(-n // page)
        cache, _ = lsh.alloc_cache(pages, H, D, page=page, device=DEV)
        table = torch.randperm(pages, generator=g, device=DEV).int()[None]
        lsh.lsh_cache_write(k, v, cache, table, ctx, page=page)
        got.append(lsh.lsh_cache_attend(q, cache, table, ctx, page=page, out_dtype=torch.float32))
        K, V, inv = lsh.lsh_cache_read(cache, table, ctx, n, D, page=page, out_dtype=torch.float32)
    K, V, inv = (t[0, :, :-1].double() for t in (K, V, inv))
    z = torch.einsum("hnd,hd->hn", K, q[0, :, 0].double()) * inv / 8
    want = torch.einsum("hn,hnd->hd", torch.softmax(z, 1), V)
    for out, lse in got:
        # weights in 1/65535 of their stage's largest, codes to 15, scales to 0.5; over 500000 keys
        # their roundings, half a step each and independent, add up to far less than the 2^-12 asked for
        assert (out[0, :, 0].double() - want).abs().max() < 2.0 ** -12
        assert (lse[0, :, 0].double() - torch.logsumexp(z, 1)).abs().max() < 1e-5


@pytest.mark.parametrize("v_size", [1e-25, 1e25, 1e35])
def test_attend_value_range(v_size):
    """Values far from 1 in size; some rows far larger than the others, at keys that hardly count."""
    g = torch.Generator().manual_seed(73)
    k, v = torch.randn(1, 1, 300, 64, generator=g), torch.randn(1, 1, 300, 64, generator=g) * v_size
    v[:, :, ::7] *= 1e-6
    c = Cache(74, B=1, H=1, D=64, dtype=torch.float32, ctx=(300,), rows=(k, v))
    for dt in (torch.float32, torch.bfloat16):
        q = torch.randn(1, 1, 1, 64, generator=g).to(dt).to(DEV)
        out, lse = lsh.lsh_cache_attend(q, c.cache, c.table, c.ctx_len, out_dtype=torch.float32, **c.form)
        _check_attend(c, q, out, lse, [1])


def test_steps_on_another_stream_keep_their_buffers():
    """What a call on a given stream allocates is not handed out again while that stream still uses it."""
    c = Cache(75, B=2, H=4, ctx=(6000, 3000))
    q = c.rand(2, 4, 1, 128).to(DEV)
    want, _ = lsh.lsh_cache_attend(q, c.cache, c.table, c.ctx_len, **c.form)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for i in range(30):
        outs.append(lsh.lsh_cache_attend(q, c.cache, c.table, c.ctx_len, stream=s, **c.form)[0])
        torch.empty(1 << 20, dtype=torch.uint8, device=DEV).fill_(0xFF)  # would reuse a workspace freed too early
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_binding_checks_on_the_device():
    c = Cache(76, B=1, H=2, ctx=(40,))
    q = c.rand(1, 2, 1, 128).to(DEV)
    with pytest.raises(ValueError):
        lsh.lsh_cache_attend(q, c.cache, c.table, c.ctx_len, page=32)           # another form's block
    with pytest.raises(ValueError):
        lsh.lsh_cache_attend(q, c.cache, c.table, c.ctx_len.long(), **c.form)
    with pytest.raises(ValueError):
        lsh.lsh_cache_attend(q, c.cache, c.table, c.ctx_len.cpu(), **c.form)
    with pytest.raises(ValueError):
        lsh.lsh_cache_attend(q.transpose(1, 3), c.cache, c.table, c.ctx_len, **c.form)
    with pytest.raises(ValueError):
        lsh.lsh_cache_attend(q.half(), c.cache, c.table, c.ctx_len, **c.form)
    with pytest.raises(ValueError):
        lsh.lsh_cache_attend(q, c.cache, c.table.repeat(2, 1), c.ctx_len, **c.form)
    with pytest.raises(lsh.LSHError):
        lsh.lsh_cache_attend(c.rand(1, 3, 1, 128).to(DEV), c.cache, c.table, c.ctx_len, **c.form)  # 3 heads over 2
    with pytest.raises(lsh.LSHError):
        lsh.lsh_cache_attend(q, c.cache, c.table, c.ctx_len, group=128, page=64)
    with pytest.raises(ValueError):
        lsh.lsh_cache_write(q, q[:, :1].contiguous(), c.cache, c.table, c.ctx_len, **c.form)
    with pytest.raises(ValueError):
        lsh.lsh_cache_select(c.cache, c.table, c.table, c.ctx_len, 1)
    many = torch.zeros(3, 2, 1, 128, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):
        lsh.lsh_cache_write(many, many, c.cache, c.table, c.ctx_len, **c.form)
    table = torch.zeros(1, 40, dtype=torch.int32, device=DEV)  # more than 1024 keys: a workspace
    with pytest.raises(lsh.LSHError):
        lsh.lsh_cache_attend(q, c.cache, table, c.ctx_len, workspace=torch.empty(16, dtype=torch.uint8, device=DEV),
                             **c.form)
    assert _status() == 0


@pytest.mark.parametrize("page,n_rounds,G,T", [(64, 4, 1, 1), (64, 8, 1, 2), (128, 8, 1, 1), (32, 8, 1, 1), (64, 16, 1, 3),
                                              (64, 8, 2, 1), (64, 6, 1, 1)])
def test_select_with_its_own_scoring_kernel(page, n_rounds, G, T):
    """More tags a head than the choice scores itself: whole batches of pages, a cut one, a missing one."""
    n = 701 * page - 5 if page < 128 else 333 * page + 1
    n_pages = -(-n // page)
    g = torch.Generator().manual_seed(page + n_rounds)
    tags = torch.randint(0, 40, (n_pages + 1, 2, n_rounds, page), generator=g, dtype=torch.int16)
    table = torch.randperm(n_pages, generator=g).to(torch.int32)[None]
    qb = torch.randint(0, 40, (1, 2 * G, n_rounds, T), generator=g, dtype=torch.int32)
    ctx = torch.tensor([n], dtype=torch.int32, device=DEV)
    logical = tags[table[0].long()].permute(1, 2, 0, 3).reshape(2, n_rounds, -1)[:, :, :n].numpy().copy()
    for bad_page, bad_bucket in ((False, False), (True, False), (False, True)):
        tb, q, lg = table.clone(), qb.clone(), logical.copy()
        if bad_page:
            tb[0, 17] = n_pages + 9
            lg[:, :, 17 * page:18 * page] = -1
        if bad_bucket:
            q[0, 0, 0, 0] = 70000
        sel, scores = lsh.lsh_cache_select(tags.to(DEV), q.to(DEV), tb.to(DEV), ctx, 40, n_local=2)
        for h in range(2):
            for t in range(T):
                want, ws = co.oracle_cache_select(lg[h], q[0, h * G:(h + 1) * G, :, t].numpy(), n - T + t, n, page,
                                                  n_pages, 40, 2, True)
                assert scores[0, h, t].tolist() == ws
                assert sel[0, h, t].tolist() == want
        assert _status() == (INVALID if bad_page else 0)
