"""How exactly attention over the cache and its storage answer: bounds tighter than the output's rounding, and
sizes of keys, values and lengths at the ends of what the entry points promise."""

from fractions import Fraction

import numpy as np
import pytest
import torch

import lsh_attention_hash_b200 as lsh
from oracle import cache_oracle as co
from tests.test_gpu_cache import DEV, Cache, _check_attend, _status, np64

pytestmark = pytest.mark.gpu

FORMS = [(64, 32, 16), (64, 64, 128), (128, 32, 32), (128, 64, 64), (256, 64, 64), (256, 32, 256)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,group,page", FORMS)
@pytest.mark.parametrize("G,wide", [(1, False), (1, True), (2, False), (8, True), (17, True)])
def test_a_lone_key_gives_its_stored_value(dtype, D, group, page, G, wide):
    """Softmax over one key is 1: the output is the stored value, rounded once.

    The weight 1 * s and its products with codes are exact (8 + 4 bits), the zero joins in float: z + s c has one
    rounding to 24 bits, as the oracle's value has on its way to float32; bf16 rounds that once more.
    """
    c = Cache(80, dtype=dtype, B=2, H=2, D=D, group=group, page=page, ctx=(1, 1))
    table = torch.full((2, 2048 // page + 1), 1 << 30, dtype=torch.int32, device=DEV) if wide else c.table.clone()
    table[:, :1] = c.table
    q = c.rand(2, 2 * G, 1, D, dtype=dtype).to(DEV)
    for out_dtype in (torch.float32, torch.bfloat16):
        out, _ = lsh.lsh_cache_attend(q, c.cache, table, c.ctx_len, unit_keys=False, out_dtype=out_dtype, **c.form)
        for b in range(2):
            for h in range(2):
                want = torch.from_numpy(c.stored(b, h)[1][0].astype(np.float32)).to(out_dtype)
                assert torch.equal(out[b, h * G:(h + 1) * G, 0].cpu(), want.expand(G, D))
    assert _status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,group,page", FORMS)
@pytest.mark.parametrize("G,wide", [(1, False), (2, True), (4, False), (16, True)])
def test_weights_keep_the_precision_of_floats(dtype, D, group, page, G, wide):
    """A few keys of very different weights, plain keys, float32 answers to either type of query.

    A weight p s is a whole number of steps of at most 2^-22 of the largest one, so n keys' roundings take n half
    steps times a code of 15 at most: n * 15 * 2^-23 of the largest p s.  Of the logits: half a step of the
    query (its largest entry / 8355711) per dim, and what float does to parts of their sizes, 2^-20; the
    exponential's argument is rounded to 2^-24 of its size and the result to 2^-22.  Sums of n floats: n 2^-24.
    """
    n = 20
    c = Cache(81, dtype=dtype, B=1, H=2, D=D, group=group, page=page, ctx=(n,))
    table = torch.full((1, 2048 // page + 1), 1 << 30, dtype=torch.int32, device=DEV) if wide else c.table.clone()
    table[:, :c.max_pages] = c.table
    q = (c.rand(1, 2 * G, 1, D) * 2).to(dtype).to(DEV)
    out, lse = lsh.lsh_cache_attend(q, c.cache, table, c.ctx_len, unit_keys=False, self_mask=False,
                                    out_dtype=torch.float32, **c.form)
    for hq in range(2 * G):
        h = hq // G
        K, V, inv = c.stored(0, h)
        _, _, zk = co.oracle_quantise(np64(c.k[0, h, :n]), group)
        _, sv, zv = co.oracle_quantise(np64(c.v[0, h, :n]), group)
        zK, zV, sV = (np.repeat(x, group, axis=1) for x in (zk, zv, sv))
        x = np64(q[0, hq, 0])
        want, wl, w, _ = co.oracle_cache_attend_row(x, K, V, inv, n - 1, n, None, page, False, True, False, None)
        code = np.abs(K - zK)
        dz = 0.5 * np.abs(x).max() / 8355711 * code.sum(1) + 2.0 ** -20 * ((code + np.abs(zK)) @ np.abs(x))
        dz = dz / np.sqrt(D)
        z = K @ x / np.sqrt(D)
        rel = 2 * dz.max() + np.abs(z - z.max()).max() * 2.0 ** -23 + 2.0 ** -21 + n * 2.0 ** -23
        bound = n * 15 * 2.0 ** -23 * (w[:, None] * sV).max(0) + rel * (w @ (np.abs(V - zV) + np.abs(zV)))
        err = np.abs(np64(out[0, hq, 0]) - want)
        assert (err <= bound).all(), (hq, (err / bound).max())
        assert abs(float(lse[0, hq, 0]) - wl) <= rel + 2.0 ** -22 * abs(wl)
    assert _status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,group,page", FORMS)
@pytest.mark.parametrize("G", [1, 2, 4, 16])
def test_small_weights_beside_a_large_one(dtype, D, group, page, G):
    """Equal probabilities, one key with a scale 2^10 times the others' but codes of 0 in all but a dim.

    Logits are 0 and probabilities 1 exactly, so the weights are the scales.  n keys are off by n half steps of 2^-22
    of the largest scale, 1, times a code of 15; the rest is sums of n floats, n 2^-23 of their sizes.
    """
    n = 20
    g = torch.Generator().manual_seed(82)
    v = torch.rand(1, 2, n, D, generator=g) * 15 * 2.0 ** -10
    v[:, :, 7] = 0.0
    v[:, :, 7, ::group] = 15.0
    k = torch.randn(1, 2, n, D, generator=g)
    c = Cache(82, B=1, H=2, D=D, group=group, page=page, ctx=(n,), rows=(k.to(dtype), v.to(dtype)))
    q = torch.zeros(1, 2 * G, 1, D, dtype=dtype, device=DEV)
    out, lse = lsh.lsh_cache_attend(q, c.cache, c.table, c.ctx_len, self_mask=False, out_dtype=torch.float32, **c.form)
    for h in range(2):
        V = c.stored(0, h)[1]
        bound = 15 * 2.0 ** -23 + n * 2.0 ** -23 * np.abs(V).mean(0)
        err = np.abs(np64(out[0, h * G:(h + 1) * G, 0]) - V.mean(0))
        assert (err <= bound).all(), (err / bound).max()
    assert (lse.double() - np.log(n)).abs().max() <= 2.0 ** -22 * np.log(n)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,group,page", FORMS)
def test_key_lengths_of_any_size(dtype, D, group, page):
    """1 / max(||row||, 1e-12) of rows whose squares overflow or vanish in a float, between ordinary ones.

    Sum of D squares: D / 8 + 5 roundings of 2^-24, then a root, a quotient and (from 2^126 on) a denormal's.
    """
    sizes = [1.0, 1e18, 1e19, 3e19, 1e20, 1.0, 1e25, 1e31, 1e36, 3e37, 0.0, 1e-13, 1e-30, 1e19, 1.0, 1e-18, 2e20]
    g = torch.Generator().manual_seed(83)
    k = torch.randn(1, 2, len(sizes) + 6, D, generator=g).clamp(-4, 4)
    k[:, :, :len(sizes)] *= torch.tensor(sizes)[:, None]
    k[:, 0, -6:, 3] = torch.tensor([float("inf"), float("-inf"), float("nan"), 1e30, 2e38, 3.3e38])
    k = k.to(dtype)
    n = k.shape[2]
    c = Cache(83, B=1, H=2, D=D, group=group, page=page, ctx=(n,), rows=(k, k.flip(3).contiguous()))
    _, _, inv = lsh.lsh_cache_read(c.cache, c.table, c.ctx_len, n, D, **c.form)
    want = co.oracle_key_inv(np64(k))
    assert np.isnan(want).sum() == 1 and (want == 0).sum() == 2
    assert np.allclose(np64(inv), want, rtol=(D / 8 + 8) * 2.0 ** -24, atol=2.0 ** -149, equal_nan=True)
    assert _status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("G", [1, 2, 8])
@pytest.mark.parametrize("unit_keys", [True, False])
@pytest.mark.parametrize("size", [1e-35, 1e-25, 1e18, 1e20, 1e30, 1e33, 1e36])
def test_keys_of_any_size(dtype, G, unit_keys, size):
    """Keys near both ends of the range, plain ones with a scale that keeps their logits ordinary."""
    g = torch.Generator().manual_seed(84)
    k = (torch.randn(1, 2, 150, 64, generator=g).clamp(-4, 4) * 0.25 * size).to(dtype)
    v = torch.randn(1, 2, 150, 64, generator=g).to(dtype)
    c = Cache(84, dtype=dtype, B=1, H=2, D=64, group=32, page=32, ctx=(150,), rows=(k, v))
    q = torch.randn(1, 2 * G, 1, 64, generator=g).clamp(-4, 4).to(dtype).to(DEV)
    scale = 0.5 if unit_keys else min(0.5 / size, 1e37)
    out, lse = lsh.lsh_cache_attend(q, c.cache, c.table, c.ctx_len, unit_keys=unit_keys, scale=scale,
                                    out_dtype=torch.float32, **c.form)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    _check_attend(c, q, out, lse, [1], unit_keys=unit_keys, scale=scale)
    assert _status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("size", [1.0, 1e-20, 1e-26, 1e-28, 1e-29, 4e-30])
def test_values_of_any_smallness(dtype, size):
    """Values down to the smallest scale (2^-100), one dominant key and many whose weights are small, in stages that
    hold masked keys too.

    As in test_weights_keep_the_precision_of_floats, with steps that end at 2^-127: n keys are then off by
    n * 15 * 2^-128.
    """
    n, T, D, group = 650, 8, 64, 32
    g = torch.Generator().manual_seed(85)
    k = torch.zeros(1, 1, n, D)
    k[..., 0] = 1.0
    k[:, :, 5, 0] = 40.0
    k[:, :, 6:, 1] = torch.rand(1, 1, n - 6, generator=g) * 6
    v = torch.randn(1, 1, n, D, generator=g) * size
    c = Cache(85, B=1, H=1, D=D, group=group, page=64, ctx=(n,), rows=(k, v))
    q = torch.zeros(1, 1, T, D, dtype=dtype)
    q[..., 0], q[..., 1] = 1.5, -1.0
    out, lse = lsh.lsh_cache_attend(q.to(DEV), c.cache, c.table, c.ctx_len, unit_keys=False, out_dtype=torch.float32,
                                    **c.form)
    K, V, inv = c.stored(0, 0)
    _, _, zk = co.oracle_quantise(np64(k[0, 0]), group)
    _, sv, zv = co.oracle_quantise(np64(v[0, 0]), group)
    zK, zV, sV = (np.repeat(x, group, axis=1) for x in (zk, zv, sv))
    for t in range(T):
        x, pos = np64(q[0, 0, t]), n - T + t
        want, wl, w, keys = co.oracle_cache_attend_row(x, K, V, inv, pos, n, None, 64, True, True, False, None)
        code = np.abs(K - zK)
        dz = (0.5 * np.abs(x).max() / 8355711 * code.sum(1) + 2.0 ** -20 * ((code + np.abs(zK)) @ np.abs(x))) / 8
        rel = 2 * dz.max() + 2.0 ** -18
        bound = n * 15 * (2.0 ** -23 * (w[:, None] * sV[keys]).max(0) + 2.0 ** -128)
        bound = bound + rel * (w @ (np.abs(V - zV) + np.abs(zV))[keys])
        err = np.abs(np64(out[0, 0, t]) - want)
        assert (err <= bound).all(), (t, (err / bound).max(), err.max() / size)
        assert abs(float(lse[0, 0, t]) - wl) <= rel + 2.0 ** -22 * abs(wl)
    assert _status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [300, 5000])
def test_values_of_any_size(dtype, n):
    """Values of one sign whose sum over the keys is 1e35, with equal weights and with the largest logit last."""
    g = torch.Generator().manual_seed(86)
    v = (1 + torch.rand(1, 1, n, 64, generator=g)) * (0.5e35 / n)
    k = torch.zeros(1, 1, n, 64)
    k[..., 0] = torch.linspace(0.0, 5.0, n)
    c = Cache(86, dtype=torch.float32, B=1, H=1, D=64, group=64, page=64, ctx=(n,), rows=(k, v))
    for q0 in (0.0, 8.0):
        q = torch.zeros(1, 1, 1, 64, dtype=dtype, device=DEV)
        q[..., 0] = q0
        out, lse = lsh.lsh_cache_attend(q, c.cache, c.table, c.ctx_len, unit_keys=False, self_mask=False,
                                        out_dtype=torch.float32, **c.form)
        assert torch.isfinite(out).all()
        _check_attend(c, q, out, lse, [1], unit_keys=False, self_mask=False)
    assert _status() == 0


def _rational_stored(x):
    """Stored values of one group in rational arithmetic (finite, no denormals)."""
    x = [Fraction(float(t)) for t in x]

    def bf16(f, nearest):  # the largest bf16 not above f, or the nearest (ties to even)
        if f == 0:
            return f
        a, e = abs(f), 0
        while a >= 2:
            a, e = a / 2, e + 1
        while a < 1:
            a, e = a * 2, e - 1
        step = Fraction(2) ** (e - 7)
        n = f / step
        low = n.numerator // n.denominator
        r = n - low
        return step * (low + (nearest and (r > Fraction(1, 2) or (r == Fraction(1, 2) and low % 2 == 1))))

    z = bf16(min(x), False)
    s = bf16((max(x) - z) / 15, True)
    if s < Fraction(2) ** -100:
        return [float(z)] * len(x)
    out = []
    for t in x:
        q = (t - z) / s
        low = q.numerator // q.denominator
        r = q - low
        c = min(15, low + (r > Fraction(1, 2) or (r == Fraction(1, 2) and low % 2 == 1)))
        out.append(z + s * c)
    return out


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantiser_next_to_every_border(dtype):
    """Scales and codes whose quotient lies on a border or as near to it as the type allows, with zeros so small
    that neither a float's nor a double's difference shows them; against rational arithmetic."""
    g = np.random.default_rng(87)
    rows = []
    for i in range(400):
        m = int(g.integers(128, 256))
        e = float(2.0 ** g.integers(-20, 20))
        z = [0.0, -2.0 ** -80, 2.0 ** -80, -3 * 2.0 ** -60, 2.0 ** -40, -1.0, 1.0, -200.0][i % 8]
        s = m * e
        top = 15 * (s + [0, 0.5 * e, e * 2.0 ** -7, -0.5 * e][(i // 8) % 4])  # on, half a step beside, near
        x = z + (g.integers(0, 15, 32) + 0.5) * s
        x = x.astype(np.float32)
        for step in (-1.0, 1.0):
            part = g.random(32) < 0.25
            x[part] = np.nextafter(x[part], np.float32(step * 3e38))
        x[0], x[1] = z, top if z else 3855.0 * e
        rows.append(x)
    x = torch.from_numpy(np.stack(rows).reshape(200, 64)).to(dtype)
    n = x.shape[0]
    c = Cache(87, dtype=dtype, B=1, H=1, D=64, group=32, page=16, ctx=(n,),
              rows=(x[None, None], x.flip(1)[None, None].contiguous()))
    k, v, _ = lsh.lsh_cache_read(c.cache, c.table, c.ctx_len, n, 64, out_dtype=torch.float32, **c.form)
    for got, src in ((k, x), (v, x.flip(1))):
        for r in range(n):
            want = []
            for a in (0, 32):
                want += _rational_stored(src[r, a:a + 32].double().tolist())
            # one rounding of the rational value to float32 (float() of a Fraction is the nearest double; where that is
            # halfway between two floats, it is the value itself)
            assert got[0, 0, r].tolist() == [float(np.float32(float(t))) for t in want], r


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("q_size,k_size", [(1e-29, 1e29), (1e-20, 1e30), (1e30, 1e-20), (1e35, 1.0)])
@pytest.mark.parametrize("unit_keys", [True, False])
def test_queries_of_any_size(dtype, q_size, k_size, unit_keys):
    """Queries near both ends of their range, with a scale that keeps the logits ordinary."""
    g = torch.Generator().manual_seed(88)
    k = (torch.randn(1, 2, 150, 64, generator=g).clamp(-4, 4) * k_size).to(dtype)
    v = torch.randn(1, 2, 150, 64, generator=g).to(dtype)
    c = Cache(88, dtype=dtype, B=1, H=2, D=64, group=32, page=32, ctx=(150,), rows=(k, v))
    q = (torch.randn(1, 2, 1, 64, generator=g).clamp(-4, 4) * q_size).to(dtype)
    q[..., 0] = q_size
    scale = 0.25 / q_size if unit_keys else 0.25 / (q_size * k_size)
    out, lse = lsh.lsh_cache_attend(q.to(DEV), c.cache, c.table, c.ctx_len, unit_keys=unit_keys, scale=scale,
                                    out_dtype=torch.float32, **c.form)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    _check_attend(c, q, out, lse, [1], unit_keys=unit_keys, scale=scale)
    assert _status() == 0
