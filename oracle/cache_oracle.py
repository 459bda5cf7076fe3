"""Float64 CPU oracle of the decoding operators: 4-bit storage of rows, attention over stored rows, and the
choice of pages by shared buckets.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).  Follows the definitions, not the packing: a
sequence is an array of stored rows by position, and pages are ranges of positions.
"""

import numpy as np


def floor_bf16(x):
    """The largest bf16 not above x (float64 array of float32 values)."""
    x = np.asarray(x, dtype=np.float64)
    out = np.zeros_like(x)
    nz = x != 0
    m, e = np.frexp(x[nz])  # x = m 2^e, 1/2 <= |m| < 1: eight bits of m stay
    step = np.ldexp(1.0, np.maximum(e - 8, -133))  # bf16 denormals end at 2^-133
    out[nz] = np.floor(x[nz] / step) * step
    return out


def round_bf16(x):
    """The nearest bf16, ties to even (finite float64 in the normal range or zero)."""
    x = np.asarray(x, dtype=np.float64)
    m, e = np.frexp(x)
    step = np.ldexp(1.0, np.maximum(e - 8, -133))
    return np.rint(x / step) * step


def oracle_quantise(x, group):
    """Codes, scale, zero of rows x [..., D]: codes [..., D] float64, s and z [..., D/group].

    A group with a non-finite value or a range that overflows float32 has scale NaN and codes 0.
    """
    x = np.asarray(x, dtype=np.float64)
    g = x.reshape(*x.shape[:-1], x.shape[-1] // group, group)
    ok = np.isfinite(g).all(-1)
    safe = np.where(ok[..., None], g, 0.0)
    lo, hi = safe.min(-1), safe.max(-1)
    z = floor_bf16(lo)
    big = np.float64(3.3895313892515355e38)  # the largest bf16
    ok &= (z >= -big) & (hi - z < 3.4028235677973366e38)  # rounds to a finite float32
    s = round_bf16(np.where(ok, hi - z, 0.0) / 15.0)
    s = np.where(s < 2.0 ** -100, 0.0, s)
    div = np.where(s > 0, s, 1.0)[..., None]
    c = np.where((s > 0)[..., None], np.clip(np.rint((safe - z[..., None]) / div), 0, 15), 0.0)
    s = np.where(ok, s, np.nan)
    return c.reshape(x.shape), s, z


def oracle_stored(x, group):
    """The stored values of rows x [..., D] in float64 (z + s c)."""
    c, s, z = oracle_quantise(x, group)
    cg = c.reshape(*s.shape, group)
    return (z[..., None] + s[..., None] * cg).reshape(c.shape)


def oracle_key_inv(x):
    x = np.asarray(x, dtype=np.float64)
    return 1.0 / np.maximum(np.sqrt((x * x).sum(-1)), 1e-12)


def oracle_cache_attend_row(q, K, V, key_inv, pos, ctx, pages, page, self_mask, causal, unit_keys, scale):
    """One query row at position pos over stored rows K, V [ctx, D].

    ``pages`` lists the logical pages it attends to (a page twice counts twice), None for all.
    Returns (out [D], lse, weights [n], positions [n]).
    """
    if pages is None:
        keys = np.arange(ctx)
    else:
        keys = [np.arange(p * page, min((p + 1) * page, ctx)) for p in pages if p >= 0 and p * page < ctx]
        keys = np.concatenate(keys) if keys else np.zeros(0, dtype=np.int64)
    if causal:
        keys = keys[keys <= pos]
    if self_mask and (keys != pos).any():
        keys = keys[keys != pos]
    D = K.shape[1]
    if pos < 0 or keys.size == 0:
        return np.zeros(D), -np.inf, np.zeros(0), keys
    z = (K[keys] @ np.asarray(q, dtype=np.float64)) * (scale if scale else 1.0 / np.sqrt(D))
    if unit_keys:
        z = z * key_inv[keys]
    m = z.max()
    p = np.exp(z - m)
    return p @ V[keys] / p.sum(), float(m + np.log(p.sum())), p / p.sum(), keys


def oracle_cache_select(tags, q_buckets, pos, ctx, page, max_pages, n_select, n_local, causal):
    """One query row: tags [n_rounds, ctx], q_buckets [G, n_rounds].  Returns (selected, scores) lists."""
    limit = 0 if pos < 0 else (pos + 1 if causal else ctx)
    n = -(-limit // page)
    scores = [-1] * max_pages
    for p in range(n):
        part = tags[:, p * page:min((p + 1) * page, limit)]
        scores[p] = int(sum((part == qb[:, None]).sum() for qb in q_buckets))
    order = sorted(range(n), key=lambda p: (p < n - n_local, -scores[p], p))
    chosen = sorted(order[:n_select])
    return chosen + [-1] * (n_select - len(chosen)), scores
