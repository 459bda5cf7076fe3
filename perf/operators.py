"""What is measured of the decoding operators: the 4-bit cache's write and read-back, attention over it, and
attention over the pages that shared hash buckets select.

``run`` computes a case in plain torch operations, or, with ``own`` set, by the package's entry points.  Both
take the same state, the packed cache included: the plain form packs and unpacks the cache's bytes itself.

The cache, as both sides hold it (uint8 [n_pages, H, page / 16 tiles]): a tile holds 16 tokens of one head,

    K codes    16 rows of D/2 bytes: byte t*(D/8) + 4*w + b holds dims 32w + 8b + 2t (low nibble) and the next one
    V codes    8 token pairs of D bytes: chunk g ^ (2*(pair & 3)) of D/8 bytes holds, for word q and token e of the
               pair, nibbles i = 0..7 = dims 64q + 8i + g
    K params   [D/group][16] words: scale (bf16, low half) and zero (bf16, high half)
    V params   the same
    K lengths  16 floats: 1 / max(||row||, 1e-12)

and a stored value is zero + scale * code.
"""

import math

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------------------------------
# Cases

def _case(kind, name=None, **kw):
    c = {"kind": kind, "dtype": "bf16", "B": 1, "H": 8, "G": 1, "T": 1, "L": 1024, "D": 128, "group": 64,
         "page": 64, "ragged": False, "self_mask": True, "causal": True, "unit_keys": True,
         "rounds": 0, "buckets": 0, "n_select": 0, "n_local": 0}
    c.update(kw)
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # one decoding step of a batch: every sequence's new row goes into its cache; latency only
        _case("append", "append_step", B=8, T=1, L=4001),
        # ragged prompts of a batch on their way into the cache, padded to the longest
        _case("append", "append_prompts", B=4, T=4099, L=6000, ragged=True),
        # a long document's rows in fp32 (head dim of the million-token workload), small pages
        _case("append", "append_document_fp32", B=1, T=262144, L=262144, D=64, page=32, dtype="fp32"),
        # generation from a short context, one sequence: latency only
        _case("attend", "attend_short", B=1, L=1021),
        # a serving batch of contexts of different lengths
        _case("attend", "attend_batch", B=8, L=16384, ragged=True),
        # the 64K workload's shape at decoding time: one new token of each of 8 sequences
        _case("attend", "attend_64k", B=8, L=65536),
        # the million-token workload's shape at decoding time
        _case("attend", "attend_1m", B=1, L=1048576, D=64, page=128),
        # fp32 rows, fine groups, an odd length
        _case("attend", "attend_fp32", B=2, H=4, L=5003, D=64, group=32, dtype="fp32", page=16),
        # several new tokens of each sequence at once, query heads that share cached heads, plain keys
        _case("attend", "attend_heads_shared", B=4, H=8, G=4, T=4, L=8190, self_mask=False, unit_keys=False),
        # hash-selected pages at a short context: latency only
        _case("sparse", "sparse_short", B=1, L=4093, rounds=4, buckets=64, n_select=16, n_local=1),
        # hash-selected pages at the 64K workload's shape: 64 of 1024 pages
        _case("sparse", "sparse_64k", B=8, L=65536, rounds=8, buckets=1024, n_select=64, n_local=2),
        # hash-selected pages at the million-token shape: 256 of 16384 pages
        _case("sparse", "sparse_1m", B=1, L=1048576, D=64, rounds=4, buckets=16384, n_select=256, n_local=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["append", "attend", "attend", "sparse"])
    D = rng.choice([64, 128, 128, 256])
    group = rng.choice([32, 64])
    page = rng.choice([16, 32, 64, 64, 128])
    B = _log(rng, 1, 12)
    H = _log(rng, 1, 10)
    ragged = rng.random() < 0.5
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    most = 1 << 21  # cached tokens times heads of a drawn case, at most half of the largest listed
    if kind == "append":
        T = _log(rng, 1, max(2, most // (B * H) // (D // 64)))
        return _case(kind, dtype=dtype, B=B, H=H, T=T, L=T + rng.randrange(0, 700), D=D, group=group, page=page,
                     ragged=ragged, rounds=rng.choice([0, 0, 4]), buckets=256)
    L = _log(rng, 1, max(2, most // (B * H) // (D // 64)))
    G = rng.choice([1, 1, 2, 4, 7])
    T = min(L, rng.choice([1, 1, 1, 2, 5]))
    c = _case(kind, dtype=dtype, B=B, H=H, G=G, T=T, L=L, D=D, group=group, page=page, ragged=ragged,
              self_mask=rng.random() < 0.6, causal=rng.random() < 0.8, unit_keys=rng.random() < 0.6)
    if kind == "sparse":
        n_select = _log(rng, 1, min(128, 2 * -(-L // page)))
        c.update(rounds=rng.choice([1, 2, 4, 8]), buckets=rng.choice([16, 64, 1024, 65536]), n_select=n_select,
                 n_local=rng.randrange(0, min(n_select, 4) + 1))
    return c


def _sizes(c):
    ng = c["D"] // c["group"]
    tile = 16 * c["D"] + 128 * ng + 64
    max_pages = -(-c["L"] // c["page"])
    return ng, tile, max_pages, tile * (c["page"] // 16)


def _lengths(c, seed):
    """Context length and new rows of every sequence (host lists, from the case and the seed)."""
    g = torch.Generator().manual_seed(seed * 7919 + 17)
    ctx, new = [], []
    for b in range(c["B"]):
        if c["ragged"]:
            n = int(torch.randint(0, c["T"] + 1, (1,), generator=g)) if b else c["T"]
            x = int(torch.randint(0, c["L"] + 1, (1,), generator=g)) if b else c["L"]
            ctx.append(max(n, x))
            new.append(n)
        else:
            ctx.append(c["L"])
            new.append(c["T"])
    return ctx, new


def work(case):
    """Bytes and operations that the case cannot do without, at the mean length of ragged batches."""
    c = case
    ng = c["D"] // c["group"]
    row = c["D"] + 8 * ng + 4  # stored bytes of a token and head, keys and values
    es = 4 if c["dtype"] == "fp32" else 2
    half = 0.5 if c["ragged"] else 1.0
    seqs = c["B"] if not c["ragged"] else 1 + (c["B"] - 1) * half
    if c["kind"] == "append":
        n = seqs * c["T"] * c["H"]
        # rows read and stored, read back and returned
        return {"bytes": n * (2 * c["D"] * es + row + row + 2 * c["D"] * es + 4), "flops": n * c["D"] * 10}
    qrows = c["B"] * c["H"] * c["G"] * c["T"]
    io = qrows * (2 * c["D"] * es + 4)
    if c["kind"] == "attend":
        n = seqs * c["L"] * c["H"]
        return {"bytes": n * row + io, "flops": n * c["G"] * c["T"] * 4 * c["D"]}
    tags = seqs * c["L"] * c["H"] * c["rounds"] * 2
    kept = min(c["L"], c["n_select"] * c["page"]) * c["H"] * (seqs if c["ragged"] else c["B"])
    max_pages = -(-c["L"] // c["page"])
    ints = c["B"] * c["H"] * c["T"] * (c["n_select"] + max_pages) * 4
    return {"bytes": tags + kept * c["T"] * row + io + ints, "flops": kept * c["T"] * c["G"] * 4 * c["D"]}


# ---------------------------------------------------------------------------------------------------
# The plain form

def _floor_bf16(x):
    """The largest bf16 that is not above x (float32 in, float32 out)."""
    y = x.to(torch.bfloat16).float()
    bits = y.view(torch.int32)
    # one bf16 step towards minus infinity where rounding went up
    down = torch.where(y > 0, bits - 0x10000, torch.where(y < 0, bits + 0x10000, torch.full_like(bits, -0x7FFF0000)))
    return torch.where(y > x, down.view(torch.float32), y)


def _quantise(x, group):
    """Codes (uint8), scale and zero (float32 holding bf16) of rows [..., D]; the quotients in 64 bits."""
    xg = x.reshape(*x.shape[:-1], x.shape[-1] // group, group).float()
    z = _floor_bf16(xg.amin(-1))
    span = xg.amax(-1).double() - z.double()
    s = _nearest_bf16(span / torch.full_like(span, 15))  # by a tensor: by a number torch multiplies with 1/15
    s = torch.where(s < 2.0 ** -100, torch.zeros_like(s), s)
    good = torch.isfinite(span.float()) & torch.isfinite(xg).all(-1)
    s = torch.where(good, s, torch.full_like(s, float("nan")))
    q = (xg.double() - z.double()[..., None]) / s.double()[..., None]
    codes = torch.where((s > 0)[..., None], torch.clamp(torch.round(q), 0, 15), torch.zeros_like(q))
    return codes.to(torch.uint8).reshape(x.shape), s, z


def _nearest_bf16(q):
    """Nearest bf16 of float64 values, ties to even, without the double rounding of a step through float32."""
    f = q.float()
    low = f.view(torch.int32) & 0xFFFF
    # a float32 on the midpoint of two bf16: which side it came from decides
    nudge = torch.where(low == 0x8000, torch.sign(q - f.double()).to(torch.int32), torch.zeros_like(low))
    return (f.view(torch.int32) + nudge).view(torch.float32).to(torch.bfloat16).float()


def _words(s, z):
    """Scale and zero words [..., 2 bytes + 2 bytes] from bf16 values held in float32."""
    return torch.stack([s.to(torch.bfloat16), z.to(torch.bfloat16)], -1).contiguous().view(torch.uint8)


def _token_bytes(c, k, v):
    """The bytes that each token of rows [..., D] puts into its tile, in the order of _token_offsets."""
    D, group = c["D"], c["group"]
    kc, ks, kz = _quantise(k, group)
    vc, vs, vz = _quantise(v, group)
    lead = k.shape[:-1]
    kn = kc.reshape(*lead, D // 32, 4, 4, 2)  # w, b, t, nibble
    kb = (kn[..., 0] | (kn[..., 1] << 4)).movedim(-1, -3).reshape(*lead, D // 2)
    vn = vc.reshape(*lead, D // 64, 4, 2, 8)  # q, i / 2, nibble, g
    vb = (vn[..., 0, :] | (vn[..., 1, :] << 4)).movedim(-1, -3).reshape(*lead, D // 2)  # g, q, i / 2
    inv = 1.0 / k.float().square().sum(-1, keepdim=True).sqrt().clamp_min(1e-12)
    return torch.cat([kb, vb, _words(ks, kz).reshape(*lead, -1), _words(vs, vz).reshape(*lead, -1),
                      inv.contiguous().view(torch.uint8)], -1)


def _token_offsets(c):
    """[16, bytes of a token]: where in a tile the bytes of its token r lie, in the order of _token_bytes."""
    D = c["D"]
    ng = D // c["group"]
    r = torch.arange(16, device=DEV)[:, None]
    koff = r * (D // 2) + torch.arange(D // 2, device=DEV)
    g, q, b = (t.reshape(1, -1) for t in torch.meshgrid(torch.arange(8, device=DEV), torch.arange(D // 64, device=DEV),
                                                        torch.arange(4, device=DEV), indexing="ij"))
    pair, e = r // 2, r % 2
    voff = 8 * D + pair * D + (g ^ (2 * (pair & 3))) * (D // 8) + q * 8 + e * 4 + b
    par = (torch.arange(ng, device=DEV)[:, None] * 64 + torch.arange(4, device=DEV)).reshape(1, -1) + 4 * r
    ioff = 16 * D + 128 * ng + 4 * r + torch.arange(4, device=DEV)
    return torch.cat([koff, voff, 16 * D + par, 16 * D + 64 * ng + par, ioff], 1)


def _positions(s):
    """Position of each of the T rows, or -1: [B, T]."""
    i = torch.arange(s["T"], device=DEV)
    start = s["ctx_len"] - s["new_len"]
    return torch.where(i[None] < s["new_len"][:, None], start[:, None] + i[None], -1)


def _store(s, k, v):
    """Puts rows [B, H, T, D] into the cache (and their buckets into the tags); returns where their bytes lie."""
    c = s["case"]
    ng, tile, max_pages, block = _sizes(c)
    pos = _positions(s).long()
    ok = pos >= 0
    at = pos.clamp_min(0)
    page = s["page_table"].long().gather(1, at // c["page"])
    page = torch.where(ok, page, s["cache"].shape[0] - 1)  # padding goes to the spare page
    h = torch.arange(c["H"], device=DEV)
    base = (page[:, None, :] * c["H"] + h[None, :, None]) * block + ((at % c["page"]) // 16 * tile)[:, None, :]
    index = base[..., None] + _token_offsets(c)[at % 16][:, None]
    s["cache"].view(-1)[index.reshape(-1)] = _token_bytes(c, k, v).reshape(-1)
    if c["rounds"]:
        n_rounds = c["rounds"]
        r = torch.arange(n_rounds, device=DEV)
        row = ((page[:, None, None, :] * c["H"] + h[None, :, None, None]) * n_rounds + r[None, None, :, None])
        idx = row * c["page"] + (at % c["page"])[:, None, None, :]
        s["tags"].view(-1)[idx.reshape(-1)] = s["new_buckets"].to(torch.int16).reshape(-1)
    return index


def _decode(c, blocks):
    """Stored K, V [..., page, D] and key lengths [..., page] in float32 of blocks [..., block bytes]."""
    D, group = c["D"], c["group"]
    ng, tile, _, _ = _sizes(c)
    lead = blocks.shape[:-1]
    t = blocks.reshape(*lead, c["page"] // 16, tile)
    kb = t[..., :8 * D].reshape(*t.shape[:-1], 16, 4, D // 32, 4)  # t, w, b
    kb = torch.stack([kb & 15, kb >> 4], -1).movedim(-4, -2)  # w, b, t, nibble
    kc = kb.reshape(*t.shape[:-1], 16, D)
    vb = t[..., 8 * D:16 * D].reshape(*t.shape[:-1], 8, 8, D // 64, 2, 4)  # pair, chunk, q, e, i / 2
    pair = torch.arange(8, device=DEV)[:, None]
    chunk = torch.arange(8, device=DEV)[None] ^ (2 * (pair & 3))
    vb = vb[..., pair, chunk, :, :, :]  # pair, g, q, e, i / 2
    vb = torch.stack([vb & 15, vb >> 4], -1).flatten(-2)  # pair, g, q, e, i
    vc = vb.movedim(-2, -4).movedim(-3, -1).reshape(*t.shape[:-1], 16, D)  # pair, e, q, i, g
    par = t[..., 16 * D:16 * D + 128 * ng].contiguous().view(torch.bfloat16).reshape(*t.shape[:-1], 2, ng, 16, 2)
    par = par.float().transpose(-3, -2)  # which, token, group, (scale, zero)
    inv = t[..., 16 * D + 128 * ng:].contiguous().view(torch.float32)

    def values(codes, p):
        x = codes.reshape(*t.shape[:-1], 16, ng, group).float()
        return (x * p[..., :1] + p[..., 1:]).reshape(*lead, c["page"], D)

    return values(kc, par[..., 0, :, :, :]), values(vc, par[..., 1, :, :, :]), inv.reshape(*lead, c["page"])


def _dtype(c):
    return torch.float32 if c["dtype"] == "fp32" else torch.bfloat16


def _plain_append(s):
    c = s["case"]
    index = _store(s, s["k"], s["v"])
    # back from the cache: the rows that were written
    raw = s["cache"].view(-1)[index]  # [B, H, T, bytes]
    live = (_positions(s) >= 0)[:, None, :, None]
    ng = _sizes(c)[0]
    D, group = c["D"], c["group"]
    lead = raw.shape[:-1]
    kb, vb = raw[..., :D // 2], raw[..., D // 2:D]
    kb = kb.reshape(*lead, 4, D // 32, 4)
    kc = torch.stack([kb & 15, kb >> 4], -1).movedim(-4, -2).reshape(*lead, ng, group)
    vb = vb.reshape(*lead, 8, D // 64, 4)
    vc = torch.stack([vb & 15, vb >> 4], -1).flatten(-2).movedim(-3, -1).reshape(*lead, ng, group)
    par = raw[..., D:D + 8 * ng].contiguous().view(torch.bfloat16).float().reshape(*lead, 2, ng, 2)
    inv = raw[..., D + 8 * ng:].contiguous().view(torch.float32)[..., 0]
    k = (kc * par[..., 0, :, :1] + par[..., 0, :, 1:]).reshape(*lead, D)
    v = (vc * par[..., 1, :, :1] + par[..., 1, :, 1:]).reshape(*lead, D)
    k = torch.where(live, k, 0.0).to(_dtype(c))
    v = torch.where(live, v, 0.0).to(_dtype(c))
    got = {"k": k, "v": v, "key_inv": torch.where(live[..., 0], inv, 0.0)}
    return {**got, "tags": s["tags"][:-1]} if c["rounds"] else got


def _softmax_attend(c, q, K, V, inv, admissible):
    """q [N, C, D], K, V [N, S, D], inv [N, S], admissible [N, C, S] (bool) -> out [N, C, D], lse [N, C]."""
    logit = torch.matmul(q.float(), K.transpose(-1, -2)) / math.sqrt(c["D"])
    if c["unit_keys"]:
        logit = logit * inv[:, None, :]
    logit = torch.where(admissible, logit, -math.inf)
    m = logit.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.where(admissible, torch.exp(logit - m), 0.0)
    l = p.sum(-1, keepdim=True)
    out = torch.matmul(p, V) / torch.where(l == 0, 1.0, l)
    return out, (m + torch.log(l))[..., 0]


def _admissible(c, keys, pos, ctx):
    """keys [..., 1, S] (position or -1), pos [..., C, 1], ctx [..., 1, 1] -> bool [..., C, S]."""
    a = (keys >= 0) & (keys < ctx) & (pos >= 0)
    if c["causal"]:
        a = a & (keys <= pos)
    if c["self_mask"]:
        other = a & (keys != pos)
        a = torch.where(other.any(-1, keepdim=True), other, a)
    return a


def _plain_attend(s):
    c = s["case"]
    B, H, G, T, D = c["B"], c["H"], c["G"], c["T"], c["D"]
    K, V, inv = _decode(c, s["cache"][s["page_table"].long()].transpose(1, 2))  # [B, H, pages, page, D]
    S = K.shape[2] * K.shape[3]
    K, V, inv = K.reshape(B * H, S, D), V.reshape(B * H, S, D), inv.reshape(B * H, S)
    keys = torch.arange(S, device=DEV)
    live = keys < s["ctx_len"][:, None, None]  # [B, 1, S]; what lies behind a sequence is not looked at
    live = live.expand(B, H, S).reshape(B * H, S)
    K = torch.where(live[..., None], K, 0.0)
    V = torch.where(live[..., None], V, 0.0)
    pos = _positions(s)[:, None, None, :].expand(B, H, G, T).reshape(B * H, G * T, 1)
    ctx = s["ctx_len"][:, None].expand(B, H).reshape(B * H, 1, 1)
    a = _admissible(c, keys[None, None], pos, ctx)
    out, lse = _softmax_attend(c, s["q"].reshape(B * H, G * T, D), K, V, torch.where(live, inv, 0.0), a)
    return {"out": out.reshape(B, H * G, T, D).to(_dtype(c)), "lse": lse.reshape(B, H * G, T)}


def _plain_sparse(s):
    c = s["case"]
    B, H, G, T, D, page = c["B"], c["H"], c["G"], c["T"], c["D"], c["page"]
    n_rounds, n_select = c["rounds"], c["n_select"]
    max_pages = s["page_table"].shape[1]
    pos = _positions(s)  # [B, T]
    limit = (pos + 1) if c["causal"] else torch.where(pos >= 0, s["ctx_len"][:, None], 0)
    # score of every page: shared buckets of the query heads with the admissible positions
    tags = s["tags"][s["page_table"].long()].to(torch.int32) & 0xFFFF  # [B, pages, H, rounds, page]
    tags = tags.permute(0, 2, 1, 3, 4)  # [B, H, pages, rounds, page]
    qb = s["q_buckets"].reshape(B, H, G, n_rounds, T)
    where = torch.arange(max_pages * page, device=DEV).reshape(max_pages, page)
    inside = where[None, None] < limit[:, :, None, None]  # [B, T, pages, page]
    score = torch.zeros(B, H, T, max_pages, dtype=torch.int64, device=DEV)
    for g in range(G):
        for r in range(n_rounds):
            same = tags[:, :, None, :, r] == qb[:, :, g, r, :, None, None]  # [B, H, T, pages, page]
            score += (same & inside[:, None]).sum(-1)
    n_pages = -(-limit // page)  # [B, T]
    idx = torch.arange(max_pages, device=DEV)
    candidate = (idx < n_pages[..., None])[:, None].expand(B, H, T, max_pages)
    scores = torch.where(candidate, score, -1).to(torch.int32)
    local = (idx >= n_pages[..., None] - c["n_local"])[:, None]
    rank = torch.where(candidate, score + torch.where(local, 1 << 24, 0), -1)
    rank = rank * max_pages + (max_pages - 1 - idx)  # ties to the lowest index
    kept = min(n_select, max_pages)
    best = rank.topk(kept, -1).indices
    taken = torch.gather(candidate, -1, best)
    best = torch.where(taken, best, max_pages).sort(-1).values
    best = torch.where(best == max_pages, -1, best)
    selected = torch.full((B, H, T, n_select), -1, dtype=torch.int32, device=DEV)
    selected[..., :kept] = best.to(torch.int32)
    # attention over those pages
    N = B * H * T
    logical = selected.long().clamp_min(0)
    phys = s["page_table"].long()[:, None, None].expand(B, H, T, max_pages).gather(-1, logical)
    heads = torch.arange(H, device=DEV)[None, :, None, None]
    K, V, inv = _decode(c, s["cache"][phys, heads])  # [B, H, T, n_select, page, D]
    S = n_select * page
    keys = logical[..., None] * page + torch.arange(page, device=DEV)
    keys = torch.where(selected[..., None] >= 0, keys, -1).reshape(N, S)
    ctx = s["ctx_len"][:, None, None].expand(B, H, T).reshape(N, 1)
    keys = torch.where(keys < ctx, keys, -1)
    live = keys >= 0
    K = torch.where(live[..., None], K.reshape(N, S, D), 0.0)
    V = torch.where(live[..., None], V.reshape(N, S, D), 0.0)
    q = s["q"].reshape(B, H, G, T, D).transpose(2, 3).reshape(N, G, D)
    p = pos[:, None].expand(B, H, T).reshape(N, 1, 1)
    a = _admissible(c, keys[:, None], p, ctx[..., None])
    out, lse = _softmax_attend(c, q, K, V, torch.where(live, inv.reshape(N, S), 0.0), a)
    out = out.reshape(B, H, T, G, D).transpose(2, 3).reshape(B, H * G, T, D)
    lse = lse.reshape(B, H, T, G).transpose(2, 3).reshape(B, H * G, T)
    return {"selected": selected, "scores": scores, "out": out.to(_dtype(c)), "lse": lse}


# ---------------------------------------------------------------------------------------------------
# State and pass

def prepare(case, seed):
    c = dict(case)
    B, H, G, T, L, D = (c[k] for k in ("B", "H", "G", "T", "L", "D"))
    ng, tile, max_pages, block = _sizes(c)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dt = _dtype(c)
    ctx, new = _lengths(c, seed)
    n_pages = B * max_pages + 1  # one spare
    s = {"case": c, "T": T,
         "ctx_len": torch.tensor(ctx, dtype=torch.int32, device=DEV),
         "new_len": torch.tensor(new, dtype=torch.int32, device=DEV),
         # pages come from one pool in any order
         "page_table": torch.randperm(n_pages - 1, generator=gen, device=DEV).to(torch.int32).reshape(B, max_pages),
         "cache": torch.zeros(n_pages, H, block, dtype=torch.uint8, device=DEV)}
    n_rounds = c["rounds"]
    if n_rounds:
        s["tags"] = torch.zeros(n_pages, H, n_rounds, c["page"], dtype=torch.int16, device=DEV)
    # rows as projections give them: channels of different size, some offset
    size = torch.exp(0.4 * torch.randn(2, H, 1, D, generator=gen, device=DEV))
    mean = 0.3 * torch.randn(2, H, 1, D, generator=gen, device=DEV)

    def rows(n, which, b):
        return (torch.randn(b, H, n, D, generator=gen, device=DEV) * size[which] + mean[which]).to(dt)

    if c["kind"] == "append":
        s["k"], s["v"] = rows(T, 0, B), rows(T, 1, B)
        if n_rounds:
            s["new_buckets"] = torch.randint(0, c["buckets"], (B, H, n_rounds, T), generator=gen, device=DEV,
                                             dtype=torch.int32)
        return s
    s["q"] = torch.cat([rows(T, 0, B) for _ in range(G)], 2).reshape(B, H, G, T, D).reshape(B, H * G, T, D)
    if c["kind"] == "sparse":
        # buckets of independent rows are uniform; one cached token in 32 is a near neighbour of the query and
        # shares each of its buckets with probability 1/2
        s["q_buckets"] = torch.randint(0, c["buckets"], (B, H * G, n_rounds, T), generator=gen, device=DEV,
                                       dtype=torch.int32)
    # the contexts, in pieces of at most 32768 tokens, stored as a prompt is
    for b in range(B):
        for a in range(0, ctx[b], 32768):
            n = min(32768, ctx[b] - a)
            part = {"case": c, "T": n, "cache": s["cache"], "page_table": s["page_table"][b:b + 1],
                    "ctx_len": torch.tensor([a + n], device=DEV), "new_len": torch.tensor([n], device=DEV)}
            if n_rounds:
                part["tags"] = s["tags"]
                bk = torch.randint(0, c["buckets"], (1, H, n_rounds, n), generator=gen, device=DEV, dtype=torch.int32)
                near = torch.rand(1, H, 1, n, generator=gen, device=DEV) < 1 / 32
                near = near & (torch.rand(1, H, n_rounds, n, generator=gen, device=DEV) < 0.5)
                mine = s["q_buckets"].reshape(B, H, G, n_rounds, T)[b:b + 1, :, 0, :, :1]
                part["new_buckets"] = torch.where(near, mine, bk)
            _store(part, rows(n, 0, 1), rows(n, 1, 1))
    return s


def _own(s):
    import lsh_attention_hash_b200 as lsh

    c = s["case"]
    form = {"page": c["page"], "group": c["group"]}
    if c["kind"] == "append":
        lsh.lsh_cache_write(s["k"], s["v"], s["cache"], s["page_table"], s["ctx_len"], new_len=s["new_len"],
                            buckets=s.get("new_buckets"), tags=s.get("tags"), **form)
        k, v, inv = lsh.lsh_cache_read(s["cache"], s["page_table"], s["ctx_len"], s["T"], c["D"],
                                       new_len=s["new_len"], out_dtype=_dtype(c), **form)
        return {"k": k, "v": v, "key_inv": inv, **({"tags": s["tags"][:-1]} if c["rounds"] else {})}
    got, selected = {}, None
    if c["kind"] == "sparse":
        selected, scores = lsh.lsh_cache_select(s["tags"], s["q_buckets"], s["page_table"], s["ctx_len"],
                                                c["n_select"], new_len=s["new_len"], n_local=c["n_local"],
                                                causal=c["causal"])
        got = {"selected": selected, "scores": scores}
    out, lse = lsh.lsh_cache_attend(s["q"], s["cache"], s["page_table"], s["ctx_len"], new_len=s["new_len"],
                                    selected=selected, self_mask=c["self_mask"], causal=c["causal"],
                                    unit_keys=c["unit_keys"], **form)
    return {**got, "out": out, "lse": lse}


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "attend": _plain_attend, "sparse": _plain_sparse}[state["case"]["kind"]](state)


# ---------------------------------------------------------------------------------------------------
# The definition in 64 bits

def _exact_group(x, group):
    """Stored values of rows [N, D] (float64): the nearest of 16 levels from the group's smallest value up."""
    N, D = x.shape
    y = x.reshape(N * (D // group), group)
    lo, hi = y.min(1).values, y.max(1).values

    def step_of(v):  # distance between bf16 values at v: a power of two, put together from its exponent
        e = torch.frexp(v.abs().clamp_min(1e-290)).exponent.to(torch.int64) - 8
        return ((e + 1023) << 52).view(torch.float64)

    u = step_of(lo)
    zero = torch.floor(lo / u) * u
    scale = (hi - zero) / torch.full_like(hi, 15)
    u = step_of(scale)
    scale = torch.round(scale / u) * u
    scale = torch.where(hi == zero, torch.zeros_like(scale), scale)
    level = torch.where(scale[:, None] > 0, (y - zero[:, None]) / scale[:, None].clamp_min(1e-300), torch.zeros_like(y))
    return (zero[:, None] + scale[:, None] * level.round().clamp(0, 15)).reshape(N, D)


def _exact_rows(s, b, h, pages):
    """Stored keys, values (float64) and key lengths of whole pages (physical numbers) of head h."""
    c = s["case"]
    D, group = c["D"], c["group"]
    ng, tile, _, _ = _sizes(c)
    raw = s["cache"][pages, h].reshape(-1, tile)  # one row for 16 tokens
    d = torch.arange(D, device=DEV)
    r = torch.arange(16, device=DEV)
    kat = r[:, None] * (D // 2) + (((d % 8) // 2) * (D // 8) + 4 * (d // 32) + (d % 32) // 8)[None]
    khi = d % 2
    i = (d % 64) // 8
    vat = (8 * D + (r // 2 * D)[:, None] + ((d % 8)[None] ^ (2 * (r // 2 % 4))[:, None]) * (D // 8)
           + (d // 64 * 8)[None] + (r % 2 * 4)[:, None] + (i // 2)[None])
    vhi = i % 2

    def nibbles(at, high):
        x = raw[:, at.reshape(-1)].reshape(-1, 16, D).to(torch.int32)
        return ((x >> (4 * high)[None, None]) & 15).double()

    def params(first):
        w = raw[:, first:first + 64 * ng].contiguous().view(torch.int32).reshape(-1, ng, 16)
        sc = (w << 16).view(torch.float32).double()
        ze = (w & -65536).view(torch.float32).double()
        g = d // group
        return sc[:, g].transpose(1, 2), ze[:, g].transpose(1, 2)

    out = []
    for at, high, first in ((kat, khi, 16 * D), (vat, vhi, 16 * D + 64 * ng)):
        sc, ze = params(first)
        out.append((ze + sc * nibbles(at, high)).reshape(-1, D))
    inv = raw[:, 16 * D + 128 * ng:].contiguous().view(torch.float32).double().reshape(-1)
    return out[0], out[1], inv


def _exact_query(c, q, K, V, inv, keys, pos, ctx):
    """One query row against its keys (positions): out [D], lse."""
    keep = (keys >= 0) & (keys < ctx) & (pos >= 0)
    if c["causal"]:
        keep = keep & (keys <= pos)
    if c["self_mask"] and bool((keep & (keys != pos)).any()):
        keep = keep & (keys != pos)
    if not bool(keep.any()):
        return torch.zeros(c["D"], dtype=torch.float64, device=DEV), -math.inf
    z = (K[keep] @ q.double()) / math.sqrt(c["D"])
    if c["unit_keys"]:
        z = z * inv[keep]
    lse = torch.logsumexp(z, 0)
    return torch.exp(z - lse) @ V[keep], float(lse)


def exact(case, seed):
    c = dict(case)
    B, H, G, T, D, page = (c[k] for k in ("B", "H", "G", "T", "D", "page"))
    s = prepare(case, seed)
    ctx, new = _lengths(c, seed)
    f64 = {"dtype": torch.float64, "device": DEV}
    if c["kind"] == "append":
        k, v = torch.zeros(B, H, T, D, **f64), torch.zeros(B, H, T, D, **f64)
        inv = torch.zeros(B, H, T, **f64)
        for b in range(B):
            for h in range(H):
                n = new[b]
                if n:
                    x = s["k"][b, h, :n].double()
                    k[b, h, :n] = _exact_group(x, c["group"])
                    v[b, h, :n] = _exact_group(s["v"][b, h, :n].double(), c["group"])
                    inv[b, h, :n] = 1 / x.norm(dim=1).clamp_min(1e-12)
        return {"k": k, "v": v, "key_inv": inv}
    out = torch.zeros(B, H * G, T, D, **f64)
    lse = torch.full((B, H * G, T), -math.inf, **f64)
    table = s["page_table"].long()
    selected = None
    if c["kind"] == "sparse":
        if B * H * T * G > 1200:
            return None
        n_pages_max = table.shape[1]
        selected = torch.full((B, H, T, c["n_select"]), -1, dtype=torch.int32)
        scores = torch.full((B, H, T, n_pages_max), -1, dtype=torch.int32)
    elif B * H * T * G > 1200:
        return None
    for b in range(B):
        if ctx[b] == 0 or new[b] == 0:
            continue
        n_pages = -(-ctx[b] // page)
        for h in range(H):
            if selected is None:
                K, V, inv = _exact_rows(s, b, h, table[b, :n_pages])
                keys = torch.arange(n_pages * page, device=DEV)
            else:
                mine = s["tags"][table[b, :n_pages], h].to(torch.int32) & 0xFFFF  # [pages, rounds, page]
            for t in range(new[b]):
                pos = ctx[b] - new[b] + t
                if selected is not None:
                    limit = pos + 1 if c["causal"] else ctx[b]
                    n = -(-limit // page)
                    tag = mine[:n].clone()
                    at = torch.arange(n * page, device=DEV).reshape(n, 1, page).expand_as(tag)
                    tag[at >= limit] = -1
                    hits = sum((tag == s["q_buckets"][b, h * G + g, :, t][None, :, None]).sum((1, 2))
                               for g in range(G)).tolist()
                    scores[b, h, t, :n] = torch.tensor(hits, dtype=torch.int32)
                    always = set(range(max(0, n - c["n_local"]), n))
                    order = sorted(range(n), key=lambda j: (j not in always, -hits[j], j))
                    picked = sorted(order[:c["n_select"]])
                    selected[b, h, t, :len(picked)] = torch.tensor(picked, dtype=torch.int32)
                    where = torch.tensor(picked, device=DEV)
                    K, V, inv = _exact_rows(s, b, h, table[b][where])
                    keys = (where[:, None] * page + torch.arange(page, device=DEV)).reshape(-1)
                for g in range(G):
                    o, l = _exact_query(c, s["q"][b, h * G + g, t], K, V, inv, keys, pos, ctx[b])
                    out[b, h * G + g, t] = o
                    lse[b, h * G + g, t] = l
    got = {"out": out, "lse": lse}
    if selected is not None:
        got.update(selected=selected.to(DEV), scores=scores.to(DEV))
    return got
