"""Positions on the way into a paged cache, and decoding of streams that share a prompt; the sizes they are measured at.

rows: rotary positions applied to rows (queries, indexer queries): the first `rot` elements of a row turn in pairs, (i, i + rot/2)
or (2i, 2i + 1), by position x frequency, with the frequencies scaled for long contexts in one of four ways.
append: the same for a step's queries and keys, the keys, values and indexer keys going into their pages (bf16 rows, or e4m3 codes
with a float32 scale a row).
prefix: decode attention for groups of streams whose first pages are the same: each stream's query reads the shared positions and
its own, softmax(q.k / 16) . v.

``run`` computes each operator in plain torch operations, or, with ``own`` set, by the calls of ``paged_kv_cache_pg_gb300.pkv``.
"""
import math

import numpy as np
import torch

own = False

D = 256          # elements of a key or value row


# ---- the cases ---------------------------------------------------------------

def _rope(**k):
    """half or interleaved pairs over the first `rot` elements; scaling: none, linear, ntk, yarn or bands, by `factor` from `original`."""
    return dict(dict(layout="half", rot=64, base=1e6, scaling="none", factor=4.0, original=8192), **k)


def _rows(name, **k):
    return dict(_rope(), **dict(dict(name=name, op="rows", streams=1, longest=300, new=1, heads=16, dim=256, given=False), **k))


def _append(name, **k):
    return dict(_rope(), **dict(dict(name=name, op="append", format="bf16", streams=1, longest=300, new=1, q_heads=16, kv_heads=2, page=256, idx=128,
                                     fused=False), **k))


def _prefix(name, **k):
    return dict(dict(name=name, op="prefix", format="bf16", groups=1, streams=8, shared=4096, longest_own=256, new=1, q_heads=16, kv_heads=2, page=256,
                     idx=128, store=True), **k)


def listed():
    return [
        # one token's queries of a model that turns a quarter of the head: a call whose latency counts
        _rows("rows: one token", longest=9001),
        # the indexer queries of a prompt chunk on a long context, frequencies scaled by parts
        _rows("rows: indexer queries of a chunk", longest=44056, new=4096, dim=128, rot=128, layout="interleaved", scaling="yarn"),
        # a short chat's new token, 4 query heads on one KV head, pages of 16
        _append("append: one short stream", q_heads=4, kv_heads=1, page=16, idx=0, rot=256, base=1e4),
        # a full launch of decoding streams
        _append("append: 64 streams", streams=64, longest=40956, scaling="bands"),
        # a whole prompt out of one projection's rows
        _append("append: whole prompt", longest=8192, new=8192, rot=256, layout="interleaved", scaling="linear", fused=True),
        # a prompt chunk into e4m3 pages
        _append("append: e4m3 chunk", format="e4m3", longest=31512, new=512, page=128, scaling="ntk"),
        # two answers to a short prompt: a call whose latency counts
        _prefix("prefix: two short streams", streams=2, shared=240, longest_own=33, q_heads=4, kv_heads=1, page=16, idx=0),
        # eight samples of one prompt
        _prefix("prefix: eight samples", shared=9000, longest_own=500),
        # a full launch on one long document
        _prefix("prefix: 64 streams on a document", streams=64, shared=31000, longest_own=1000),
        # the same in e4m3 pages
        _prefix("prefix: e4m3 pages", format="e4m3", streams=32, shared=24000, longest_own=600, page=128, store=False),
        # four system prompts with eight streams each, pages that end inside a tile
        _prefix("prefix: four prompts", groups=4, shared=8000, longest_own=300, page=48),
        # speculative decoding: four draft tokens a stream
        _prefix("prefix: draft windows", streams=16, shared=16384, longest_own=700, new=4, page=128),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.99)))))))


def draw(rng):
    op = rng.choice(["rows", "append", "append", "prefix", "prefix", "prefix"])
    page = rng.choice([4, 16, 20, 48, 64, 128, 256])
    rope = dict(layout=rng.choice(["half", "interleaved"]), base=rng.choice([1e4, 5e5, 1e6]), scaling=rng.choice(["none", "linear", "ntk", "yarn", "bands"]),
                factor=rng.choice([2.0, 4.0, 8.0]), original=rng.choice([4096, 8192, 32768]))
    streams = _log(rng, 1, 64)
    if op == "rows":
        dim, new = rng.choice([128, 256]), _log(rng, 1, max(1, 4096 // streams))
        return _rows("", streams=streams, new=new, longest=new + _log(rng, 1, 1000000), heads=rng.choice([1, 2, 5, 8, 16]), dim=dim,
                     rot=rng.choice([dim, dim // 2, dim // 4, 2 * rng.randint(2, dim // 2)]), given=rng.random() < 0.3, **rope)
    kv = rng.choice([1, 2, 2, 4])
    if op == "append":
        new = _log(rng, 1, max(1, 4096 // streams))
        return _append("", format=rng.choice(["bf16", "bf16", "e4m3"]), streams=streams, new=new, longest=new + _log(rng, 1, 40000),
                       q_heads=kv * rng.choice([1, 2, 4, 5, 8]), kv_heads=kv, page=page, idx=rng.choice([0, 128]), fused=rng.random() < 0.5,
                       rot=rng.choice([256, 128, 64, 2 * rng.randint(2, 128)]), **rope)
    new = rng.choice([1, 1, 1, 2, 3, 4])
    group = rng.choice([1, 2, 4, 5, 8]) if new > 1 else rng.choice([1, 2, 4, 5, 8, 16])
    groups = rng.choice([1, 1, 2, 3, 5])
    each = _log(rng, 2, 64 // groups)
    c = _prefix("", format=rng.choice(["bf16", "bf16", "e4m3"]), groups=groups, streams=each, shared=_log(rng, 1, 31000 if kv < 4 else 15000),
                longest_own=new + _log(rng, 1, 900 if kv < 4 else 400), new=new, q_heads=kv * group, kv_heads=kv, page=page, idx=rng.choice([0, 128]),
                store=rng.random() < 0.6)
    while work(c)["flops"] > 3.2e10:
        c["shared"] = c["shared"] * 2 // 3
    return c


# ---- shapes ------------------------------------------------------------------

def _page_elems(c):
    """16-bit elements of a page (one layer)."""
    kv = 2 * c["kv_heads"] * c["page"] * D
    if c["format"] == "e4m3":
        kv = kv // 2 + 4 * c["kv_heads"] * c["page"]
    return kv + c["page"] * c["idx"] + c["page"] // 4 * c["idx"]


def _spread(most, least, n):
    """n lengths: the longest first, then spread over its lower half and above."""
    return [most if i == 0 else least + int((most - least) * (0.25 + 0.75 * ((i * 0.6180339887) % 1.0))) for i in range(n)]


def _lengths(c):
    return _spread(c["longest"], c["new"], c["streams"])


def _shared(c):
    """Each group's shared positions: whole pages."""
    return [max(1, n // c["page"]) * c["page"] for n in _spread(c["shared"], c["page"], c["groups"])]


def _own_lengths(c):
    """Each stream's positions behind the shared ones, its new tokens included."""
    return _spread(c["longest_own"], c["new"], c["groups"] * c["streams"])


def _row_bytes(c):
    """Bytes of a position's K and V rows in its page."""
    return c["kv_heads"] * (2 * (D + 4) if c["format"] == "e4m3" else 4 * D)


def work(c):
    if c["op"] == "rows":
        n = c["streams"] * c["new"] * c["heads"]
        return {"bytes": n * c["dim"] * 4 + (4 * c["streams"] * c["new"] if c["given"] else 0), "flops": n * c["rot"] * 3}
    q = c["q_heads"]
    if c["op"] == "append":
        n = c["streams"] * c["new"]
        return {"bytes": n * (q * D * 4 + c["kv_heads"] * D * 4 + _row_bytes(c) + c["idx"] * 4), "flops": n * (q + c["kv_heads"]) * c["rot"] * 3}
    by = sum(_shared(c)) * _row_bytes(c)
    pairs = sum(_shared(c)) * c["streams"] * c["new"]
    for own_n in _own_lengths(c):
        by += own_n * _row_bytes(c) + c["new"] * q * D * 4
        by += c["new"] * (c["kv_heads"] * D * 4 + c["idx"] * 4) if c["store"] else 0
        pairs += c["new"] * own_n - c["new"] * (c["new"] - 1) // 2
    return {"bytes": by, "flops": pairs * q * 4 * D}


# ---- what a user's program has in hand ---------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 29)
    return g


def _parts(c, arena):
    """Views of the parts of every page of `arena` [pages][elements] of 16 bits: k, v [pages][heads][page][D], ks, vs, ik."""
    h, p, i = c["kv_heads"], c["page"], c["idx"]
    out = {}
    if c["format"] == "e4m3":
        b, at = arena.view(torch.uint8), 0
        for name in ("k", "v"):
            out[name] = b[:, at:at + h * p * D].view(torch.float8_e4m3fn).unflatten(1, (h, p, D))
            at += h * p * D
        for name in ("ks", "vs"):
            out[name] = b[:, at:at + 4 * h * p].view(torch.float32).unflatten(1, (h, p))
            at += 4 * h * p
        at //= 2
    else:
        size = h * p * D
        out["k"] = arena[:, :size].view(torch.bfloat16).unflatten(1, (h, p, D))
        out["v"] = arena[:, size:2 * size].view(torch.bfloat16).unflatten(1, (h, p, D))
        at = 2 * size
    if i:
        out["ik"] = arena[:, at:at + p * i].view(torch.bfloat16).unflatten(1, (p, i))
    return out


def _bf16(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def _positions(c, lens):
    """Each new token's position, in stream order."""
    length = torch.tensor(lens, device="cuda")
    return (length[:, None] - c["new"] + torch.arange(c["new"], device="cuda")).flatten()


def _prepare_rows(c, seed):
    g = _generator(seed)
    n = c["streams"] * c["new"]
    pos = _positions(c, _lengths(c))
    if c["given"]:  # positions of the program's own, as for a prompt whose parts count anew
        pos = (pos * torch.rand(n, generator=g, device="cuda").to(torch.float64)).long()
    x = _bf16(g, n, c["heads"], c["dim"])
    return {"case": c, "lens": _lengths(c), "pos": pos, "pos32": pos.to(torch.int32) if c["given"] else None, "x": x, "out": torch.empty_like(x)}


def _prepare_append(c, seed):
    g = _generator(seed)
    b, h, p, new, q, i = c["streams"], c["kv_heads"], c["page"], c["new"], c["q_heads"], c["idx"]
    lens = _lengths(c)
    wide = -(-max(lens) // p)
    held = np.zeros((b, wide), dtype=bool)     # the pages that the new rows go to; the others are not looked at
    for s, n in enumerate(lens):
        held[s, (n - new) // p:-(-n // p)] = True
    count = int(held.sum())
    ids = torch.randperm(count + 2, generator=g, device="cuda").to(torch.int32)[:count]
    tables = torch.zeros((b, wide), dtype=torch.int32, device="cuda")
    tables[torch.from_numpy(held).to("cuda")] = ids
    arena = torch.zeros((count + 2, _page_elems(c)), dtype=torch.int16, device="cuda")
    _parts(c, arena)["v"].view(torch.uint8).random_(0, 40, generator=g)  # rows that others hold
    n = b * new
    if c["fused"]:  # rows of one projection: queries, keys, values, indexer keys side by side
        flat = _bf16(g, n, (q + 2 * h) * D + i)
        rows = [flat[:, :q * D].unflatten(1, (q, D)), flat[:, q * D:(q + h) * D].unflatten(1, (h, D)),
                flat[:, (q + h) * D:(q + 2 * h) * D].unflatten(1, (h, D)), flat[:, (q + 2 * h) * D:] if i else None]
    else:
        rows = [_bf16(g, n, q, D), _bf16(g, n, h, D), _bf16(g, n, h, D), _bf16(g, n, i) if i else None]
    return {"case": c, "arena": arena, "tables": tables, "lens": lens, "n_pages": count + 2, "pos": _positions(c, lens), "q": rows[0], "k_new": rows[1],
            "v_new": rows[2], "ik_new": rows[3], "q_out": torch.empty((n, q, D), dtype=torch.bfloat16, device="cuda"),
            "status": torch.zeros(1, dtype=torch.int32, device="cuda")}


def _prepare_prefix(c, seed):
    g = _generator(seed)
    h, p, new, m = c["kv_heads"], c["page"], c["new"], c["streams"]
    shared, mine = _shared(c), _own_lengths(c)
    b = c["groups"] * m
    first = [shared[s // m] for s in range(b)]                 # shared positions of each stream
    lens = [f + n for f, n in zip(first, mine)]
    wide = -(-max(lens) // p)
    slots = sum(n // p for n in shared) + sum(-(-n // p) for n in mine)
    n_pages = slots + 3
    ids = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32).cpu().numpy()
    host, at = np.full((b, wide), -1, dtype=np.int32), 0
    for k, n in enumerate(shared):
        host[k * m:(k + 1) * m, :n // p] = ids[at:at + n // p]
        at += n // p
    for s in range(b):
        f, e = first[s] // p, -(-lens[s] // p)
        host[s, f:e] = ids[at:at + e - f]
        at += e - f
    tables = torch.from_numpy(host).to("cuda")
    arena = torch.zeros((n_pages, _page_elems(c)), dtype=torch.int16, device="cuda")
    parts = _parts(c, arena)
    # keys that share a direction in the first few tokens, which the queries lean to, as trained models have it
    u = torch.where(torch.rand(D, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    if c["format"] == "e4m3":
        for name in ("k", "v"):
            x = torch.randn(n_pages, h, p, D, generator=g, device="cuda")
            if name == "k":
                x[tables[:, 0].long(), :, :4] += 2.0 * u
            scale = x.abs().amax(-1) / 448.0
            parts[name].copy_((x / scale[..., None]).to(torch.float8_e4m3fn))
            parts[name + "s"].copy_(scale)
    else:
        parts["k"].normal_(generator=g)
        parts["k"][tables[:, 0].long(), :, :4] += (2.0 * u).to(torch.bfloat16)
        parts["v"].normal_(generator=g)
    q = (2.0 * torch.randn((b * new, c["q_heads"], D), generator=g, device="cuda") + 0.25 * u).to(torch.bfloat16)
    st = {"case": c, "arena": arena, "tables": tables, "lens": lens, "lengths": torch.tensor(lens, device="cuda"), "shared": torch.tensor(shared, device="cuda"),
          "n_pages": n_pages, "pages": [n // p for n in shared], "q": q, "out": torch.empty_like(q), "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if c["store"]:
        st["k_new"], st["v_new"] = _bf16(g, b * new, h, D), _bf16(g, b * new, h, D)
        st["ik_new"] = _bf16(g, b * new, c["idx"]) if c["idx"] else None
    return st


def prepare(case, seed):
    return {"rows": _prepare_rows, "append": _prepare_append, "prefix": _prepare_prefix}[case["op"]](case, seed)


# ---- the plain forms ------------------------------------------------------------------

def _frequencies(c):
    """Radians a position of each pair, and the factor of cos and sin, in 64 bits."""
    d, factor, kind = c["rot"], c["factor"], c["scaling"]
    i = torch.arange(0, d, 2, device="cuda", dtype=torch.float64)
    base = c["base"] * factor ** (d / (d - 2)) if kind == "ntk" else c["base"]
    f = base ** (-i / d)
    if kind == "linear":
        f = f / factor
    if kind == "yarn":
        at = [d * math.log(c["original"] / (turns * 2 * math.pi)) / (2 * math.log(c["base"])) for turns in (32.0, 1.0)]
        low, high = max(0, math.floor(at[0])), min(d - 1, math.ceil(at[1]))
        ramp = ((i / 2 - low) / max(high - low, 1e-3)).clamp(0, 1)
        f = f / factor * ramp + f * (1 - ramp)
    if kind == "bands":
        t = ((c["original"] * f / (2 * math.pi) - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        f = f * t + f / factor * (1 - t)
    return f, 0.1 * math.log(factor) + 1.0 if kind == "yarn" else 1.0


def _turn(c, pos, *rows):
    """Rows [tokens][heads][dim] rotated by their positions, in 32 bits."""
    f, scale = _frequencies(c)
    angle = pos.to(torch.float64)[:, None] * f
    cos, sin = ((t(angle) * scale).float()[:, None] for t in (torch.cos, torch.sin))
    half, rot = c["rot"] // 2, c["rot"]
    a, b = (slice(0, half), slice(half, rot)) if c["layout"] == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    done = [x.float() for x in rows]
    done = [x.clone() if x.data_ptr() == r.data_ptr() else x for x, r in zip(done, rows)]
    pairs = [(x[..., a].clone(), x[..., b].clone()) for x in done]
    [(x[..., a].copy_(u * cos - v * sin), x[..., b].copy_(v * cos + u * sin)) for x, (u, v) in zip(done, pairs)]
    return done


def _place(c, st, pos, k, v, ik):
    """float32 K and V rows and indexer rows of the new tokens into their pages."""
    p, parts = c["page"], _parts(c, st["arena"])
    at = pos // p
    pid, row = st["tables"].repeat_interleave(c["new"], 0).gather(1, at[:, None])[:, 0].long(), pos % p
    if c["format"] == "e4m3":
        ks, vs = (x.abs().amax(-1) / 448.0 for x in (k, v))
        parts["ks"][pid, :, row], parts["vs"][pid, :, row] = ks, vs
        k, v = ((x / torch.where(s > 0, s, 1.0)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8) for x, s in ((k, ks), (v, vs)))
        parts["k"].view(torch.uint8)[pid, :, row], parts["v"].view(torch.uint8)[pid, :, row] = k, v
    else:
        parts["k"][pid, :, row], parts["v"][pid, :, row] = k.to(torch.bfloat16), v.to(torch.bfloat16)
    if c["idx"]:
        parts["ik"][pid, row] = ik
    return parts


def _plain_rows(st):
    return _turn(st["case"], st["pos"], st["x"])[0].to(torch.bfloat16)


def _plain_append(st):
    c = st["case"]
    q, k = _turn(c, st["pos"], st["q"], st["k_new"])
    return dict(_place(c, st, st["pos"], k, st["v_new"].float(), st["ik_new"]), q=q.to(torch.bfloat16))


def _values(c, parts, pid, row):
    """K and V of the rows at (page, row), in 32 bits: [...][heads][D]."""
    if c["format"] == "e4m3":
        return [parts[n].view(torch.uint8)[pid, :, row].view(torch.float8_e4m3fn).float() * parts[n + "s"][pid, :, row][..., None] for n in ("k", "v")]
    return [parts[n][pid, :, row].float() for n in ("k", "v")]


def _plain_prefix(st):
    c = st["case"]
    n_g, m, h, p, new = c["groups"], c["streams"], c["kv_heads"], c["page"], c["new"]
    b, grp, dev, length = n_g * m, c["q_heads"] // c["kv_heads"], st["q"].device, st["lengths"]
    out = {}
    if c["store"]:  # the new rows go to their pages first
        pos = (length[:, None] - new + torch.arange(new, device=dev)).flatten()
        out = _place(c, st, pos, st["k_new"].float(), st["v_new"].float(), st["ik_new"])
    parts, tables = _parts(c, st["arena"]), st["tables"]
    q = st["q"].float().view(b, new, h, grp, D).permute(0, 2, 1, 3, 4)           # [b][h][new][grp][D]
    # the shared positions, once a group
    key = torch.arange(_shared(c)[0] if n_g == 1 else max(_shared(c)), device=dev).expand(n_g, -1)
    live = key < st["shared"][:, None]
    key = torch.where(live, key, 0)
    k, v = _values(c, parts, tables[::m].gather(1, key // p).long(), key % p)      # [groups][keys][h][D]
    qg = q.reshape(n_g, m, h, new * grp, D).transpose(1, 2).reshape(n_g, h, m * new * grp, D)
    x1 = torch.matmul(qg, k.permute(0, 2, 3, 1)) / 16.0
    x1 = torch.where(live[:, None, None], x1, float("-inf"))
    # each stream's own
    first = st["shared"].repeat_interleave(m)[:, None]
    i = torch.arange(c["longest_own"], device=dev)
    pos = torch.where(first + i < length[:, None], first + i, first)
    k2, v2 = _values(c, parts, tables.gather(1, pos // p).long(), pos % p)
    x2 = torch.matmul(q.reshape(b, h, new * grp, D), k2.permute(0, 2, 3, 1)) / 16.0
    at = (length[:, None] - new + torch.arange(new, device=dev)).repeat_interleave(grp, 1)
    x2 = torch.where((first + i)[:, None, None] <= at[:, None, :, None], x2, float("-inf"))
    # one softmax over both
    x1 = x1.view(n_g, h, m, new * grp, -1).transpose(1, 2).reshape(b, h, new * grp, -1)
    top = torch.maximum(x1.amax(-1, keepdim=True), x2.amax(-1, keepdim=True))
    x1, x2 = torch.exp(x1 - top), torch.exp(x2 - top)
    total = x1.sum(-1, keepdim=True) + x2.sum(-1, keepdim=True)
    o = torch.matmul(x1.view(n_g, m, h, new * grp, -1).transpose(1, 2).reshape(n_g, h, m * new * grp, -1), v.permute(0, 2, 1, 3))
    o = o.view(n_g, h, m, new * grp, D).transpose(1, 2).reshape(b, h, new * grp, D)
    o = (o + torch.matmul(x2, v2.permute(0, 2, 1, 3))) / total
    o = o.view(b, h, new, grp, D).permute(0, 2, 1, 3, 4).reshape(b * new, c["q_heads"], D)
    return dict(out, out=o.to(torch.bfloat16))


# ---- the framework's calls -----------------------------------------------------------

def _handle(st):
    """What a serving program keeps: the layout, the streams, the rope, the workspace."""
    from paged_kv_cache_pg_gb300 import pkv
    c = st["case"]
    if c["op"] != "prefix":
        kinds = {"none": pkv.ROPE_PLAIN, "linear": pkv.ROPE_LINEAR, "ntk": pkv.ROPE_NTK, "yarn": pkv.ROPE_YARN, "bands": pkv.ROPE_BANDS}
        rope = pkv.rope(c["rot"], c["base"], pkv.ROPE_HALF if c["layout"] == "half" else pkv.ROPE_INTERLEAVED, kinds[c["scaling"]],
                        factor=c["factor"], original=c["original"])
    if c["op"] == "rows":
        st["handle"] = (pkv, rope, pkv.batch([pkv.seq(pkv.Pg(), n, c["new"]) for n in st["lens"]]))
        return st["handle"]
    lay = pkv.layout(1, c["kv_heads"], D, c["idx"], pkv.KV_E4M3 if c["format"] == "e4m3" else pkv.KV_BF16)
    ps = pkv.page_elems(lay, c["page"])
    seqs = pkv.batch([pkv.seq(pkv.pg(st["arena"], t, ps, c["page"], st["n_pages"]), n, c["new"]) for t, n in zip(st["tables"].unbind(0), st["lens"])])
    if c["op"] == "append":
        st["handle"] = (pkv, lay, seqs, rope, _parts(c, st["arena"]))
        return st["handle"]
    groups = pkv.groups([(c["streams"], n) for n in st["pages"]])
    ws = torch.empty(max(64, pkv.prefix_decode_ws_size(lay, seqs, groups, c["q_heads"]) // 4), dtype=torch.float32, device="cuda")
    st["handle"] = (pkv, lay, seqs, groups, ws, _parts(c, st["arena"]) if c["store"] else {})
    return st["handle"]


def _own_rows(st):
    c = st["case"]
    pkv, rope, seqs = st.get("handle") or _handle(st)
    pkv.rope_rows(rope, seqs, c["heads"], st["x"], st["out"], pos=st["pos32"])
    return st["out"]


def _own_append(st):
    c = st["case"]
    pkv, lay, seqs, rope, parts = st.get("handle") or _handle(st)
    pkv.rope_store(lay, seqs, 0, rope, st["k_new"], st["v_new"], st["ik_new"], n_q_heads=c["q_heads"], q=st["q"], q_out=st["q_out"], status=st["status"])
    return dict(parts, q=st["q_out"])


def _own_prefix(st):
    c = st["case"]
    pkv, lay, seqs, groups, ws, parts = st.get("handle") or _handle(st)
    pkv.prefix_decode(lay, seqs, groups, 0, c["q_heads"], st["q"], st["out"], ws, status=st["status"], k_new=st.get("k_new"), v_new=st.get("v_new"),
                      ik_new=st.get("ik_new"))
    return dict(parts, out=st["out"])


def run(state):
    op = state["case"]["op"]
    if own:
        return {"rows": _own_rows, "append": _own_append, "prefix": _own_prefix}[op](state)
    return {"rows": _plain_rows, "append": _plain_append, "prefix": _plain_prefix}[op](state)


# ---- the definition in 64 bits -----------------------------------------------------------

def _exact_turn(c, pos, x):
    """Complex numbers turned by unit ones: pair (a, b) is a + ib."""
    d, factor, kind, original = c["rot"], c["factor"], c["scaling"], c["original"]
    freq, scale = [], 1.0
    for i in range(d // 2):
        f = math.exp(-2.0 * i / d * math.log(c["base"]))
        if kind == "linear":
            f /= factor
        elif kind == "ntk":
            f = math.exp(-2.0 * i / d * (math.log(c["base"]) + d / (d - 2.0) * math.log(factor)))
        elif kind == "yarn":
            pair_at = lambda turns: d / 2.0 * math.log(original / (2 * math.pi * turns)) / math.log(c["base"])  # noqa: E731
            low, high = max(0, math.floor(pair_at(32.0))), min(d - 1, math.ceil(pair_at(1.0)))
            slow = min(1.0, max(0.0, (i - low) / max(high - low, 1e-3)))
            f, scale = f * (1.0 - slow) + f / factor * slow, 1.0 + math.log(factor) / 10.0
        elif kind == "bands":
            turns = original * f / (2 * math.pi)
            f = f if turns > 4.0 else f / factor if turns < 1.0 else f / factor + (f - f / factor) * (turns - 1.0) / 3.0
        freq.append(f)
    turn = torch.polar(torch.tensor(scale, dtype=torch.float64, device="cuda"), pos.double()[:, None] * torch.tensor(freq, dtype=torch.float64, device="cuda"))
    y = x.double()
    part, rest = y[..., :d], y[..., d:]
    z = torch.view_as_complex(part.unflatten(-1, (d // 2, 2)).contiguous()) if c["layout"] != "half" else torch.complex(part[..., :d // 2], part[..., d // 2:])
    z = z * turn[:, None]
    part = torch.view_as_real(z).flatten(-2) if c["layout"] != "half" else torch.cat([z.real, z.imag], -1)
    return torch.cat([part, rest], -1)


def _exact_place(c, st, lens, k, v, ik):
    """The pages' parts in 64 bits with each new row put in its place; codes as the values nearest x / scale."""
    parts = {n: t.double() for n, t in _parts(c, st["arena"]).items()}
    p, new, tables = c["page"], c["new"], st["tables"].cpu().numpy()
    pos = np.concatenate([np.arange(n - new, n) for n in lens])
    of = np.repeat(np.arange(len(lens)), new)
    pid, row = torch.from_numpy(tables[of, pos // p].astype(np.int64)).cuda(), torch.from_numpy(pos % p).cuda()
    for n, x in (("k", k), ("v", v)):
        x = x.double()
        if c["format"] == "e4m3":
            scale = x.abs().max(-1).values / 448.0
            parts[n + "s"][pid, :, row] = scale
            x = x / torch.where(scale > 0, scale, 1.0)[..., None]
            e = torch.frexp(x).exponent.double().clamp(min=-5) - 4   # steps of 2^-3 of the value's power of two, 2^-9 at least
            x = torch.round(x * 2.0 ** -e) * 2.0 ** e
        parts[n][pid, :, row] = x
    if c["idx"]:
        parts["ik"][pid, row] = ik.double()
    return parts


def exact(case, seed):
    st, c = prepare(case, seed), case
    if c["op"] == "rows":
        return _exact_turn(c, st["pos"], st["x"])
    if c["op"] == "append":
        return dict(_exact_place(c, st, st["lens"], _exact_turn(c, st["pos"], st["k_new"]), st["v_new"], st["ik_new"]), q=_exact_turn(c, st["pos"], st["q"]))
    # every query head of every stream by itself over all its positions
    h, p, new, m = c["kv_heads"], c["page"], c["new"], c["streams"]
    grp, out = c["q_heads"] // h, {}
    parts = _exact_place(c, st, st["lens"], st["k_new"], st["v_new"], st["ik_new"]) if c["store"] else None
    if parts is not None:
        out = dict(parts)
    if parts is None:
        parts = {n: t.double() for n, t in _parts(c, st["arena"]).items()}
    o = torch.zeros((c["groups"] * m, new, c["q_heads"], D), dtype=torch.float64, device="cuda")
    for s, n in enumerate(st["lens"]):
        ids = st["tables"][s, :-(-n // p)].long()
        rows = {}
        for name in ("k", "v"):
            t = parts[name][ids].transpose(0, 1).reshape(h, -1, D)[:, :n]
            if c["format"] == "e4m3":
                t = t * parts[name + "s"][ids].transpose(0, 1).reshape(h, -1)[:, :n, None]
            if c["store"]:  # rows of this step count as they are stored
                t = t.to(torch.bfloat16).double() if c["format"] != "e4m3" else t
            rows[name] = t
        hidden = torch.arange(n, device="cuda")[None, :] > torch.arange(n - new, n, device="cuda")[:, None]
        q = st["q"].view(-1, new, c["q_heads"], D)[s].double()
        for head in range(c["q_heads"]):
            x = (q[:, head] @ rows["k"][head // grp].T) / math.sqrt(D)
            o[s, :, head] = torch.softmax(x.masked_fill(hidden, -math.inf), -1) @ rows["v"][head // grp]
    return dict(out, out=o.view(-1, c["q_heads"], D))
