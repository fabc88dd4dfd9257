"""The operators of a long-running paged cache, and the sizes they are measured at.

Windowed attention: a query at position p reads the keys j <= p with
j > p - window or j < sinks (the first few tokens stay visible), through a
page table whose entries behind the window may be gone.  Its decode form takes
one to a few new tokens a stream (stored by the same call or before it), its
prefill form a whole chunk.  Page maintenance: copies of pages inside the
arena (a fork's tails, whole pages), and the compaction of an arena: its pages
copied down and the streams' tables rewritten.

``run`` computes each operator in plain torch operations, or, with ``own``
set, by the calls of ``paged_kv_cache_pg_gb300.pkv``.
"""
import math

import numpy as np
import torch

own = False

D = 256          # elements of a key or value row
STALE = 0x7FC1   # bits of rows that nothing placed: a bf16 NaN


# ---- the cases ---------------------------------------------------------------

def _decode(name, **k):
    return dict(dict(name=name, op="decode", format="bf16", streams=1, longest=300, new=1, q_heads=16,
                     kv_heads=2, window=1024, sinks=4, page=256, idx=128, store=False), **k)


def _prefill(name, **k):
    return dict(dict(name=name, op="prefill", format="bf16", streams=1, longest=1000, new=512, q_heads=16,
                     kv_heads=2, window=1024, sinks=4, page=256, idx=128, store=False), **k)


def _copy(name, **k):
    return dict(dict(name=name, op="copy", format="bf16", layers=13, kv_heads=2, idx=128, page=256,
                     pages=4, positions=0), **k)


def _compact(name, **k):
    return dict(dict(name=name, op="compact", format="bf16", layers=13, kv_heads=2, idx=128, page=64,
                     streams=4, each=16, moves=16), **k)


def listed():
    return [
        # one short chat, 4 query heads on one KV head, pages of 16: a call whose latency counts
        _decode("decode: one short stream", q_heads=4, kv_heads=1, window=128, page=16, idx=0),
        # four ragged streams, the new token stored by the call
        _decode("decode: four streams", streams=4, longest=9001, store=True),
        # a full launch of long streams: bound by the window's K and V bytes
        _decode("decode: 64 long streams", streams=64, longest=40956, window=4096, store=True),
        # the same in the e4m3 page format
        _decode("decode: e4m3 pages", format="e4m3", streams=32, longest=24000, window=4096, page=128),
        # speculative decoding: four draft tokens a stream, an odd window, pages that end inside a tile
        _decode("decode: draft windows", streams=8, longest=16384, new=4, window=2047, sinks=3, page=48, store=True),
        # short ragged prompt chunks on pages of 20
        _prefill("prefill: short chunks", streams=3, longest=1000, new=40, q_heads=4, kv_heads=1, window=500, sinks=1,
                 page=20, idx=0),
        # a 512-token chunk on a long context
        _prefill("prefill: chunk at 31000", longest=31512, window=4096),
        # a whole prompt of 8192 tokens
        _prefill("prefill: whole prompt", longest=8192, new=8192),
        # a fork of four streams in the middle of a page: the tails' rows
        _copy("copy: tails of a fork", positions=77),
        # whole pages of 7.9 MB each
        _copy("copy: whole pages", pages=96),
        # a small arena of e4m3 pages made dense again
        _compact("compact: small pages", format="e4m3", layers=4, page=16, streams=4, each=40, moves=50),
        # a serving arena: 16 streams, 300 pages moved down and every table rewritten
        _compact("compact: serving arena", streams=16, each=40, moves=300),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.99)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prefill", "copy", "compact"])
    kv = rng.choice([1, 2, 2, 4])
    page = rng.choice([4, 16, 20, 48, 64, 128, 256])
    idx = rng.choice([0, 128])
    if op == "decode":
        new = rng.choice([1, 1, 1, 2, 3, 4])
        group = rng.choice([1, 2, 4, 5, 8, 16]) if new == 1 else rng.choice([1, 3, 4, 8])
        streams, window = _log(rng, 1, 64), _log(rng, 1, 4096)
        if kv == 4:
            streams = min(streams, 32)
        fp8 = rng.random() < 0.35
        return _decode("", format="e4m3" if fp8 else "bf16", streams=streams, longest=_log(rng, new + 1, 40956), new=new,
                       q_heads=kv * group, kv_heads=kv, window=window, sinks=rng.choice([0, 1, 4, 17, 64]), page=page,
                       idx=idx, store=not fp8 and rng.random() < 0.7)
    if op == "prefill":
        new = _log(rng, 2, 4096)
        streams = min(_log(rng, 1, 8), max(1, 4096 // new))
        return _prefill("", streams=streams, longest=new + _log(rng, 1, 20000) - 1, new=new, q_heads=kv * rng.choice([1, 2, 4, 8] if kv < 4 else [1, 2, 4]),
                        kv_heads=kv, window=_log(rng, 1, 2048), sinks=rng.choice([0, 1, 4, 17, 64]), page=page, idx=idx)
    fmt, layers = rng.choice(["bf16", "bf16", "e4m3"]), rng.choice([1, 3, 13])
    if op == "copy":
        return _copy("", format=fmt, layers=layers, kv_heads=kv, idx=idx, page=page, pages=_log(rng, 1, 48),
                     positions=rng.choice([0, rng.randint(1, page), rng.randint(1, page)]))
    streams, each = _log(rng, 1, 16), _log(rng, 2, 20)
    return _compact("", format=fmt, layers=layers, kv_heads=kv, idx=idx, page=min(page, 64), streams=streams, each=each,
                    moves=rng.randint(1, streams * each))


# ---- shapes ------------------------------------------------------------------

def _layer_elems(c):
    """16-bit elements of one layer's block in a page."""
    kv = 2 * c["kv_heads"] * c["page"] * D
    if c["format"] == "e4m3":
        kv = kv // 2 + 4 * c["kv_heads"] * c["page"]
    return kv + c["page"] * c["idx"] + c["page"] // 4 * c["idx"]


def _lengths(c):
    """Each stream's length, its new tokens included: the longest first, then spread over its lower half and above."""
    most, new = c["longest"], c["new"]
    return [most if i == 0 else new + int((most - new) * (0.25 + 0.75 * ((i * 0.6180339887) % 1.0))) for i in range(c["streams"])]


def _seen(c, n):
    """Positions that some query of a stream of n positions reads, and its (query, key) pairs."""
    w, s, q0 = c["window"], c["sinks"], n - c["new"]
    lo = max(0, q0 + 1 - w)
    pairs = 0
    for p in (range(q0, n) if c["new"] <= 64 else ()):
        a = max(0, p + 1 - w)
        pairs += p + 1 - a + min(s, a)
    if c["new"] > 64:
        p = np.arange(q0, n, dtype=np.int64)
        a = np.maximum(0, p + 1 - w)
        pairs = int((p + 1 - a + np.minimum(s, a)).sum())
    return n - lo + min(s, lo), pairs


def work(c):
    h, q = c["kv_heads"], c.get("q_heads", 0)
    if c["op"] in ("decode", "prefill"):
        row = h * (2 * (D + 4) if c["format"] == "e4m3" else 4 * D)
        by = fl = 0
        for n in _lengths(c):
            rows, pairs = _seen(c, n)
            by += rows * row + c["new"] * q * D * 4 + (c["new"] * (row + 2 * c["idx"] * 2) if c["store"] else 0)
            fl += pairs * q * 4 * D
        return {"bytes": by, "flops": fl}
    if c["op"] == "copy":
        n = c["positions"] or c["page"]
        per = h * n * (2 * (D + 4) if c["format"] == "e4m3" else 4 * D) + n * c["idx"] * 2 + n // 4 * c["idx"] * 2
        return {"bytes": 2 * c["pages"] * c["layers"] * per, "flops": 0}
    return {"bytes": 2 * c["moves"] * c["layers"] * _layer_elems(c) * 2 + 2 * 4 * c["streams"] * c["each"], "flops": 0}


# ---- what a user's program has in hand ---------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)
    return g


def _parts(c, arena):
    """Views of the first layer's parts of every page of `arena` [pages][elements] of 16 bits."""
    h, p, i = c["kv_heads"], c["page"], c["idx"]
    out, n = {}, arena.shape[0]
    if c["format"] == "e4m3":
        b, at = arena.view(torch.uint8), 0
        for name, size in (("k", h * p * D), ("v", h * p * D)):
            out[name] = b[:, at:at + size].view(torch.float8_e4m3fn).unflatten(1, (h, p, D))
            at += size
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


def _prepare_attention(c, seed):
    g = _generator(seed)
    dev = "cuda"
    b, h, p, new, w, s = c["streams"], c["kv_heads"], c["page"], c["new"], c["window"], c["sinks"]
    lens = _lengths(c)
    # pages still held: those with a sink or a position of the windows; the others are given back (-1)
    wide = -(-max(lens) // p)
    held = np.zeros((b, wide), dtype=bool)
    for i, n in enumerate(lens):
        lo = max(0, n - new + 1 - w)
        held[i, lo // p:-(-n // p)] = True
        held[i, :-(-min(s, n) // p)] = True
    count = int(held.sum())
    n_pages = count + 3
    ids = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)[:count]
    tables = torch.full((b, wide), -1, dtype=torch.int32, device=dev)
    tables[torch.from_numpy(held).to(dev)] = ids
    ps = _layer_elems(c)
    arena = torch.full((n_pages, ps), STALE, dtype=torch.int16, device=dev)
    parts = _parts(c, arena)
    # keys with a common direction in the sink tokens, which the queries lean to, as trained models have it
    u = torch.where(torch.rand(D, generator=g, device=dev) < 0.5, -1.0, 1.0)
    length = torch.tensor(lens, device=dev)
    # every position that a query reads, with its page row
    pos = torch.arange(wide * p, device=dev).expand(b, -1)
    lo = (length - new + 1 - w).clamp(min=0)[:, None]
    live = (pos < length[:, None]) & ((pos >= lo) | (pos < s))
    bi, ji = live.nonzero(as_tuple=True)
    pid, row = tables[bi, ji // p].long(), ji % p
    fresh = ji >= (length - new)[bi]
    k = torch.randn((bi.numel(), h, D), generator=g, device=dev) + 2.0 * u * (ji < s)[:, None, None]
    v = torch.randn((bi.numel(), h, D), generator=g, device=dev)
    state = {"case": c, "arena": arena, "tables": tables, "lens": lens, "n_pages": n_pages, "lengths": length}
    if c["format"] == "e4m3":
        for name, x in (("k", k), ("v", v)):
            scale = x.abs().amax(-1) / 448.0
            parts[name].view(torch.uint8)[pid, :, row] = (x / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
            parts[name + "s"][pid, :, row] = scale
    else:
        stored = ~fresh if c["store"] else torch.ones_like(fresh)
        for name, x in (("k", k), ("v", v)):
            parts[name].view(torch.int16)[pid[stored], :, row[stored]] = x[stored].to(torch.bfloat16).view(torch.int16)
    q = 2.0 * torch.randn((b * new, c["q_heads"], D), generator=g, device=dev) + 0.25 * u
    state["q"] = q.to(torch.bfloat16)
    if c["store"]:  # the new rows, in stream order
        state["k_new"] = k[fresh].to(torch.bfloat16).contiguous()
        state["v_new"] = v[fresh].to(torch.bfloat16).contiguous()
        state["ik_new"] = torch.randn((b * new, c["idx"]), generator=g, device=dev).to(torch.bfloat16) if c["idx"] else None
    state["out"] = torch.empty_like(state["q"])
    state["status"] = torch.zeros(1, dtype=torch.int32, device=dev)
    return state


def _prepare_pages(c, seed):
    g = _generator(seed)
    rng = np.random.default_rng(seed)
    ps = c["layers"] * _layer_elems(c)
    if c["op"] == "copy":
        n_pages = 2 * c["pages"] + 3
        ids = rng.permutation(n_pages).astype(np.int32)
        src, dst = ids[:c["pages"]], ids[c["pages"]:2 * c["pages"]]
        tables = None
    else:
        # the held pages lie anywhere in an arena with as many holes as moves: the highest ones go to the lowest holes
        live = c["streams"] * c["each"]
        n_pages = live + c["moves"]
        src = np.sort(rng.choice(np.arange(live, n_pages), size=c["moves"], replace=False)).astype(np.int32)
        dst = np.sort(rng.choice(live, size=c["moves"], replace=False)).astype(np.int32)
        ids = rng.permutation(np.concatenate([np.setdiff1d(np.arange(live), dst), src])).astype(np.int32)
        tables = torch.from_numpy(ids.reshape(c["streams"], c["each"])).cuda()
    arena = torch.randint(-32768, 32767, (n_pages, ps), generator=g, device="cuda", dtype=torch.int16)
    n_pos = np.full(src.size, c["positions"], dtype=np.int32) if c.get("positions") else None
    return {"case": c, "arena": arena, "tables": tables, "n_pages": n_pages, "src": np.ascontiguousarray(src),
            "dst": np.ascontiguousarray(dst), "n_pos": n_pos, "src_dev": torch.from_numpy(src.astype(np.int64)).cuda(),
            "dst_dev": torch.from_numpy(dst.astype(np.int64)).cuda()}


def prepare(case, seed):
    return (_prepare_attention if case["op"] in ("decode", "prefill") else _prepare_pages)(case, seed)


# ---- the plain forms ------------------------------------------------------------------

def _plain_attention(st):
    c = st["case"]
    b, h, p, new, s = c["streams"], c["kv_heads"], c["page"], c["new"], c["sinks"]
    w, grp = min(c["window"], c["longest"]), c["q_heads"] // c["kv_heads"]
    dev, length, parts = st["q"].device, st["lengths"], _parts(c, st["arena"])
    q0 = length - new
    if c["store"]:  # the new rows go to their pages first
        j = q0[:, None] + torch.arange(new, device=dev)
        pid, row = torch.gather(st["tables"], 1, j // p).long().flatten(), (j % p).flatten()
        parts["k"].view(torch.int16)[pid, :, row] = st["k_new"].view(torch.int16)
        parts["v"].view(torch.int16)[pid, :, row] = st["v_new"].view(torch.int16)
        if c["idx"]:
            parts["ik"].view(torch.int16)[pid, row] = st["ik_new"].view(torch.int16)
    # slots: the sinks before the windows, then the positions from the first query's window on
    lo = (q0 + 1 - w).clamp(min=0)[:, None]
    i = torch.arange(s + w + new - 1, device=dev)
    pos = torch.where(i < s, i, lo + i - s)
    live = torch.where(i < s, i < lo, pos < length[:, None])
    pos = torch.where(live, pos, q0[:, None])
    pid, row = torch.gather(st["tables"], 1, pos // p).long(), pos % p
    if c["format"] == "e4m3":
        k, v = (parts[n].view(torch.uint8)[pid, :, row].view(torch.float8_e4m3fn).float() * parts[n + "s"][pid, :, row][..., None]
                for n in ("k", "v"))
    else:
        k, v = (parts[n][pid, :, row].float() for n in ("k", "v"))     # [b][slots][h][D]
    q = st["q"].float().view(b, new, h, grp, D).permute(0, 2, 1, 3, 4).reshape(b, h, new * grp, D)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * (1.0 / 16.0)           # [b][h][new * grp][slots]
    p_q = (q0[:, None] + torch.arange(new, device=dev)).repeat_interleave(grp, 1)[:, :, None]
    key = pos[:, None, :]
    sees = live[:, None, :] & (key <= p_q) & ((key > p_q - c["window"]) | (key < s))
    x = torch.where(sees[:, None], x, float("-inf"))
    x = torch.exp(x - x.amax(-1, keepdim=True))
    o = torch.matmul(x, v.permute(0, 2, 1, 3)) / x.sum(-1, keepdim=True)
    o = o.view(b, h, new, grp, D).permute(0, 2, 1, 3, 4).reshape(b * new, c["q_heads"], D).to(torch.bfloat16)
    return {"out": o, "arena": st["arena"]} if c["store"] else {"out": o}


def _plain_copy(st):
    c, arena, src, dst = st["case"], st["arena"], st["src_dev"], st["dst_dev"]
    n = c.get("positions", 0)
    if not n or n == c["page"]:
        wide = arena.view(torch.int64)
        wide[dst] = wide[src]
        return
    # a page's first n positions: the rows of each part, seen as bytes of the layers' blocks
    h, p, idx, fp8 = c["kv_heads"], c["page"], c["idx"], c["format"] == "e4m3"
    raw = arena.view(torch.uint8).view(arena.shape[0], c["layers"], -1)
    at = 0
    for heads, rows, size, take in ((2 * h, p, D if fp8 else 2 * D, n), (2 * h if fp8 else 0, p, 4, n),
                                    (1 if idx else 0, p, 2 * idx, n), (1 if idx else 0, p // 4, 2 * idx, n // 4)):
        part = raw[:, :, at:at + heads * rows * size].unflatten(2, (heads, rows, size)) if heads else None
        if heads and take:
            part[dst, :, :, :take] = part[src, :, :, :take]
        at += heads * rows * size


def _plain_pages(st):
    _plain_copy(st)
    if st["tables"] is None:
        return {"arena": st["arena"]}
    to = torch.arange(st["n_pages"], device="cuda", dtype=torch.int32)
    to[st["src_dev"]] = st["dst_dev"].to(torch.int32)
    st["tables"].copy_(to[st["tables"].long()])
    return {"arena": st["arena"], "tables": st["tables"]}


# ---- the framework's calls -----------------------------------------------------------

def _layout(pkv, c):
    return pkv.layout(c.get("layers", 1), c["kv_heads"], D, c["idx"], pkv.KV_E4M3 if c["format"] == "e4m3" else pkv.KV_BF16)


def _handle(st):
    """The layout, the streams and the workspace that a serving program keeps."""
    from paged_kv_cache_pg_gb300 import pkv
    c = st["case"]
    lay = _layout(pkv, c)
    if c["op"] in ("copy", "compact"):
        tables = [] if st["tables"] is None else list(st["tables"].unbind(0))
        st["handle"] = (pkv, lay, tables)
        return st["handle"]
    ps = pkv.page_elems(lay, c["page"])
    seqs = pkv.batch([pkv.seq(pkv.pg(st["arena"], t, ps, c["page"], st["n_pages"]), n, c["new"])
                      for t, n in zip(st["tables"].unbind(0), st["lens"])])
    size = pkv.window_decode_ws_size if c["op"] == "decode" else pkv.window_prefill_ws_size
    ws = torch.empty(max(64, size(lay, seqs, c["q_heads"], c["window"], c["sinks"]) // 4), dtype=torch.float32, device="cuda")
    st["handle"] = (pkv, lay, seqs, ws)
    return st["handle"]


def _own_attention(st):
    c = st["case"]
    pkv, lay, seqs, ws = st.get("handle") or _handle(st)
    if c["op"] == "decode":
        pkv.window_decode(lay, seqs, 0, c["q_heads"], c["window"], c["sinks"], st["q"], st["out"], ws, status=st["status"],
                          k_new=st.get("k_new"), v_new=st.get("v_new"), ik_new=st.get("ik_new"))
    else:
        pkv.window_prefill(lay, seqs, 0, c["q_heads"], c["window"], c["sinks"], st["q"], st["out"], ws, status=st["status"])
    return {"out": st["out"], "arena": st["arena"]} if c["store"] else {"out": st["out"]}


def _own_pages(st):
    c = st["case"]
    pkv, lay, tables = st.get("handle") or _handle(st)
    pkv.pages_copy(lay, c["page"], st["arena"], st["n_pages"], st["src"], st["dst"], n_pos=st["n_pos"])
    if st["tables"] is None:
        return {"arena": st["arena"]}
    pkv.tables_remap(tables, st["src"], st["dst"])
    return {"arena": st["arena"], "tables": st["tables"]}


def run(state):
    attention = state["case"]["op"] in ("decode", "prefill")
    if own:
        return (_own_attention if attention else _own_pages)(state)
    return (_plain_attention if attention else _plain_pages)(state)


# ---- the definition in 64 bits -----------------------------------------------------------

def exact(case, seed):
    """Each query head of each stream by itself, its keys found one page at a time; None for what is moved and not computed."""
    if case["op"] not in ("decode", "prefill"):
        return None
    st = prepare(case, seed)
    c, arena, new = case, st["arena"], case["new"]
    h, p, grp = c["kv_heads"], c["page"], c["q_heads"] // c["kv_heads"]
    tables, raw = st["tables"].cpu().numpy(), arena.view(torch.uint8)
    fp8 = c["format"] == "e4m3"
    out = torch.zeros((c["streams"], new, c["q_heads"], D), dtype=torch.float64, device="cuda")
    for s, n in enumerate(st["lens"]):
        first = max(0, n - new + 1 - c["window"])
        need = [j for j in range(n) if j >= first or j < c["sinks"]]
        rows = {"k": [], "v": []}
        kept = np.array([j for j in need if not (c["store"] and j >= n - new)], dtype=np.int64)
        for js in np.split(kept, np.flatnonzero(np.diff(kept // p)) + 1) if kept.size else []:
            pg = int(js[0]) // p
            at = torch.from_numpy(js - pg * p).cuda()
            block = raw[int(tables[s, pg])]
            for which, name in enumerate(("k", "v")):
                if fp8:
                    codes = block[which * h * p * D:(which + 1) * h * p * D].view(torch.float8_e4m3fn).view(h, p, D)
                    z = 2 * h * p * D + which * 4 * h * p
                    scale = block[z:z + 4 * h * p].view(torch.float32).view(h, p)
                    rows[name].append(codes.to(torch.float64)[:, at] * scale.to(torch.float64)[:, at, None])
                else:
                    z = which * 2 * h * p * D
                    rows[name].append(block[z:z + 2 * h * p * D].view(torch.bfloat16).view(h, p, D)[:, at].to(torch.float64))
        if c["store"]:
            for name in ("k", "v"):
                rows[name].append(st[name + "_new"].view(-1, new, h, D)[s].to(torch.float64).transpose(0, 1))
        k, v = torch.cat(rows["k"], 1), torch.cat(rows["v"], 1)
        key = torch.tensor(need, device="cuda")[None, :]
        at = torch.arange(n - new, n, device="cuda")[:, None]
        hidden = (key > at) | ((key <= at - c["window"]) & (key >= c["sinks"]))
        q = st["q"].view(c["streams"], new, c["q_heads"], D)[s].to(torch.float64)
        for head in range(c["q_heads"]):
            x = (q[:, head] @ k[head // grp].T) / math.sqrt(D)
            out[s, :, head] = torch.softmax(x.masked_fill(hidden, -math.inf), -1) @ v[head // grp]
    out = out.view(c["streams"] * new, c["q_heads"], D)
    return {"out": out, "arena": None} if c["store"] else {"out": out}
