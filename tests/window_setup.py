"""Set-up of the windowed-attention tests: streams placed so that only the rows
some query reads hold values, and the attention's definition in float64."""
from __future__ import annotations

import numpy as np

import oracle as orc
from paged_kv_cache_pg_gb300 import pkv, synth

from gpu_setup import CANARY, GUARD, dev_u16, torch


def read_rows(length, n_new, window, sinks):
    """Positions that some of a stream's last n_new queries read."""
    j = np.arange(length)
    return j[(j >= max(0, length - n_new + 1 - window)) | (j < sinks)]


def values(bits, fmt):
    """Rows of bf16 bits as the values a cache of the format holds, float64."""
    x = orc.bf16_to_float(bits)
    if fmt != pkv.KV_E4M3:
        return x
    scale = (np.abs(x).max(-1).astype(np.float32) / np.float32(448)).astype(np.float32)
    safe = np.where(scale > 0, scale, np.float32(1))
    codes = orc.e4m3_from_float((x.astype(np.float32) / safe[..., None]).astype(np.float32))
    return orc.e4m3_to_double(codes) * scale.astype(np.float64)[..., None]


def attend(k, v, q, length, window, sinks):
    """Float64 attention of the last queries; k, v [T][H][D] float64, q bf16
    bits [nq][Hq][D] -> [nq][Hq][D]."""
    nq, hq, d = q.shape
    grp = hq // k.shape[1]
    qf = orc.bf16_to_float(q)
    out = np.zeros((nq, hq, d))
    j = np.arange(length)
    for i in range(nq):
        p = length - nq + i
        see = j[(j <= p) & ((j > p - window) | (j < sinks))]
        for h in range(hq):
            s = (k[see, h // grp] @ qf[i, h]) / np.sqrt(d)
            w = np.exp(s - s.max())
            out[i, h] = (w @ v[see, h // grp]) / w.sum()
    return out


class Windowed:
    """Streams in one arena (ptok) or their own buffers (None).  Rows that no
    query reads, and the new rows when the call stores them, hold NaN bits;
    table entries of pages without a row that is read are -1."""

    def __init__(self, lay, streams, n_new, window, sinks, ptok, seed=0, fused=False, spare=2):
        t = torch()
        self.lay, self.streams, self.n_new, self.window, self.sinks = lay, streams, n_new, window, sinks
        shape = orc.Shape(lay.n_layers, lay.n_kv_heads, 256, lay.idx_dim, lay.kv_format)
        fp8 = lay.kv_format == pkv.KV_E4M3
        put = orc.put_rows8 if fp8 else orc.put_rows
        self.pgs, self.keep, self.hosts, self.ocaches = [], [], [], []
        if ptok is not None:
            counts = [synth.pages_for(s.length, ptok) for s in streams]
            n_pages = sum(counts) + spare
            ps = pkv.page_elems(lay, ptok)
            tables = synth.shuffled_tables(seed, n_pages, counts)
            arena = np.full(n_pages * ps, CANARY, np.uint16)
        for i, (s, n) in enumerate(zip(streams, n_new)):
            if ptok is None:
                cap = max(4, -(-s.length // 4) * 4)
                ps = pkv.page_elems(lay, cap)
                arena = np.full(ps, CANARY, np.uint16)
                oc = orc.Cache(arena, cap, ps, None, 1)
            else:
                oc = orc.Cache(arena, ptok, ps, tables[i], n_pages)
            rows = read_rows(s.length, n, window, sinks) if n else np.arange(0)
            if fused:
                rows = rows[rows < s.length - n]
            runs = np.split(rows, np.flatnonzero(np.diff(rows) != 1) + 1) if rows.size else []
            for layer in range(lay.n_layers):
                for r in runs:
                    a, b = int(r[0]), int(r[-1]) + 1
                    put(shape, oc, layer, orc.K, a, s.k[layer][a:b])
                    put(shape, oc, layer, orc.V, a, s.v[layer][a:b])
            self.ocaches.append(oc)
            if ptok is None:
                self._buffer(arena)
                self.pgs.append(pkv.pg(self._body(-1), None, ps, cap))
        if ptok is not None:
            self._buffer(arena)
            for i, (s, n) in enumerate(zip(streams, n_new)):
                tab = np.full(tables[i].size, -1, np.int32)
                live = np.unique(read_rows(s.length, n, window, sinks) // ptok) if n else np.arange(0)
                tab[live] = tables[i][live]
                dev = t.from_numpy(np.concatenate([tab, np.full(1, -1, np.int32)])).cuda()
                self.keep.append(dev)
                self.pgs.append(pkv.pg(self._body(0), dev, ps, ptok, n_pages, max(1, tab.size)))
        self.shape = shape

    def _buffer(self, arena):
        guarded = np.full(arena.size + 2 * GUARD, CANARY, np.uint16)
        guarded[GUARD:-GUARD] = arena
        self.hosts.append(guarded)
        self.keep.append(dev_u16(guarded))
        self.bufs = getattr(self, "bufs", []) + [self.keep[-1]]

    def _body(self, i):
        return self.bufs[i][GUARD:self.bufs[i].numel() - GUARD]

    def seqs(self):
        return [pkv.seq(g, s.length, n) for g, s, n in zip(self.pgs, self.streams, self.n_new)]

    def new_rows(self, layer):
        """(k_new, v_new, ik_new) of the streams' new tokens on the device."""
        cat = lambda f: dev_u16(np.concatenate([getattr(s, f)[layer][s.length - n:] for s, n in zip(self.streams, self.n_new)]))
        return cat("k"), cat("v"), cat("ik") if self.lay.idx_dim else None

    def reference(self, layer, q_list):
        return np.concatenate([attend(values(s.k[layer], self.lay.kv_format), values(s.v[layer], self.lay.kv_format), q,
                                      s.length, self.window, self.sinks) for s, q in zip(self.streams, q_list)])


def streams_of(lens, hkv, idx=0, layers=1, seed=0):
    return [synth.make_stream(seed + i, layers, T, hkv, 256, idx) for i, T in enumerate(lens)]


def queries_of(n_new, hq, seed=0):
    """Queries of the streams; every other stream's are eight times as large."""
    return [synth.scale_pow2(synth.queries(seed + i, n, hq, 256), 3 * (i & 1)) for i, n in enumerate(n_new)]
