"""Set-up of the tests of decoding over shared pages: groups of streams placed in one arena, and the
attention's definition in float64."""
import numpy as np

from paged_kv_cache_pg_gb300 import pkv

from gpu_setup import torch
from rope_setup import bf16_bits, bf16_values, random_rows
from window_setup import values


class Shared:
    """groups: (streams' own lengths, shared pages); n_new: new tokens of each stream (one number, or a list).
    Unplaced rows are bf16 NaN, and with `fused` the new tokens' too.  ballast: that many streams more, of one new
    token each behind a prefix of 16,384 positions, the call's last group: their rows are so many that the call
    reads shared rows together, where one of the groups alone would be decoded stream by stream."""

    def __init__(self, lay, groups, n_new, ptok, fused=False, seed=0, layer=0, n_q_heads=8, spread=0, late=False, gain=1.0, ballast=0):
        t = torch()
        rng = np.random.default_rng(seed)
        h, fp8 = lay.n_kv_heads, lay.kv_format == pkv.KV_E4M3
        own = [n for g, _ in groups for n in g]
        new = [n_new] * len(own) if isinstance(n_new, int) else list(n_new)
        shared = [pages for g, pages in groups for _ in g]
        self.lay, self.layer, self.ptok, self.new, self.n_q_heads, self.fused = lay, layer, ptok, new, n_q_heads, fused
        self.lens = [o + s * ptok for o, s in zip(own, shared)]
        deep = -(-16384 // ptok)
        slots = sum(p for _, p in groups) + sum(-(-o // ptok) for o in own) + (ballast + deep if ballast else 0)
        self.n_pages = slots + 3
        self.ids = rng.permutation(self.n_pages).astype(np.int32)
        at, s, self.tables, self.k, self.v = 0, 0, [], [], []
        rows = lambda n: random_rows(rng, n, h, 256)  # noqa: E731
        for lengths, pages in groups:
            common, at = self.ids[at:at + pages], at + pages
            sk, sv = rows(pages * ptok), rows(pages * ptok)
            if spread:  # value rows of very different sizes
                sv = bf16_bits(bf16_values(sv) * 2.0 ** rng.integers(-spread, spread + 1, sv.shape[:2])[..., None])
            for n in lengths:
                p = -(-n // ptok)
                self.tables.append(np.concatenate([common, self.ids[at:at + p]]).astype(np.int32))
                at += p
                self.k.append(np.concatenate([sk, rows(n)]))
                self.v.append(np.concatenate([sv, rows(n)]))
                s += 1
        tokens = sum(new)
        self.q = bf16_bits(gain * bf16_values(random_rows(rng, tokens, n_q_heads, 256)))
        if late:  # a shared key along each stream's first query, far above the others, near the prefix's end
            tok = 0
            for i, m in enumerate(new):
                if m and shared[i]:
                    self.k[i][shared[i] * ptok - 5] = bf16_bits(2.0 * bf16_values(self.q[tok, ::n_q_heads // h]))
                    for j in range(len(new)):   # the same row for the streams that share it
                        if shared[j] and self.tables[j][0] == self.tables[i][0]:
                            self.k[j][shared[i] * ptok - 5] = self.k[i][shared[i] * ptok - 5]
                tok += m
        self.ik = random_rows(rng, tokens, lay.idx_dim) if lay.idx_dim else None
        # place: everything but the new tokens when the call stores them
        self.ps = pkv.page_elems(lay, ptok)
        self.mem = t.full((self.n_pages, self.ps), 0x7FC1, dtype=t.int16, device="cuda")
        self.dev_tables = [t.from_numpy(x).cuda() if x.size else t.zeros(1, dtype=t.int32, device="cuda") for x in self.tables]
        self.pgs = [pkv.pg(self.mem, x, self.ps, ptok, self.n_pages) for x in self.dev_tables]
        self.groups = [(len(g), p) for g, p in groups]
        d = self.dev
        for i in range(len(own)):
            n = self.lens[i] - (new[i] if fused else 0)
            if n:
                ik = t.zeros((n, lay.idx_dim), dtype=t.int16, device="cuda") if lay.idx_dim else None
                pkv.store(lay, [pkv.seq(self.pgs[i], n, n)], layer, d(self.k[i][:n]), d(self.v[i][:n]), ik)
        self.seqs = [pkv.seq(g, n, m) for g, n, m in zip(self.pgs, self.lens, new)]
        tail = lambda x: np.concatenate([x[i][self.lens[i] - new[i]:] for i in range(len(own))])  # noqa: E731
        self.k_new, self.v_new = d(tail(self.k)), d(tail(self.v))
        self.ik_new = d(self.ik) if lay.idx_dim else None
        self.dq = d(self.q)
        self.checked = tokens
        if ballast:
            gen = t.Generator("cuda").manual_seed(seed)
            some = lambda *shape: t.randn(shape, generator=gen, device="cuda").to(t.bfloat16).view(t.int16)  # noqa: E731
            for i in range(ballast):
                self.tables.append(np.concatenate([self.ids[at:at + deep], self.ids[at + deep + i:at + deep + i + 1]]).astype(np.int32))
                self.dev_tables.append(t.from_numpy(self.tables[-1]).cuda())
                self.pgs.append(pkv.pg(self.mem, self.dev_tables[-1], self.ps, ptok, self.n_pages))
            n = deep * ptok
            extra = [pkv.seq(g, n + 1, 1) for g in self.pgs[-ballast:]]
            new_rows = some(ballast, h, 256), some(ballast, h, 256), some(ballast, lay.idx_dim) if lay.idx_dim else None
            pkv.store(lay, [pkv.seq(self.pgs[-1], n, n)], layer, some(n, h, 256), some(n, h, 256), some(n, lay.idx_dim) if lay.idx_dim else None)
            if not fused:
                pkv.store(lay, extra, layer, *new_rows)
            self.seqs += extra
            self.groups.append((ballast, deep))
            self.lens, self.new = self.lens + [n + 1] * ballast, self.new + [1] * ballast
            self.k_new, self.v_new = t.cat([self.k_new, new_rows[0]]), t.cat([self.v_new, new_rows[1]])
            self.ik_new = t.cat([self.ik_new, new_rows[2]]) if lay.idx_dim else None
            self.dq = t.cat([self.dq, some(ballast, n_q_heads, 256)])

    @staticmethod
    def dev(bits):
        return torch().from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda()

    def ws(self, groups=None, seqs=None):
        t = torch()
        size = pkv.prefix_decode_ws_size(self.lay, seqs or self.seqs, self.groups if groups is None else groups, self.n_q_heads)
        return t.full((max(64, -(-size // 4)),), float("nan"), dtype=t.float32, device="cuda")

    def call(self, ws=None, out=None, stream=None, groups=None, status=None):
        t = torch()
        st = t.zeros(1, dtype=t.int32, device="cuda") if status is None else status
        out = t.full((self.dq.shape[0] + 1, self.n_q_heads, 256), 77, dtype=t.int16, device="cuda") if out is None else out
        kw = dict(k_new=self.k_new, v_new=self.v_new, ik_new=self.ik_new) if self.fused else {}
        pkv.prefix_decode(self.lay, self.seqs, self.groups if groups is None else groups, self.layer, self.n_q_heads, self.dq, out,
                          self.ws(groups) if ws is None else ws, status=st, stream=stream, **kw)
        if status is None:
            assert int(st) == 0
        return out

    def reference(self):
        """In float64, [tokens][heads][256]: outputs, sums of weight x |value|, and the part of the bound that fp16's
        grid of 2^-24 takes: the same sums with each weight (times the row's scale, e4m3) no more than 2^-23 of the
        largest, and bf16 values below 2^-14 half a step off."""
        t = torch()
        fmt, h, d, grp = self.lay.kv_format, self.lay.n_kv_heads, 256, self.n_q_heads // self.lay.n_kv_heads
        q = t.from_numpy(bf16_values(self.q)).cuda()
        out, size, small, tok = t.zeros_like(q), t.zeros_like(q), t.zeros_like(q), 0

        for i, m in enumerate(self.new[:len(self.k)]):
            if m == 0:
                continue
            n = self.lens[i]
            k, v = (t.from_numpy(values(x[i], fmt)).cuda().transpose(0, 1) for x in (self.k, self.v))   # [h][n][d]
            x = q[tok:tok + m].view(m, h, grp, d).permute(1, 0, 2, 3).reshape(h, m * grp, d) @ k.transpose(1, 2) / 16.0
            pos = t.arange(n - m, n, device="cuda").repeat_interleave(grp)
            x = x.masked_fill(t.arange(n, device="cuda")[None, :] > pos[:, None], float("-inf"))
            p = t.softmax(x, -1)
            top = v.abs().amax(-1, keepdim=True).clamp_min(1e-300) if fmt == pkv.KV_E4M3 else t.ones_like(v[..., :1])   # a row's scale x 448
            w = p * top.transpose(1, 2)
            off = (v.abs() < 2.0 ** -14).double() * 2.0 ** -25 if fmt == pkv.KV_BF16 else t.zeros_like(v)
            low = t.minimum(w, 2.0 ** -23 * w.amax(-1, keepdim=True))
            for to, val in ((out, p @ v), (size, p @ v.abs()), (small, low @ (v.abs() / top) + p @ off)):
                to[tok:tok + m] = val.view(h, m, grp, d).permute(1, 0, 2, 3).reshape(m, self.n_q_heads, d)
            tok += m
        return out.cpu().numpy(), size.cpu().numpy(), small.cpu().numpy()

    def check(self, out):
        """A weight has 11 significant bits (2^-11 of it at most): that much of the sum of weight x |value|; float32
        scores and sums of a few thousand terms stay below 2^-14 of it; the output is rounded to bf16.  A weight
        under 2^-14 of fp16's one, near which the largest lies or above (e4m3: weight x scale, no less than half of
        it below), is rounded to the grid of 2^-24: no more than itself off, nor than 2^-25 of the largest (e4m3:
        four times that, as the largest times its scale may be half of one, and a scale's mantissa is below 2).  A bf16
        value below 2^-14 is rounded to that grid too: 2^-25 off."""
        got = bf16_values(out.cpu().numpy().view(np.uint16))
        want, size, small = self.reference()
        assert np.isfinite(got[:-1]).all()
        got = got[:self.checked]
        err = np.abs(got - want) - (2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -14) * size + small + 1e-30)
        assert (err <= 0).all(), (err.max(), np.unravel_index(err.argmax(), err.shape))
        assert (out[-1] == 77).all()
