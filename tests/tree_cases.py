"""Drafted trees on both caches: inputs, the library's calls, and plain answers in 64 bits."""

from __future__ import annotations

import math

import numpy as np

import oracle
from mixed_precision_bit_gb300 import synth
from tests.kitty_cases import dev16, dev32

P, D = 32, 128
SM = float(np.float32(1 / math.sqrt(D)))


def dev64(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a).view(np.int64)).cuda()


def starts(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def random_parents(r, n):
    """A tree of n nodes: half its nodes follow the node before, the others any earlier one or none."""
    return np.array([i - 1 if r.random() < 0.5 else int(r.integers(-1, i)) if i else -1 for i in range(n)], np.int32)


def masks_of(parents):
    m = []
    for i, p in enumerate(parents):
        m.append((m[p] if 0 <= p < i else 0) | 1 << i)
    return np.array(m, np.uint64)


def visible_of(kind, r, counts, pad=0):
    """Masks of every row of ragged trees, uint64 [sum + pad]; None for chains."""
    if kind == "chain":
        return None
    rows = []
    for n in counts:
        if kind == "tree":
            rows += [int(x) for x in masks_of(random_parents(r, n))]
        else:  # any bits, those of nodes that are not there too; some rows none
            rows += [0 if r.random() < 0.3 else int(r.integers(0, 1 << 63)) << 1 | int(r.integers(0, 2)) for _ in range(n)]
    return np.array(rows + [(1 << 64) - 1] * pad, np.uint64)


def sees(visible, start, b):
    """bool [n, n] of sequence b."""
    lo, n = int(start[b]), int(start[b + 1] - start[b])
    if visible is None:
        return np.tril(np.ones((n, n), bool))
    return np.array([[int(visible[lo + i]) >> j & 1 for j in range(n)] for i in range(n)], bool).reshape(n, n)


class Base:
    sm = SM

    def _rows(self, r, counts, sigma, pad, visible, q_scale):
        self.counts, self.start, self.visible = list(counts), starts(counts), visible
        self.T = int(self.start[-1]) + pad
        H = self.Hq + 2 * self.Hkv
        x = r.standard_normal((self.T, H, D))
        x[:, :self.Hq] *= q_scale
        x[:, self.Hq:self.Hq + self.Hkv] *= sigma
        self.rows = synth.to_bits(x, self.dt)
        self.put_rows()

    def put_rows(self):
        """The rows on the device, queries, keys and values as slices of one projection."""
        self.d_rows = dev16(self.rows)
        Hq, Hkv = self.Hq, self.Hkv
        self.d = dict(q=self.d_rows[:, :Hq], k=self.d_rows[:, Hq:Hq + Hkv], v=self.d_rows[:, Hq + Hkv:],
                      start=dev32(self.start), visible=None if self.visible is None else dev64(self.visible))

    def run(self, out_dtype="f32", status=None, **kw):
        import torch
        t = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[out_dtype]
        out = torch.full((self.T, self.Hq, D), 7.0, dtype=t, device="cuda")
        self.call(out, status=status, **kw)
        torch.cuda.synchronize()
        assert (out[int(self.start[-1]):] == 7.0).all()  # rows behind the last sequence
        return out[:int(self.start[-1])].float().cpu().numpy().astype(np.float64)

    def max_nodes(self):
        return max(max(self.counts), 1)

    def workspace(self):
        import torch
        n = self.size(self.cfg, self.B, self.T, self.max_nodes(), self.max_pages, self.n_prefix)
        return torch.full((max(n, 16) // 4,), float("nan"), dtype=torch.float32, device="cuda")

    def prefix_args(self):
        if not self.n_prefix:
            return {}
        return dict(prefix_table=dev32(self.prefix), prefix_pages=None if self.shared is None else dev32(self.shared))

    def answer(self, rounding=1.0):
        """(outputs [T, Hq, 128] in 64 bits, how far each may be off).  What is rounded: a probability
        to fp16 or to two halves of a type (2^-11 of it at most); the middle of a group of Values to fp16
        (2^-11 of it, which is no more than the group's largest Value), a tail's or a node's Value times 2^-4
        at least to fp16 (exact, or off by half a step of the smallest numbers: 2^-25 * 2^4);
        for 8-bit boosted Keys step * code (2^-11); the fp32 sums of a score move it by less than 2^-19 of
        the sum of its products' magnitudes (8 chunks of 16 exact products, each sum cut off at 2^-23; on
        packed pages q . (step * code) and q . minimum are formed apart), so a weight by the
        exponential of that; and since the weights sum to 1,
          |out' - out| <= sum p (2^-11 + expm1(d)) |v - out| exp(max d) + 2^-11 sum p max|v| + 2^-21."""
        Hq, Hkv, g = self.Hq, self.Hkv, self.Hq // self.Hkv
        x = synth.from_bits(self.rows, self.dt).astype(np.float64)
        out = np.zeros((int(self.start[-1]), Hq, D))
        off = np.zeros_like(out)
        for b in range(self.B):
            lo, n = int(self.start[b]), self.counts[b]
            if n == 0:
                continue
            seen = sees(self.visible, self.start, b)
            for h in range(Hkv):
                k, v, part, size, most = self.cached(b, h)
                c = k.shape[0]
                k = np.concatenate([k, x[lo:lo + n, Hq + h]])
                v = np.concatenate([v, x[lo:lo + n, Hq + Hkv + h]])
                part = np.concatenate([part, np.zeros((n, D))])
                size = np.concatenate([size, np.abs(x[lo:lo + n, Hq + h])])
                most = np.concatenate([most, np.abs(x[lo:lo + n, Hq + Hkv + h])])
                q = x[lo:lo + n, h * g:(h + 1) * g].reshape(n * g, D)
                on = np.concatenate([np.ones((n, c), bool), seen], 1).repeat(g, 0)
                with np.errstate(invalid="ignore"):
                    k, v, part, size, most = (np.where(np.isfinite(y), y, 0.0) for y in (k, v, part, size, most))
                s = np.where(on, SM * (q @ k.T), -np.inf)
                m = s.max(1, initial=-np.inf, keepdims=True)
                p = np.where(on, np.exp(s - np.where(np.isfinite(m), m, 0)), 0.0)
                total = p.sum(1, keepdims=True)
                p = np.divide(p, total, out=np.zeros_like(p), where=total > 0)
                o = p @ v
                d = SM * (2.0 ** -19 * (np.abs(q) @ size.T) + 2.0 ** -11 * (np.abs(q) @ part.T))
                grow = np.exp(np.where(on, d, 0).max(1, initial=0.0))
                rows = slice(lo, lo + n), slice(h * g, (h + 1) * g)
                out[rows] = o.reshape(n, g, D)
                e = np.stack([((p[i] * (rounding * 2.0 ** -11 + np.expm1(d[i]))) @ np.abs(v - o[i])) * grow[i]
                              + rounding * 2.0 ** -11 * (p[i] @ most) + 2.0 ** -21 for i in range(n * g)])
                off[rows] = e.reshape(n, g, D)
        return out, off


class PackedTree(Base):
    """B sequences with own[b] pages and tails[b] tail tokens, behind n_prefix shared pages (shared[b]
    of them), and counts[b] drafted tokens."""

    def __init__(self, Hkv, Hq, dt, own, tails, counts, kind="tree", n_prefix=0, shared=None, seed=0, n_hi=32,
                 lo_bit=2, v_bit=2, pad=0, q_scale=1.0):
        import torch
        from mixed_precision_bit_gb300 import kitty
        r = np.random.default_rng(seed)
        self.size = kitty.tree_workspace_bytes
        self.B, self.Hkv, self.Hq, self.dt, self.n_prefix, self.shared = len(own), Hkv, Hq, dt, n_prefix, shared
        self.n_hi, self.lo_bit, self.v_bit = n_hi, lo_bit, v_bit
        self.cfg = kitty.Config(num_kv_heads=Hkv, num_q_heads=Hq, n_hi=n_hi, in_dtype=dt, hi_bit=2 * lo_bit,
                                lo_bit=lo_bit, v_bit=v_bit)
        self.own, self.tails = np.asarray(own), np.asarray(tails)
        total = n_prefix + int(self.own.sum())
        self.pool_pages = total + 1
        ids = r.permutation(total + 1)[:total].astype(np.int32)
        self.prefix = ids[:n_prefix].copy()
        self.max_pages = int(self.own.max()) + 1
        self.bt = np.full((self.B, self.max_pages), -1, np.int32)
        at = n_prefix
        for b in range(self.B):
            self.bt[b, :self.own[b]] = ids[at:at + self.own[b]]
            at += self.own[b]
        sigma = np.exp(r.standard_normal((Hkv, D)))
        self.pool = torch.zeros(self.pool_pages * kitty.page_bytes(self.cfg)[1], dtype=torch.uint8, device="cuda")
        if total:
            k = synth.to_bits(r.standard_normal((total * P, Hkv, D)) * sigma, dt)
            v = synth.to_bits(r.standard_normal((total * P, Hkv, D)), dt)
            kitty.quantize_pages(self.cfg, dev16(k), dev16(v), dev32(ids), self.pool, self.pool_pages)
        self.tail_k = synth.to_bits(r.standard_normal((self.B, Hkv, P, D)) * sigma[:, None], dt)
        self.tail_v = synth.to_bits(r.standard_normal((self.B, Hkv, P, D)), dt)
        self.put_cache()
        self._rows(r, counts, sigma, pad, visible_of(kind, r, counts, pad), q_scale)

    def put_cache(self):
        self.c = dict(bt=dev32(self.bt), own=dev32(self.own), tails=dev32(self.tails), tail_k=dev16(self.tail_k),
                      tail_v=dev16(self.tail_v))

    def call(self, out, status=None, ws=None, stream=None, max_nodes=None):
        from mixed_precision_bit_gb300 import kitty
        d, c = self.d, self.c
        kitty.tree_attention(self.cfg, d["q"], d["k"], d["v"], d["start"], d["visible"],
                             max_nodes or self.max_nodes(), self.pool, self.pool_pages, c["bt"], c["own"],
                             c["tail_k"], c["tail_v"], c["tails"], self.sm, out,
                             workspace=self.workspace() if ws is None else ws, status=status, stream=stream,
                             **self.prefix_args())

    def cached(self, b, h):
        """Keys, Values, of each Key the part that is rounded to fp16, the magnitudes whose products a
        score sums, and the largest Value of each Value's group, of what b holds."""
        if not hasattr(self, "_pages"):
            self._pages, self._blobs = {}, self.pool.cpu().numpy().reshape(self.pool_pages, self.Hkv, -1)
        ids = np.concatenate([self.prefix[:self.n_prefix if self.shared is None else self.shared[b]],
                              self.bt[b, :self.own[b]]])
        ks, vs, parts, sizes, mosts = ([np.zeros((0, D))] for _ in range(5))
        for pid in ids:
            if (pid, h) not in self._pages:
                blob = self._blobs[pid, h]
                k, v, _ = oracle.dequant_page(blob, self.n_hi, self.lo_bit, self.v_bit)
                part = np.zeros((P, D))
                if self.lo_bit == 4 and self.n_hi:
                    ch = np.asarray(oracle.page_channels(blob, self.n_hi, 4), int)
                    part[:, ch] = (k - k.min(0))[:, ch]
                # (the token of a channel's minimum has code 0)
                self._pages[pid, h] = (k, v, part, np.abs(k.min(0)) + (k - k.min(0)),
                                       np.abs(v).reshape(P, 4, 32).max(2).repeat(32, 1))
            for lst, y in zip((ks, vs, parts, sizes, mosts), self._pages[pid, h]):
                lst.append(y)
        n = self.tails[b]
        for lst, y in ((ks, self.tail_k), (vs, self.tail_v)):
            lst.append(synth.from_bits(y[b, h, :n], self.dt).astype(np.float64))
        parts.append(np.zeros((n, D)))
        sizes.append(np.abs(ks[-1]))
        mosts.append(np.abs(vs[-1]))
        return tuple(np.concatenate(x) for x in (ks, vs, parts, sizes, mosts))


class Plain16Tree(Base):
    """The same on 16-bit pages; lens[b] cached tokens.  What lies behind a sequence's last token in
    its last page is not a number."""

    def __init__(self, Hkv, Hq, dt, lens, counts, kind="tree", n_prefix=0, shared=None, seed=0, pad=0, q_scale=1.0):
        from mixed_precision_bit_gb300 import kitty
        r = np.random.default_rng(seed)
        self.size = kitty.f16kv_tree_workspace_bytes
        self.B, self.Hkv, self.Hq, self.dt, self.n_prefix, self.shared = len(lens), Hkv, Hq, dt, n_prefix, shared
        self.cfg = kitty.Config(num_kv_heads=Hkv, num_q_heads=Hq, in_dtype=dt)
        self.lens = np.asarray(lens)
        npg = (self.lens + P - 1) // P
        total = n_prefix + int(npg.sum())
        self.pool_pages = total + 1
        ids = r.permutation(self.pool_pages)[:total].astype(np.int32)
        self.prefix = ids[:n_prefix].copy()
        self.max_pages = int(npg.max()) + 1
        self.bt = np.full((self.B, self.max_pages), -1, np.int32)
        sigma = np.exp(r.standard_normal((Hkv, D)))
        self.host = np.zeros((self.pool_pages, Hkv, 2, P, D), np.uint16)
        self.host[:, :, 0] = synth.to_bits(r.standard_normal((self.pool_pages, Hkv, P, D)) * sigma[:, None], dt)
        self.host[:, :, 1] = synth.to_bits(r.standard_normal((self.pool_pages, Hkv, P, D)), dt)
        at = n_prefix
        for b in range(self.B):
            self.bt[b, :npg[b]] = ids[at:at + npg[b]]
            at += npg[b]
            if self.lens[b] % P:
                self.host[self.bt[b, npg[b] - 1], :, :, self.lens[b] % P:] = 0x7FFF  # NaN in both types
        self.put_cache()
        self._rows(r, counts, sigma, pad, visible_of(kind, r, counts, pad), q_scale)

    def put_cache(self):
        self.pool = dev16(self.host)
        self.c = dict(bt=dev32(self.bt), lens=dev32(self.lens))

    def call(self, out, status=None, ws=None, stream=None, max_nodes=None):
        from mixed_precision_bit_gb300 import kitty
        d, c = self.d, self.c
        kitty.f16kv_tree_attention(self.cfg, d["q"], d["k"], d["v"], d["start"], d["visible"],
                                   max_nodes or self.max_nodes(), self.pool, self.pool_pages, c["bt"], c["lens"],
                                   self.sm, out, workspace=self.workspace() if ws is None else ws, status=status,
                                   stream=stream, **self.prefix_args())

    def cached(self, b, h):
        n = int(self.lens[b])
        ids = np.concatenate([self.prefix[:self.n_prefix if self.shared is None else self.shared[b]],
                              self.bt[b, :(n + P - 1) // P]])
        x = synth.from_bits(self.host[ids, h], self.dt).astype(np.float64)  # [pages, 2, 32, 128]
        n += P * (len(ids) - (n + P - 1) // P)
        k, v = x[:, 0].reshape(-1, D)[:n], x[:, 1].reshape(-1, D)[:n]
        return k, v, np.zeros_like(k), np.abs(k), np.abs(v)


def half_step(x, out_dtype):
    return {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[out_dtype] * np.abs(x) + (2.0 ** -25 if out_dtype == "f16" else 0.0)


def check(c, out_dtype="f32", status=None, rows=None, **kw):
    """The call's outputs within the derived bounds of the plain answer."""
    got = c.run(out_dtype, status=status, **kw)
    ref, off = c.answer()
    bound = off + half_step(np.abs(ref) + off, out_dtype) + 1e-30
    bad = ~(np.abs(got - ref) <= bound)
    if rows is not None:
        bad = bad[rows]
    assert not bad.any(), "%d of %d off, by up to %.2f of the bound" % (
        bad.sum(), bad.size, np.nanmax(np.abs(got - ref) / bound))
    return got
