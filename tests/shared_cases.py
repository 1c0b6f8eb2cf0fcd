"""A batch that shares a prefix, on both caches: inputs, the library's call and the oracle's
answer (its decode over each sequence's prefix pages followed by its own)."""

from __future__ import annotations

import math

import numpy as np

import oracle
from mixed_precision_bit_gb300 import synth
from tests.kitty_cases import dev16, dev32

P, D = 32, 128
SM = float(np.float32(1 / math.sqrt(D)))


def torch_type(dt):
    import torch
    return torch.bfloat16 if dt == synth.BF16 else torch.float16


class Packed:
    """B sequences behind n_prefix packed pages; own[b] pages and tails[b] tokens of their own."""

    sm = SM

    def __init__(self, Hkv, Hq, dt, n_prefix, shared, own, tails, seed=0, n_hi=32, lo_bit=2, v_bit=2,
                 spare=0, q_scale=1.0):
        import torch
        from mixed_precision_bit_gb300 import kitty
        r = np.random.default_rng(seed)
        B = len(own)
        self.B, self.Hkv, self.Hq, self.dt, self.n_prefix = B, Hkv, Hq, dt, n_prefix
        self.n_hi, self.lo_bit, self.v_bit = n_hi, lo_bit, v_bit
        self.cfg = kitty.Config(num_kv_heads=Hkv, num_q_heads=Hq, n_hi=n_hi, in_dtype=dt, hi_bit=2 * lo_bit,
                                lo_bit=lo_bit, v_bit=v_bit)
        self.shared = np.full(B, n_prefix) if shared is None else np.asarray(shared)
        self.prefix_pages = None if shared is None else np.asarray(shared, np.int32)
        self.own, self.tails = np.asarray(own), np.asarray(tails)
        total = n_prefix + int(self.own.sum())
        self.pool_pages = total + 1 + spare
        ids = (spare + r.permutation(total + 1))[:total].astype(np.int32)
        self.prefix = ids[:n_prefix].copy()
        self.max_pages = int(self.own.max()) if B else 0
        self.bt = np.full((B, self.max_pages), -1, np.int32)
        at = n_prefix
        for b in range(B):
            self.bt[b, :self.own[b]] = ids[at:at + self.own[b]]
            at += self.own[b]
        sigma = np.exp(r.standard_normal((Hkv, D)))
        self.pool = torch.zeros(self.pool_pages * kitty.page_bytes(self.cfg)[1], dtype=torch.uint8, device="cuda")
        self.k = synth.to_bits(r.standard_normal((total * P, Hkv, D)) * sigma, dt)
        self.v = synth.to_bits(r.standard_normal((total * P, Hkv, D)), dt)
        self.ids = ids
        if total:
            kitty.quantize_pages(self.cfg, dev16(self.k), dev16(self.v), dev32(ids), self.pool, self.pool_pages)
        self.tail_k = synth.to_bits(r.standard_normal((B, Hkv, P, D)) * sigma[:, None], dt)
        self.tail_v = synth.to_bits(r.standard_normal((B, Hkv, P, D)), dt)
        self.q = synth.to_bits(r.standard_normal((B, Hq, D)) * q_scale, dt)
        self.dev = dict(q=dev16(self.q), prefix=dev32(self.prefix), bt=dev32(self.bt), own=dev32(self.own),
                        tail_k=dev16(self.tail_k), tail_v=dev16(self.tail_v), tails=dev32(self.tails),
                        shared=None if shared is None else dev32(self.prefix_pages))

    def workspace(self):
        import torch
        from mixed_precision_bit_gb300 import kitty
        n = kitty.shared_workspace_bytes(self.cfg, self.B, self.n_prefix, self.max_pages)
        # partials of an earlier call must not matter
        return torch.full((max(n, 16) // 4,), float("nan"), dtype=torch.float32, device="cuda")

    def call(self, out, status=None, ws=None, stream=None):
        from mixed_precision_bit_gb300 import kitty
        d = self.dev
        kitty.decode_attention_shared(self.cfg, d["q"], self.pool, self.pool_pages, d["prefix"], d["shared"],
                                      d["bt"], d["own"], d["tail_k"], d["tail_v"], d["tails"], self.sm, out,
                                      workspace=self.workspace() if ws is None else ws, status=status,
                                      stream=stream)

    def run(self, out_dtype="f32", status=None):
        import torch
        t = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[out_dtype]
        out = torch.full((self.B, self.Hq, D), float("nan"), dtype=t, device="cuda")
        self.call(out, status)
        torch.cuda.synchronize()
        return out.float().cpu().numpy().astype(np.float64)

    def oracle(self, pool=None):
        pool = self.pool.cpu().numpy() if pool is None else pool
        n = self.shared + self.own
        bt = np.full((self.B, max(int(n.max()), 1)), -1, np.int32)
        for b in range(self.B):
            bt[b, :n[b]] = np.concatenate([self.prefix[:self.shared[b]], self.bt[b, :self.own[b]]])
        oracle.set_threads(8)
        return oracle.decode_attention(self.Hkv, self.Hq, self.n_hi, self.dt, self.q, pool, self.pool_pages, bt,
                                       n.astype(np.int32), self.tail_k, self.tail_v,
                                       self.tails.astype(np.int32), self.sm, lo_bit=self.lo_bit, v_bit=self.v_bit)


class Plain16:
    """The same on 16-bit pages; lens[b] own tokens."""

    sm = SM

    def __init__(self, Hkv, Hq, dt, n_prefix, shared, lens, seed=0, q_scale=1.0):
        import torch
        from mixed_precision_bit_gb300 import kitty
        r = np.random.default_rng(seed)
        B = len(lens)
        self.B, self.Hkv, self.Hq, self.dt, self.n_prefix = B, Hkv, Hq, dt, n_prefix
        self.cfg = kitty.Config(num_kv_heads=Hkv, num_q_heads=Hq, in_dtype=dt)
        self.shared = np.full(B, n_prefix) if shared is None else np.asarray(shared)
        self.lens = np.asarray(lens)
        npg = (self.lens + P - 1) // P
        total = n_prefix + int(npg.sum())
        self.pool_pages = total + 1
        ids = r.permutation(self.pool_pages)[:total].astype(np.int32)
        self.prefix = ids[:n_prefix].copy()
        self.max_pages = int(npg.max()) if B else 0
        self.bt = np.full((B, self.max_pages), -1, np.int32)
        at = n_prefix
        for b in range(B):
            self.bt[b, :npg[b]] = ids[at:at + npg[b]]
            at += npg[b]
        sigma = np.exp(r.standard_normal((Hkv, 1, D)))
        self.host = np.zeros((self.pool_pages, Hkv, 2, P, D), np.uint16)
        self.host[:, :, 0] = synth.to_bits(r.standard_normal((self.pool_pages, Hkv, P, D)) * sigma, dt)
        self.host[:, :, 1] = synth.to_bits(r.standard_normal((self.pool_pages, Hkv, P, D)), dt)
        self.q = synth.to_bits(r.standard_normal((B, Hq, D)) * q_scale, dt)
        self.pool = dev16(self.host)
        self.dev = dict(q=dev16(self.q), prefix=dev32(self.prefix), bt=dev32(self.bt), lens=dev32(self.lens),
                        shared=None if shared is None else dev32(self.shared))

    def workspace(self):
        import torch
        from mixed_precision_bit_gb300 import kitty
        n = kitty.f16kv_shared_workspace_bytes(self.cfg, self.B, self.n_prefix, self.max_pages)
        return torch.full((max(n, 16) // 4,), float("nan"), dtype=torch.float32, device="cuda")

    def call(self, out, status=None, ws=None, stream=None):
        from mixed_precision_bit_gb300 import kitty
        d = self.dev
        kitty.f16kv_decode_shared(self.cfg, d["q"], self.pool, self.pool_pages, d["prefix"], d["shared"], d["bt"],
                                  d["lens"], self.sm, out, workspace=self.workspace() if ws is None else ws,
                                  status=status, stream=stream)

    run = Packed.run

    def oracle(self):
        n = self.shared * P + self.lens
        bt = np.full((self.B, max(int((n.max() + P - 1) // P), 1)), -1, np.int32)
        for b in range(self.B):
            m = (self.lens[b] + P - 1) // P
            bt[b, :self.shared[b] + m] = np.concatenate([self.prefix[:self.shared[b]], self.bt[b, :m]])
        return oracle.decode_f16kv(self.Hkv, self.Hq, self.dt, self.q, self.host, self.pool_pages, bt,
                                   n.astype(np.int32), self.sm)
