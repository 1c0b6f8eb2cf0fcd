"""Paged Kitty KV cache state for a decode loop (the runtime around the kernels).

Per layer: a pool of packed pages, a block table, per-sequence unquantized
tails, running channel statistics and a host page allocator.  The host keeps a
mirror of every tail length and page count, so it decides flushes (which
sequences complete a 32-token page this step, and which physical page each one
gets) without reading device memory; the device state is only ever changed by
the library's kernels.  Paper: Abstract (page-centric layout, lightweight
runtime pipeline); VeloxQuant-MLX docs, Decode phase.

Beside the calls on rotated keys there are those from the projections (prefill_rope,
extend_rope, append_rope, step_rope: norms and rotation on the way), and a prefix that the
sequences share (share_prefix: its pages are stored once and attended once a call for the
whole batch).

Drafted tokens, chains or trees of them, are checked in one call (plan_trees, attend_tree) and
the accepted path is appended (reserve, commit_tree).  How many that are is known on the device
alone, so the page allocator moves there meanwhile (pages_to_device, pages_to_host): a step of
drafting needs nothing from the host and can be captured into a graph.
"""

from __future__ import annotations

import dataclasses
import math

import numpy as np
import torch

from . import kitty

PAGE = 32
D = 128


class _SharedPrefix:
    """Pages that the sequences of a layer's cache share: attended once for all of them, in
    front of each sequence's own.  What both caches keep of it."""

    prefix = None        # device int32 [n]: page ids of the shared prefix; None: there is none
    prefix_pages = None  # device int32 [B]: pages of it that each sequence sees; None: all
    pos_base = None      # device int32 [B]: positions ahead of a sequence's own tokens
    h_prefix = 0         # host mirror: pages that each sequence sees
    epoch = 0            # counts what a step captured before cannot follow: prefixes and clears

    def _prefix_plan(self, k_pages, v_pages, pages_of):
        """(pages of the prefix, pages of it that each sequence sees), checked."""
        self._host_plans()
        if self.prefix is not None:
            raise ValueError("the cache has a shared prefix (drop_prefix)")
        if self.kv_tokens():
            raise ValueError("the sequences hold tokens already (clear): their positions begin at the prefix's end")
        n = k_pages.shape[0] // PAGE
        rows = (n * PAGE, self.cfg.num_kv_heads, D)
        for t in (k_pages, v_pages):
            if t.shape != rows or t.element_size() != 2:
                raise ValueError("a prefix is 16-bit [pages * %d, %d, %d] (got %s, %s)"
                                 % (PAGE, *rows[1:], tuple(t.shape), t.dtype))
            kitty._same_type(t, self.cfg.in_dtype)
        pages = np.full(self.B, n, np.int32) if pages_of is None else np.asarray(pages_of, np.int32)
        if pages.shape != (self.B,) or (pages < 0).any() or (pages > n).any():
            raise ValueError("pages_of: one count in [0, %d] for each of %d sequences" % (n, self.B))
        return n, pages

    def _install_prefix(self, ids, pages, pages_of, write):
        """The prefix of these pages, once write(page ids on the device) has been accepted: a
        refusal leaves the cache without one, its pages free."""
        try:
            self._set_prefix(ids, pages, pages_of)
            if ids.size:
                write(self.prefix)
        except BaseException:
            self.prefix = self.prefix_pages = self.pos_base = None
            self.h_prefix = 0
            self.alloc.free(ids)
            raise
        self.epoch += 1

    def _set_prefix(self, ids, pages, pages_of):
        dev = self.pool.device
        self.prefix = torch.from_numpy(ids.astype(np.int32)).to(dev)
        self.prefix_pages = None if pages_of is None else torch.from_numpy(pages.copy()).to(dev)
        self.pos_base = torch.from_numpy(pages * PAGE).to(dev)
        self.h_prefix = pages.astype(np.int64)
        self._size_shared()

    def _size_shared(self):
        """A workspace for the shared call, grown when its plan needs more."""
        if self.prefix is None:
            return
        need = max(self._shared_bytes(self.cfg, self.B, self.prefix.numel(), self.max_pages), 16)
        self.shared_workspace = self._grown(self.shared_workspace, need)

    shared_workspace = None

    def _grown(self, ws, need):
        """A workspace of at least `need` bytes: ws, or a new one, of at least twice its size.
        The old one stays allocated as long as the cache, because a captured step writes its
        partials there; doubling keeps all of them together below twice the last one's size."""
        have = 0 if ws is None else ws.numel() * ws.element_size()
        if have >= need:
            return ws
        if ws is not None:
            self._outgrown = (*self._outgrown, ws)
        return torch.empty((max(need, 2 * have) + 3) // 4, dtype=torch.float32, device=self.pool.device)

    _outgrown = ()

    def drop_prefix(self):
        """Forget the shared prefix and give its pages back: between batches (clear), as the tokens
        of the sequences stand behind it.  Running statistics of the sequences that saw it start
        afresh.  Graphs captured with the prefix are not to be replayed any more."""
        self._host_plans()
        if self.prefix is not None:
            self.alloc.free(self.prefix.cpu().numpy())
            self._forget_statistics(self.h_prefix > 0)
            self.prefix = self.prefix_pages = self.pos_base = None
            self.h_prefix = 0
            self.epoch += 1

    def clear(self):
        """Empty the sequences, between batches: every page but the shared prefix's goes back to
        the allocator (those of a flush that was planned and not made, too), and lengths and
        running statistics start afresh, behind the prefix if there is one.  On the current
        stream."""
        self._host_plans()
        self.alloc.alloc(self.alloc.free_count)  # so that all pages are in use
        keep = [] if self.prefix is None else self.prefix.cpu().numpy()
        self.alloc.free(np.setdiff1d(np.arange(self.pool_pages), keep))
        self.block_table.fill_(-1)
        self._forget_tokens()
        self.epoch += 1

    def _forget_statistics(self, seqs):
        """Nothing to forget without running statistics."""

    def _prefix_tokens(self) -> int:
        return int(np.sum(self.h_prefix)) * PAGE

    def _prefix_bytes(self) -> int:
        """The prefix's pages and table, read once for the whole batch."""
        if self.prefix is None:
            return 0
        return self.prefix.numel() * (self.cfg.num_kv_heads * self.blob + 4)


class _DraftedTrees:
    """Trees of drafted tokens behind the sequences of a layer's cache, and the pages of their
    accepted ones.  What both caches keep of it: _device_lens (device lengths: num_pages or None,
    and tokens behind them), _partial (whether a last, partial page is one), _held_pages (of each
    sequence, by the host), _read_lens (host mirrors from the device's lengths), _mirrored (whether they
    are the same)."""

    free_ids = None    # device int32 [pool_pages]: a stack of free pages; None: the host plans
    free_count = None  # device int32 [1]: its height
    held = None        # device int32 [B]: pages in each row of the block table
    tree_workspace = None
    _on_device = None  # those three tensors, kept: captured steps use them after the next pages_to_device, too

    def _host_plans(self):
        if self.free_ids is not None:
            raise ValueError("the cache's pages are planned on the device (pages_to_host)")

    def pages_to_device(self):
        """Hand the free pages to the device: from now on reserve takes them, lengths change by
        commit_tree, and what the host plans (prefill, plan_flush, plan_extend, prefixes, clear)
        is refused, until pages_to_host.  Refused while an append is planned and not made, as in the
        layers of a ServingStep with graphs (cleared, or with graphs=False, they can be handed
        over).  On the current stream; synchronises."""
        self._host_plans()
        if not self._mirrored():
            raise ValueError("lengths on the device are not the host's: a planned append has not been made (a ServingStep "
                             "with graphs plans one step ahead: only clear() frees its layers)")
        if self._on_device is None:
            self._on_device = tuple(torch.empty(n, dtype=torch.int32, device=self.pool.device)
                                    for n in (self.pool_pages, 1, self.B))
        ids = np.full(self.pool_pages, -1, np.int32)
        n = self.alloc.free_count
        ids[:n] = self.alloc.alloc(n)[::-1]  # the stack's top is the page that the host would take
        for mine, value in zip(self._on_device, (ids, [n], self._held_pages())):
            mine.copy_(torch.from_numpy(np.asarray(value, np.int32)))
        self.free_ids, self.free_count, self.held = self._on_device

    def pages_to_host(self):
        """Give back what no token needs, and let the host plan again: synchronises."""
        if self.free_ids is None:
            raise ValueError("the cache's pages are planned on the host")
        self.reserve(0)
        self._read_lens()
        n = int(self.free_count.item())
        self.alloc.free(self.free_ids[:n].cpu().numpy())
        self.free_count.fill_(-1)  # a step captured before that is replayed now finds no stack: reported, no page taken
        self.free_ids = self.free_count = self.held = None

    def plan_trees(self, parents, seq_start, visible, positions, stream=None):
        """kitty.tree_plan behind this cache's tokens: which nodes each drafted token sees
        (visible) and where it stands (positions), from parents [n] and seq_start [B + 1]."""
        num_pages, lens = self._device_lens()
        kitty.tree_plan(parents, seq_start, lens, visible, positions, num_pages=num_pages,
                        pos_base=self.pos_base, status=self.status, stream=stream)

    def reserve(self, extra: int, stream=None):
        """Pages for `extra` more tokens of each sequence, as many as a path may be long and its row of
        the block table has room for, on the device; pages beyond them go back to the stack."""
        if self.free_ids is None:
            raise ValueError("the cache's pages are planned on the host (pages_to_device)")
        num_pages, lens = self._device_lens()
        kitty.page_tables(lens, self.held, self.block_table, self.free_ids, self.free_count,
                          num_pages=num_pages, extra=extra, partial=self._partial, shrink=True,
                          status=self.status, stream=stream)

    def _tree_call(self, q, max_nodes, sm_scale):
        """(scale, keywords) of a call for q [n, Hq, 128], with a workspace that its plan fits: the
        cache's own, so one call at a time."""
        need = self._tree_bytes(self.cfg, self.B, q.shape[0], max_nodes, self.max_pages,
                                0 if self.prefix is None else self.prefix.numel())
        self.tree_workspace = self._grown(self.tree_workspace, max(need, 16))
        sm = 1.0 / math.sqrt(D) if sm_scale is None else sm_scale
        return sm, dict(prefix_table=self.prefix, prefix_pages=self.prefix_pages,
                        workspace=self.tree_workspace, status=self.status)


class LayerCache(_DraftedTrees, _SharedPrefix):
    _shared_bytes = staticmethod(kitty.shared_workspace_bytes)
    _tree_bytes = staticmethod(kitty.tree_workspace_bytes)
    _partial = False  # what does not fill a page stands in the tail

    def __init__(self, cfg: kitty.Config, B: int, max_pages: int, pool_pages: int,
                 device="cuda"):
        self.cfg, self.B, self.max_pages, self.pool_pages = cfg, B, max_pages, pool_pages
        blob, per_page = kitty.page_bytes(cfg)
        self.blob, self.per_page = blob, per_page
        Hkv = cfg.num_kv_heads
        dev = torch.device(device)
        self.pool = torch.zeros(pool_pages * per_page, dtype=torch.uint8, device=dev)
        self.block_table = torch.full((B, max_pages), -1, dtype=torch.int32, device=dev)
        self.num_pages = torch.zeros(B, dtype=torch.int32, device=dev)
        self.tail_k = torch.zeros((B, Hkv, PAGE, D), dtype=torch.int16, device=dev)
        self.tail_v = torch.zeros_like(self.tail_k)
        self.tail_len = torch.zeros(B, dtype=torch.int32, device=dev)
        running = cfg.rank_mode != kitty.RANK_PAGE  # running or sequence-wide ranking
        self.run_sum = torch.zeros((B, Hkv, D), dtype=torch.float32, device=dev) if running else None
        self.run_sumsq = torch.zeros_like(self.run_sum) if running else None
        self.run_count = torch.zeros((B, Hkv), dtype=torch.int32, device=dev) if running else None
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.alloc = kitty.PageAllocator(pool_pages)
        self.h_tail = np.zeros(B, np.int64)
        self.h_pages = np.zeros(B, np.int64)
        ws = kitty.decode_workspace_bytes(cfg, B, max_pages)
        self.workspace = torch.empty(max(ws, 16) // 4, dtype=torch.float32, device=dev)

    # -- prefill: n_pages[b] full pages and a tail of tails[b] tokens per sequence
    def prefill(self, k_pages, v_pages, n_pages, k_tail=None, v_tail=None, tails=None,
                page_order=None, stream=None):
        """k_pages, v_pages: 16-bit tensors (int16 view) [sum(n_pages)*32, Hkv, D],
        sequence-major; k_tail, v_tail: [B, Hkv, 32, D] with tails[b] valid rows.
        page_order: optional permutation of the allocated ids (shuffled block table)."""
        self._host_plans()
        n_pages = np.asarray(n_pages, np.int64)
        tails = np.zeros(self.B, np.int64) if tails is None else np.asarray(tails, np.int64)
        tot = int(n_pages.sum())
        dev = self.pool.device
        ids = self.alloc.alloc(tot)
        if page_order is not None:
            ids = ids[np.asarray(page_order)]
        bt = np.full((self.B, self.max_pages), -1, np.int32)
        off = 0
        for b in range(self.B):
            bt[b, :n_pages[b]] = ids[off:off + n_pages[b]]
            off += n_pages[b]
        self.block_table.copy_(torch.from_numpy(bt))
        self.num_pages.copy_(torch.from_numpy(n_pages.astype(np.int32)))
        run = {}
        if self.run_sum is not None:
            seq = np.repeat(np.arange(self.B), n_pages).astype(np.int32)
            run = dict(seq_of_page=torch.from_numpy(seq).to(dev), n_seqs=self.B,
                       run_sum=self.run_sum, run_sumsq=self.run_sumsq, run_count=self.run_count)
        if tot:
            kitty.quantize_pages(self.cfg, k_pages, v_pages,
                                 torch.from_numpy(ids.astype(np.int32)).to(dev), self.pool,
                                 self.pool_pages, status=self.status, stream=stream, **run)
        if k_tail is not None:
            self.tail_k.copy_(k_tail)
            self.tail_v.copy_(v_tail)
        self.tail_len.copy_(torch.from_numpy(tails.astype(np.int32)))
        self.h_tail[:] = tails
        self.h_pages[:] = n_pages
        self.set_plan_hint()
        return ids

    def set_plan_hint(self, total_pages=None, max_pages=None):
        """Give the decode split planner the batch's total and largest page counts
        (default: the host mirror's) on this cache's own copy of the config, and
        grow the workspaces if that plan needs more.  Any values are correct;
        close ones balance the splits better.  Steps that were captured before keep
        their plan and their workspaces."""
        total = int(self.h_pages.sum()) if total_pages is None else int(total_pages)
        mx = int(self.h_pages.max()) if max_pages is None and self.B else int(max_pages or 0)
        self.cfg = dataclasses.replace(self.cfg, decode_total_pages=total, decode_max_pages=mx)
        self.workspace = self._grown(self.workspace,
                                     kitty.decode_workspace_bytes(self.cfg, self.B, self.max_pages))
        self._size_shared()

    def share_prefix(self, k_pages, v_pages, pages_of=None):
        """Quantize a prefix that the sequences share, once: k_pages, v_pages 16-bit
        [n * 32, Hkv, D], rotated as the sequences' own keys are (n full pages; a prompt's
        remainder is each sequence's own).  pages_of: how many of its pages each sequence sees
        (default: all); with running or sequence-wide ranking all or none of them, and those
        sequences' channel statistics go on from the prefix's.  Before the prefill or the first
        append of the sequences, on the current stream; returns the page ids.  Steps that were
        captured before do not attend it."""
        n, pages = self._prefix_plan(k_pages, v_pages, pages_of)
        dev, run = self.pool.device, {}
        if self.run_sum is not None:
            if not ((pages == 0) | (pages == n)).all():
                raise ValueError("running statistics: a sequence sees all of the prefix or none")
            one = (torch.zeros_like(self.run_sum[:1]), torch.zeros_like(self.run_sum[:1]),
                   torch.zeros_like(self.run_count[:1]))
            run = dict(seq_of_page=torch.zeros(n, dtype=torch.int32, device=dev), n_seqs=1,
                       run_sum=one[0], run_sumsq=one[1], run_count=one[2])
        ids = self.alloc.alloc(n)
        self._install_prefix(ids, pages, pages_of, lambda at: kitty.quantize_pages(
            self.cfg, k_pages, v_pages, at, self.pool, self.pool_pages, status=self.status, **run))
        if run:
            self._prefix_stats = one
            self._start_statistics()
        return ids

    _prefix_stats = None  # running statistics of the shared prefix: sums, sums of squares, counts

    def _stats(self):
        return () if self.run_sum is None else (self.run_sum, self.run_sumsq, self.run_count)

    def _start_statistics(self):
        """Statistics of sequences without tokens: the prefix's where they see it, else none."""
        for mine in self._stats():
            mine.zero_()
        if self.prefix is not None:
            sees = torch.from_numpy(np.nonzero(self.h_prefix)[0]).to(self.pool.device)
            for mine, theirs in zip(self._stats(), self._prefix_stats or ()):
                mine.index_copy_(0, sees, theirs.expand_as(mine)[:sees.numel()])

    def _forget_statistics(self, seqs):
        at = torch.from_numpy(np.nonzero(seqs)[0]).to(self.pool.device)
        for mine in self._stats():
            mine.index_fill_(0, at, 0)
        self._prefix_stats = None

    def _forget_tokens(self):
        self.num_pages.zero_()
        self.tail_len.zero_()
        self.h_tail[:] = 0
        self.h_pages[:] = 0
        self._start_statistics()
        self.set_plan_hint()

    def prefill_rope(self, rope: kitty.Rope, q, k, v, lens, q_out):
        """Prompts straight from the projections: q [T, Hq, D], k, v [T, Hkv, D] 16-bit (any
        token stride), lens[b] tokens of each sequence one after the other, behind the shared
        prefix if there is one.  Queries and keys are normed and rotated (kitty.norm_rope; the
        queries into q_out; q and q_out may be None), full pages quantized, the rest goes to the
        tails.  On the current stream."""
        lens = np.asarray(lens, np.int64)
        dev, T = self.pool.device, int(lens.sum())
        if lens.shape != (self.B,) or (lens < 0).any() or (lens // PAGE > self.max_pages).any():
            raise ValueError("lens: one length up to %d pages for each of %d sequences"
                             % (self.max_pages, self.B))
        if k.shape != (T, self.cfg.num_kv_heads, D) or v.shape != k.shape:
            raise ValueError("k, v: [%d, %d, %d] (got %s, %s)"
                             % (T, self.cfg.num_kv_heads, D, tuple(k.shape), tuple(v.shape)))
        if v.element_size() != 2:  # the binding checks the other rows
            raise ValueError("v: 16-bit values (got %s)" % v.dtype)
        kitty._same_type(v, self.cfg.in_dtype)
        start = np.concatenate([[0], np.cumsum(lens)])
        n_pages, tails = lens // PAGE, lens % PAGE
        pos = np.concatenate([np.arange(n) for n in lens]) if T else np.zeros(0)
        pos = pos + np.repeat(np.broadcast_to(np.asarray(self.h_prefix), self.B) * PAGE, lens)
        k_rot = torch.empty((T, self.cfg.num_kv_heads, D), dtype=k.dtype, device=dev)
        kitty.norm_rope(self.cfg, rope, q, k, torch.from_numpy(pos.astype(np.int32)).to(dev), q_out,
                        k_rot)
        full = [np.arange(start[b], start[b] + n_pages[b] * PAGE) for b in range(self.B)]
        sel = torch.from_numpy(np.concatenate(full).astype(np.int64)).to(dev)
        tail_k, tail_v = torch.zeros_like(self.tail_k), torch.zeros_like(self.tail_v)
        for b in np.nonzero(tails)[0]:
            rows = slice(int(start[b + 1] - tails[b]), int(start[b + 1]))
            for t, x in ((tail_k, k_rot), (tail_v, v)):
                t[b, :, :tails[b]] = x[rows].view(torch.int16).transpose(0, 1)
        return self.prefill(k_rot.index_select(0, sel), v.index_select(0, sel), n_pages, tail_k, tail_v,
                            tails)

    def plan_flush(self) -> np.ndarray:
        """Host decision for the next append: a fresh page id for each sequence whose
        tail completes a page, -1 elsewhere; advances the host mirror."""
        self._host_plans()
        fl = np.full(self.B, -1, np.int32)
        full = np.nonzero(self.h_tail + 1 == PAGE)[0]
        full = full[self.h_pages[full] < self.max_pages]
        if full.size:
            fl[full] = self.alloc.alloc(full.size)
        self.h_tail += 1
        self.h_tail[full] = 0
        self.h_pages[full] += 1
        return fl

    def step(self, k_new, v_new, flush_ids, q, out, sm_scale=None, stream=None):
        """append(k_new, v_new, flush_ids) then attend(q, out) as one fused launch
        (plus the split combine).  The fused call takes query groups of at most 4
        heads per kv head and no shared prefix; otherwise the two calls are made."""
        if self.prefix is not None or self.cfg.num_q_heads // self.cfg.num_kv_heads > 4:
            self.append(k_new, v_new, flush_ids, stream=stream)
            self.attend(q, out, sm_scale, stream=stream)
            return
        sm = 1.0 / math.sqrt(D) if sm_scale is None else sm_scale
        kitty.append_decode(self.cfg, k_new, v_new, q, self.tail_k, self.tail_v, self.tail_len,
                            self.run_sum, self.run_sumsq, self.run_count, flush_ids,
                            self.block_table, self.num_pages, self.pool, self.pool_pages, sm, out,
                            workspace=self.workspace, status=self.status, stream=stream)

    def capture_step(self, k_new, v_new, flush_ids, q, out, sm_scale=None):
        """A CUDA graph of one fused step(k_new, v_new, flush_ids, q, out) on these
        tensors: replaying it runs the call on what the tensors hold then, on the
        current stream.  Capturing runs nothing; the cache state changes only on
        replay."""
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self.step(k_new, v_new, flush_ids, q, out, sm_scale)
        return g

    def append(self, k_new, v_new, flush_ids, stream=None):
        kitty.append_token(self.cfg, k_new, v_new, self.tail_k, self.tail_v, self.tail_len,
                           self.run_sum, self.run_sumsq, self.run_count, flush_ids,
                           self.block_table, self.num_pages, self.pool, self.pool_pages,
                           status=self.status, stream=stream)

    def append_rope(self, rope: kitty.Rope, q, k_new, v_new, flush_ids, q_out, stream=None):
        """append from the projections: norms and rotation of q, k_new at each sequence's
        position (behind the shared prefix) on the way; the queries go to q_out."""
        kitty.append_rope(self.cfg, rope, q, k_new, v_new, q_out, self.tail_k, self.tail_v,
                          self.tail_len, self.run_sum, self.run_sumsq, self.run_count, flush_ids,
                          self.block_table, self.num_pages, self.pool, self.pool_pages,
                          pos_base=self.pos_base, status=self.status, stream=stream)

    def step_rope(self, rope: kitty.Rope, q, k_new, v_new, flush_ids, q_out, out, sm_scale=None,
                  stream=None):
        """append_rope, then attend with the rotated queries."""
        self.append_rope(rope, q, k_new, v_new, flush_ids, q_out, stream=stream)
        self.attend(q_out, out, sm_scale, stream=stream)

    def attend(self, q, out, sm_scale=None, stream=None):
        sm = 1.0 / math.sqrt(D) if sm_scale is None else sm_scale
        if self.prefix is not None:
            kitty.decode_attention_shared(self.cfg, q, self.pool, self.pool_pages, self.prefix,
                                          self.prefix_pages, self.block_table, self.num_pages,
                                          self.tail_k, self.tail_v, self.tail_len, sm, out,
                                          workspace=self.shared_workspace, status=self.status,
                                          stream=stream)
            return
        kitty.decode_attention(self.cfg, q, self.pool, self.pool_pages, self.block_table,
                               self.num_pages, self.tail_k, self.tail_v, self.tail_len, sm, out,
                               workspace=self.workspace, status=self.status, stream=stream)

    def attend_tree(self, q, k, v, seq_start, visible, max_nodes: int, out, sm_scale=None, stream=None):
        """Drafted tokens q [n, Hq, 128], rotated at their positions, attend to their sequences'
        tokens, the shared prefix among them, and to the drafted k, v [n, Hkv, 128] that they see
        (kitty.tree_attention).  Nothing is stored."""
        sm, more = self._tree_call(q, max_nodes, sm_scale)
        kitty.tree_attention(self.cfg, q, k, v, seq_start, visible, max_nodes, self.pool, self.pool_pages,
                             self.block_table, self.num_pages, self.tail_k, self.tail_v, self.tail_len,
                             sm, out, stream=stream, **more)

    def commit_tree(self, k, v, seq_start, path, path_len, stream=None):
        """Append each sequence's accepted drafted tokens, rows path[b, :path_len[b]] of its own in
        k, v (kitty.tree_commit), into pages that reserve has taken for them.  A sequence that has no
        room for its path is not appended to, and its path_len becomes 0."""
        if self.free_ids is None:
            raise ValueError("the cache's pages are planned on the host (pages_to_device)")
        kitty.tree_commit(self.cfg, k, v, seq_start, path, path_len, self.tail_k, self.tail_v, self.tail_len,
                          self.run_sum, self.run_sumsq, self.run_count, self.block_table, self.num_pages,
                          self.pool, self.pool_pages, status=self.status, stream=stream)

    def _device_lens(self):
        return self.num_pages, self.tail_len

    def _held_pages(self):
        return self.h_pages

    def _read_lens(self):
        self.h_pages[:] = self.num_pages.cpu().numpy()
        self.h_tail[:] = self.tail_len.cpu().numpy()

    def _mirrored(self):
        return (np.array_equal(self.h_pages, self.num_pages.cpu().numpy())
                and np.array_equal(self.h_tail, self.tail_len.cpu().numpy()))

    def append_bytes(self, flush_ids, fused: bool = False) -> int:
        """Bytes one append must move: the new K/V token read and written into the
        tail and, per flushed (sequence, kv head), the full tail read, the page blob
        written and the running statistics read and written.  fused: the flushed
        page is attended from on-chip memory, so the read of it that
        algorithmic_bytes counts is taken off here."""
        Hkv = self.cfg.num_kv_heads
        nf = int((np.asarray(flush_ids) >= 0).sum())
        stats = 2 * 2 * D * 4 + 2 * 4 if self.run_sum is not None else 0
        page = PAGE * D * 2 * 2 + self.blob + stats - (self.blob if fused else 0)
        return self.B * Hkv * D * 2 * 2 * 2 + nf * Hkv * page

    def kv_tokens(self) -> int:
        """Cached tokens one decode call attends to, over the batch (host mirror):
        full pages and unquantized tail tokens."""
        self._host_plans()
        return int(self.h_pages.sum()) * PAGE + int(self.h_tail.sum()) + self._prefix_tokens()

    def algorithmic_bytes(self) -> int:
        """Bytes one decode call must move: packed pages + tails + Q + O + block
        table entries (host mirror of the current lengths)."""
        self._host_plans()
        Hkv, Hq = self.cfg.num_kv_heads, self.cfg.num_q_heads
        pages = int(self.h_pages.sum())
        return (pages * Hkv * self.blob + int(self.h_tail.sum()) * Hkv * D * 2 * 2
                + self.B * Hq * D * 2 * 2 + pages * 4 + self._prefix_bytes())


class F16LayerCache(_DraftedTrees, _SharedPrefix):
    """The unquantized 16-bit paged KV cache of one layer (the paper's comparison
    layout for its same-budget claims, Abstract), with the same decode-loop
    interface as LayerCache: every token lives in a 32-token page (no tail), a
    token that starts a page gets a fresh page id from the host allocator, and
    the host mirrors every length."""

    _shared_bytes = staticmethod(kitty.f16kv_shared_workspace_bytes)
    _tree_bytes = staticmethod(kitty.f16kv_tree_workspace_bytes)
    _partial = True

    def __init__(self, cfg: kitty.Config, B: int, max_pages: int, pool_pages: int,
                 device="cuda"):
        self.cfg, self.B, self.max_pages, self.pool_pages = cfg, B, max_pages, pool_pages
        blob, per_page = kitty.f16kv_page_bytes(cfg)
        self.blob, self.per_page = blob, per_page
        dev = torch.device(device)
        self.pool = torch.zeros(pool_pages * per_page, dtype=torch.uint8, device=dev)
        self.block_table = torch.full((B, max_pages), -1, dtype=torch.int32, device=dev)
        self.ctx_len = torch.zeros(B, dtype=torch.int32, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.alloc = kitty.PageAllocator(pool_pages)
        self.h_len = np.zeros(B, np.int64)
        ws = kitty.f16kv_workspace_bytes(cfg, B, max_pages)
        self.workspace = torch.empty(max(ws, 16) // 4, dtype=torch.float32, device=dev)

    def prefill(self, k_pages, v_pages, n_pages, k_tail=None, v_tail=None, tails=None,
                page_order=None, stream=None):
        """As LayerCache.prefill: n_pages[b] full pages (k_pages, v_pages 16-bit
        [sum(n_pages)*32, Hkv, D], sequence-major) and tails[b] more tokens
        (k_tail, v_tail [B, Hkv, 32, D]), which go to a last, partial page."""
        self._host_plans()
        n_pages = np.asarray(n_pages, np.int64)
        tails = np.zeros(self.B, np.int64) if tails is None else np.asarray(tails, np.int64)
        tot = int(n_pages.sum())
        dev = self.pool.device
        ids = self.alloc.alloc(tot)
        if page_order is not None:
            ids = ids[np.asarray(page_order)]
        with_tail = np.nonzero(tails > 0)[0]
        tail_ids = self.alloc.alloc(with_tail.size) if with_tail.size else np.zeros(0, np.int32)
        bt = np.full((self.B, self.max_pages), -1, np.int32)
        off = 0
        for b in range(self.B):
            bt[b, :n_pages[b]] = ids[off:off + n_pages[b]]
            off += n_pages[b]
        for i, b in enumerate(with_tail):
            bt[b, n_pages[b]] = tail_ids[i]
        self.block_table.copy_(torch.from_numpy(bt))
        if tot:
            kitty.f16kv_write_pages(self.cfg, k_pages, v_pages,
                                    torch.from_numpy(ids.astype(np.int32)).to(dev), self.pool,
                                    self.pool_pages, status=self.status, stream=stream)
        if with_tail.size:
            sel = torch.from_numpy(with_tail).to(dev)
            kt = k_tail.index_select(0, sel).transpose(1, 2).contiguous()  # [n, 32, Hkv, D]
            vt = v_tail.index_select(0, sel).transpose(1, 2).contiguous()
            kitty.f16kv_write_pages(self.cfg, kt, vt,
                                    torch.from_numpy(tail_ids.astype(np.int32)).to(dev),
                                    self.pool, self.pool_pages, status=self.status, stream=stream)
        self.h_len[:] = n_pages * PAGE + tails
        self.ctx_len.copy_(torch.from_numpy(self.h_len.astype(np.int32)))
        return ids

    def plan_flush(self) -> np.ndarray:
        """Host decision for the next append: a fresh page id for each sequence whose
        next token starts a page, -1 elsewhere; advances the host mirror."""
        self._host_plans()
        fl = np.full(self.B, -1, np.int32)
        new = np.nonzero(self.h_len % PAGE == 0)[0]
        new = new[self.h_len[new] // PAGE < self.max_pages]
        if new.size:
            fl[new] = self.alloc.alloc(new.size)
        self.h_len += 1
        return fl

    def share_prefix(self, k_pages, v_pages, pages_of=None):
        """As LayerCache.share_prefix (any pages_of)."""
        n, pages = self._prefix_plan(k_pages, v_pages, pages_of)
        ids = self.alloc.alloc(n)
        self._install_prefix(ids, pages, pages_of, lambda at: kitty.f16kv_write_pages(
            self.cfg, k_pages, v_pages, at, self.pool, self.pool_pages, status=self.status))
        return ids

    def plan_extend(self, lens):
        """Host decision for appending lens[b] tokens to each sequence: (new_page_ids [T],
        seq_start [B + 1]), a fresh page id at every token that begins a page; advances the
        host mirror."""
        self._host_plans()
        lens = np.asarray(lens, np.int64)
        if lens.shape != (self.B,) or (lens < 0).any():
            raise ValueError("lens: one length for each of %d sequences" % self.B)
        if ((self.h_len + lens) > self.max_pages * PAGE).any():
            raise ValueError("a sequence has no room for its new tokens")
        start = np.concatenate([[0], np.cumsum(lens)])
        ids = np.full(int(start[-1]), -1, np.int32)
        at = np.concatenate([np.arange(start[b] + (-self.h_len[b]) % PAGE, start[b + 1], PAGE)
                             for b in range(self.B)]).astype(np.int64)
        ids[at] = self.alloc.alloc(at.size)
        self.h_len += lens
        return ids, start.astype(np.int32)

    def extend_rope(self, rope: kitty.Rope, q, k, v, lens, q_out):
        """Append lens[b] tokens to each sequence (prompts, or parts of them) from the projections
        q [T, Hq, D], k, v [T, Hkv, D], normed and rotated at their positions (behind the shared
        prefix) on the way into the pages; the queries go to q_out (q and q_out may be None).
        On the current stream."""
        T, Hq, Hkv = int(np.sum(lens)), self.cfg.num_q_heads, self.cfg.num_kv_heads
        for x, heads in ((q, Hq), (q_out, Hq), (k, Hkv), (v, Hkv)):  # before pages are taken
            if x is not None and x.shape != (T, heads, D):
                raise ValueError("expected rows [%d, %d, %d] (got %s)" % (T, heads, D, tuple(x.shape)))
        plan = self.plan_extend(lens)
        try:
            ids, start = (torch.from_numpy(x).to(self.pool.device) for x in plan)
            kitty.f16kv_append_rope(self.cfg, rope, q, k, v, q_out, self.pool, self.pool_pages,
                                    self.block_table, self.ctx_len, ids, seq_start=start,
                                    pos_base=self.pos_base, status=self.status)
        except BaseException:  # nothing was appended: the plan is taken back
            self.alloc.free(plan[0][plan[0] >= 0])
            self.h_len -= np.asarray(lens, np.int64)
            raise

    def _forget_tokens(self):
        self.ctx_len.zero_()
        self.h_len[:] = 0

    def append_rope(self, rope: kitty.Rope, q, k_new, v_new, new_page_ids, q_out, stream=None):
        """append from the projections, as LayerCache.append_rope."""
        kitty.f16kv_append_rope(self.cfg, rope, q, k_new, v_new, q_out, self.pool, self.pool_pages,
                                self.block_table, self.ctx_len, new_page_ids, pos_base=self.pos_base,
                                status=self.status, stream=stream)

    def step_rope(self, rope: kitty.Rope, q, k_new, v_new, new_page_ids, q_out, out, sm_scale=None,
                  stream=None):
        """append_rope, then attend with the rotated queries."""
        self.append_rope(rope, q, k_new, v_new, new_page_ids, q_out, stream=stream)
        self.attend(q_out, out, sm_scale, stream=stream)

    def append(self, k_new, v_new, new_page_ids, stream=None):
        kitty.f16kv_append(self.cfg, k_new, v_new, self.pool, self.pool_pages, self.block_table,
                           self.ctx_len, new_page_ids, status=self.status, stream=stream)

    def attend(self, q, out, sm_scale=None, stream=None):
        sm = 1.0 / math.sqrt(D) if sm_scale is None else sm_scale
        if self.prefix is not None:
            kitty.f16kv_decode_shared(self.cfg, q, self.pool, self.pool_pages, self.prefix,
                                      self.prefix_pages, self.block_table, self.ctx_len, sm, out,
                                      workspace=self.shared_workspace, status=self.status,
                                      stream=stream)
            return
        kitty.f16kv_decode(self.cfg, q, self.pool, self.pool_pages, self.block_table,
                           self.ctx_len, sm, out, workspace=self.workspace, status=self.status,
                           stream=stream)

    def step(self, k_new, v_new, new_page_ids, q, out, sm_scale=None, stream=None):
        """append then attend (the append's two kernels, the decode and its combine)."""
        self.append(k_new, v_new, new_page_ids, stream=stream)
        self.attend(q, out, sm_scale, stream=stream)

    def attend_tree(self, q, k, v, seq_start, visible, max_nodes: int, out, sm_scale=None, stream=None):
        """As LayerCache.attend_tree."""
        sm, more = self._tree_call(q, max_nodes, sm_scale)
        kitty.f16kv_tree_attention(self.cfg, q, k, v, seq_start, visible, max_nodes, self.pool,
                                   self.pool_pages, self.block_table, self.ctx_len, sm, out,
                                   stream=stream, **more)

    def commit_tree(self, k, v, seq_start, path, path_len, stream=None):
        """As LayerCache.commit_tree."""
        if self.free_ids is None:
            raise ValueError("the cache's pages are planned on the host (pages_to_device)")
        kitty.f16kv_tree_commit(self.cfg, k, v, seq_start, path, path_len, self.pool, self.pool_pages,
                                self.block_table, self.ctx_len, status=self.status, stream=stream)

    def _device_lens(self):
        return None, self.ctx_len

    def _held_pages(self):
        return (self.h_len + PAGE - 1) // PAGE

    def _read_lens(self):
        self.h_len[:] = self.ctx_len.cpu().numpy()

    def _mirrored(self):
        return np.array_equal(self.h_len, self.ctx_len.cpu().numpy())

    def append_bytes(self, new_page_ids, fused: bool = False) -> int:
        """The new K/V token read and written into its page."""
        return self.B * self.cfg.num_kv_heads * D * 2 * 2 * 2

    def kv_tokens(self) -> int:
        self._host_plans()
        return int(self.h_len.sum()) + self._prefix_tokens()

    def algorithmic_bytes(self) -> int:
        """Bytes one decode call must move: the K and V rows of every cached token,
        Q, O and the block-table entries (host mirror of the lengths)."""
        self._host_plans()
        Hkv, Hq = self.cfg.num_kv_heads, self.cfg.num_q_heads
        pages = int(((self.h_len + PAGE - 1) // PAGE).sum())
        return (int(self.h_len.sum()) * Hkv * D * 2 * 2 + self.B * Hq * D * 2 * 2 + pages * 4
                + self._prefix_bytes())


def capture_layers_step(layers, k_new, v_new, flush_ids, q, out, sm_scale=None,
                        fused: bool = True):
    """One CUDA graph of a decode step over every layer: per layer l in order, the
    fused step(k_new[l], v_new[l], flush_ids[l], q[l], out[l]) (fused=False:
    append then attend).  Each argument is indexed by layer (a list, or a tensor
    with a leading layer dimension).  The layers' kernels run back to back inside
    one graph, so a step costs one graph launch instead of one per layer.
    Capturing runs nothing; replaying runs the calls on what the tensors hold then,
    on the current stream."""
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for l, lc in enumerate(layers):
            if fused:
                lc.step(k_new[l], v_new[l], flush_ids[l], q[l], out[l], sm_scale)
            else:
                lc.append(k_new[l], v_new[l], flush_ids[l])
                lc.attend(q[l], out[l], sm_scale)
    return g


class ServingStep:
    """One decode step of every layer from pinned host memory, with the copies
    overlapped with the kernels.

    Per layer, the query rows and the new Key/Value token sit in one contiguous
    pinned block (views: q[l], k_new[l], v_new[l]; the caller writes them before
    run()), copied up with one transfer on an upload stream; the layer's call
    waits only for its own block, and its output comes back on a download stream
    while later layers compute.  run() returns once every output is in `out`
    (pinned host, [L][B][Hq][D]).

    graphs=True: the whole step (uploads, every layer's call, downloads) is one
    CUDA graph, so a step costs one graph launch.  The flush ids of the next
    step are planned on the host while the graph of this one runs (the host
    mirrors of the layers run one step ahead between calls); two graphs read
    the plans from alternating pinned buffers.  Between run() calls the layers
    must not be driven by other calls, nor their pages handed to the device; a
    layer whose prefix has changed, or that was cleared, since the graphs were
    captured is refused (they attend what it had then).
    graphs=False: direct calls; the flush plan of layer l is made just before
    its block goes up, so planning overlaps the kernels of the layers before it.
    fused=False runs append then attend per layer.
    """

    def __init__(self, layers, graphs: bool = True, fused: bool = True, sm_scale=None):
        self.layers = layers
        lc0 = layers[0]
        L, B = len(layers), lc0.B
        Hq, Hkv = lc0.cfg.num_q_heads, lc0.cfg.num_kv_heads
        dev = lc0.pool.device
        self.sizes = [B * Hq * D * 2, B * Hkv * D * 2, B * Hkv * D * 2, B * 4]
        per = sum(self.sizes)
        self.block = (per + 255) // 256 * 256  # 256-byte aligned per-layer blocks
        self.h_in = torch.empty(L * self.block, dtype=torch.uint8).pin_memory()
        self.d_in = torch.empty(L * self.block, dtype=torch.uint8, device=dev)
        self.q, self.k_new, self.v_new, self.flush = [], [], [], []
        self._dq, self._dk, self._dv, self._dfl = [], [], [], []
        for l in range(L):
            hv_, dv_ = self._views(self.h_in, l, B, Hq, Hkv), self._views(self.d_in, l, B, Hq, Hkv)
            for lst, x in zip((self.q, self.k_new, self.v_new, self.flush), hv_):
                lst.append(x)
            for lst, x in zip((self._dq, self._dk, self._dv, self._dfl), dv_):
                lst.append(x)
        out_dt = torch.bfloat16 if lc0.cfg.in_dtype == kitty.BF16 else torch.float16
        self.d_out = torch.empty((L, B, Hq, D), dtype=out_dt, device=dev)
        self.out = torch.empty((L, B, Hq, D), dtype=out_dt).pin_memory()
        self.up, self.down = torch.cuda.Stream(dev), torch.cuda.Stream(dev)
        self.ev_in = [torch.cuda.Event() for _ in range(L)]
        self.ev_out = [torch.cuda.Event() for _ in range(L)]
        self.fused, self.sm_scale = fused, sm_scale
        self.graphs = None
        if graphs:
            # flush plans of two consecutive steps, and their device copy
            self.h_fl = [torch.empty((L, B), dtype=torch.int32).pin_memory() for _ in range(2)]
            self.d_fl = torch.empty((L, B), dtype=torch.int32, device=dev)
            self.graphs = [self._capture(p) for p in range(2)]
            self._epochs = [lc.epoch for lc in layers]
            self._parity = 0
            self._planned = 0  # layers whose flushes of the pending step are planned

    def _views(self, buf, l, B, Hq, Hkv):
        o = l * self.block
        s = self.sizes
        q = buf[o:o + s[0]].view(torch.int16).view(B, Hq, D)
        k = buf[o + s[0]:o + s[0] + s[1]].view(torch.int16).view(B, Hkv, D)
        v = buf[o + s[0] + s[1]:o + s[0] + s[1] + s[2]].view(torch.int16).view(B, Hkv, D)
        f = buf[o + s[0] + s[1] + s[2]:o + s[0] + s[1] + s[2] + s[3]].view(torch.int32)
        return q, k, v, f

    def _call(self, l, flush_ids):
        lc = self.layers[l]
        if self.fused:
            lc.step(self._dk[l], self._dv[l], flush_ids, self._dq[l], self.d_out[l], self.sm_scale)
        else:
            lc.append(self._dk[l], self._dv[l], flush_ids)
            lc.attend(self._dq[l], self.d_out[l], self.sm_scale)

    def _capture(self, parity):
        """The graph of one step reading its flush plan from h_fl[parity]."""
        qkv = sum(self.sizes[:3])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            cap = torch.cuda.current_stream()
            self.up.wait_stream(cap)
            self.down.wait_stream(cap)
            with torch.cuda.stream(self.up):
                self.d_fl.copy_(self.h_fl[parity], non_blocking=True)
                for l in range(len(self.layers)):
                    o = l * self.block
                    self.d_in[o:o + qkv].copy_(self.h_in[o:o + qkv], non_blocking=True)
                    self.ev_in[l].record(self.up)
            for l in range(len(self.layers)):
                cap.wait_event(self.ev_in[l])
                self._call(l, self.d_fl[l])
                self.ev_out[l].record(cap)
                with torch.cuda.stream(self.down):
                    self.down.wait_event(self.ev_out[l])
                    self.out[l].copy_(self.d_out[l], non_blocking=True)
            cap.wait_stream(self.down)
        return g

    def _plan(self, parity):
        """Plans the pending step's flushes into h_fl[parity], from the first layer
        not yet planned: a layer whose page allocation fails raises, and the next
        call resumes at that layer."""
        fl = self.h_fl[parity].numpy()
        while self._planned < len(self.layers):
            fl[self._planned] = self.layers[self._planned].plan_flush()
            self._planned += 1

    def bytes_up(self) -> int:
        return len(self.layers) * sum(self.sizes)

    def bytes_down(self) -> int:
        return self.out.numel() * self.out.element_size()

    def run(self):
        cur = torch.cuda.current_stream()
        if self.graphs is not None:
            for l, lc in enumerate(self.layers):
                if lc.epoch != self._epochs[l]:
                    raise ValueError("layer %d was cleared, or its shared prefix changed, after the step was "
                                     "captured: make a new ServingStep" % l)
            self._plan(self._parity)  # nothing left to do unless the look-ahead stopped
            self.graphs[self._parity].replay()
            self._parity ^= 1
            self._planned = 0
            try:
                self._plan(self._parity)  # the next step's flushes, while this one runs
            except kitty.KittyError:
                pass  # e.g. the pool is full: raised by the next run(), before its step
            cur.synchronize()
            return self.out
        # the device input blocks and outputs may still be in use by work queued
        # before this call
        self.up.wait_stream(cur)
        self.down.wait_stream(cur)
        for l, lc in enumerate(self.layers):
            self.flush[l].numpy()[:] = lc.plan_flush()
            o = l * self.block
            with torch.cuda.stream(self.up):
                self.d_in[o:o + self.block].copy_(self.h_in[o:o + self.block], non_blocking=True)
                self.ev_in[l].record(self.up)
            cur.wait_event(self.ev_in[l])
            self._call(l, self._dfl[l])
            self.ev_out[l].record(cur)
            with torch.cuda.stream(self.down):
                self.down.wait_event(self.ev_out[l])
                self.out[l].copy_(self.d_out[l], non_blocking=True)
        self.down.synchronize()
        return self.out
