"""Layers that share one set of lengths: the first commit advances them, the later ones find them counted
already.  A sequence that the first one refuses keeps its tokens in every layer, byte for byte."""

import numpy as np
import pytest

from mixed_precision_bit_gb300 import synth
from tests.kitty_cases import dev16, dev32

pytestmark = pytest.mark.gpu
BF16 = synth.BF16
P, D, Hkv, Hq, M, B = 32, 128, 2, 4, 4, 3
CODES = dict(node=12, count=12, negative=12, page=4, full=8, length=5, starts=9)


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixed_precision_bit_gb300 import kitty
    kitty.load()


class Layer:
    """Pages, tails and statistics of one layer, of random bytes."""

    def __init__(self, packed, rank, seed):
        import torch
        from mixed_precision_bit_gb300 import kitty
        self.packed = packed
        self.cfg = kitty.Config(num_kv_heads=Hkv, num_q_heads=Hq, n_hi=16, in_dtype=BF16, rank_mode=rank)
        per_page = (kitty.page_bytes if packed else kitty.f16kv_page_bytes)(self.cfg)[1]
        g = torch.Generator("cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.pool = torch.randint(0, 256, (B * M * per_page,), generator=g, device="cuda", dtype=torch.uint8)
        self.tail_k, self.tail_v = (rand(B, Hkv, P, D).bfloat16() for _ in range(2))
        self.run = ((rand(B, Hkv, D), rand(B, Hkv, D).square(), torch.full((B, Hkv), P, dtype=torch.int32, device="cuda"))
                    if rank else (None, None, None))

    def commit(self, rows, start, path, n, bt, pages, tail, lens, counted, status):
        from mixed_precision_bit_gb300 import kitty
        k, v = rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
        if self.packed:
            kitty.tree_commit(self.cfg, k, v, start, path, n, self.tail_k, self.tail_v, tail, *self.run, bt, pages,
                              self.pool, B * M, counted=counted, status=status)
        else:
            kitty.f16kv_tree_commit(self.cfg, k, v, start, path, n, self.pool, B * M, bt, lens, counted=counted,
                                    status=status)

    def bytes(self):
        import torch
        parts = [self.pool] + ([self.tail_k, self.tail_v, *(x for x in self.run if x is not None)] if self.packed else [])
        return torch.cat([x.contiguous().view(torch.uint8).flatten() for x in parts])

    def of(self, b):
        """The bytes of sequence b: its own pages, tail and statistics."""
        import torch
        parts = [self.pool.view(B, -1)[b]]
        if self.packed:
            parts += [x[b].contiguous().view(torch.uint8).flatten() for x in (self.tail_k, self.tail_v, *self.run) if x is not None]
        return torch.cat(parts)


@pytest.mark.parametrize("fault", list(CODES))
@pytest.mark.parametrize("packed,rank", [(True, 0), (True, 1), (False, 0)], ids=["page", "running", "16"])
def test_a_refused_sequence_is_refused_in_every_layer(packed, rank, fault):
    import torch
    r = np.random.default_rng(7)
    start, n = np.array([0, 5, 10, 15], np.int32), np.array([3, 4, 5], np.int32)
    path = np.tile(np.arange(5, dtype=np.int32), (B, 1))
    bt = np.arange(B * M, dtype=np.int32).reshape(B, M)
    pages, tail, lens = np.array([1, 1, 1]), np.array([30, 30, 3]), np.array([62, 62, 35])
    if fault == "node":
        path[1, 2] = 5
    if fault == "count":
        n[1] = 6
    if fault == "negative":
        n[1] = -1
    if fault == "page":
        bt[1, 1] = -1 if packed else B * M
    if fault == "full":
        pages[1], lens[1] = 4, 126
    if fault == "length":
        pages[1], lens[1] = 5, 130
    if fault == "starts":
        start[2] = 4
    d = [dev32(x) for x in (start, path, n, bt, pages, tail, lens)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    rows = [dev16(synth.to_bits(r.standard_normal((15, Hq + 2 * Hkv, D)), BF16)) for _ in range(3)]
    layers, alike = ([Layer(packed, rank, s) for s in range(3)] for _ in range(2))
    before = [x.of(1).clone() for x in layers]
    for i, layer in enumerate(layers):
        layer.commit(rows[i], *d, counted=i > 0, status=status)
        assert int(status.item()) == CODES[fault] or (i > 0 and int(status.item()) == 0)
        status.zero_()
    # each as if it had lengths of its own and its commit advanced them
    for i, layer in enumerate(alike):
        own = [dev32(x) for x in (start, path, n, bt, pages, tail, lens)]
        layer.commit(rows[i], *own, counted=False, status=status)
        assert all(torch.equal(x, y) for x, y in zip(d[4:], own[4:]))
    for old, x, y in zip(before, layers, alike):
        assert torch.equal(x.of(1), old)
        assert torch.equal(x.bytes(), y.bytes())
    # what was appended of each, for the layers behind and for the caller
    assert d[2].cpu().tolist() == [3, 0, 5]
