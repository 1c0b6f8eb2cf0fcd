"""A cache that is used for one batch after another: what an earlier shared prefix or batch left
does not show in the next, byte for byte against a fresh cache, with every ranking."""

import numpy as np
import pytest

import oracle
from mixed_precision_bit_gb300 import synth
from tests.kitty_cases import dev16

pytestmark = pytest.mark.gpu
P, D, B, Hkv, Hq, M = 32, 128, 3, 2, 8, 6
OWN = np.array([3, 0, 2])
DT = synth.BF16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixed_precision_bit_gb300 import kitty
    kitty.load()


def _rows(n, seed):
    """Keys whose large channels differ from one seed to the next, and Values."""
    r = np.random.default_rng(seed)
    sigma = np.exp(1.5 * r.standard_normal((Hkv, D)))
    return (synth.to_bits(r.standard_normal((n * P, Hkv, D)) * sigma, DT),
            synth.to_bits(r.standard_normal((n * P, Hkv, D)), DT))


def _cache(rank):
    from mixed_precision_bit_gb300 import kitty
    from mixed_precision_bit_gb300.cache import LayerCache
    cfg = kitty.Config(num_kv_heads=Hkv, num_q_heads=Hq, in_dtype=DT, rank_mode=rank, n_hi=32)
    return LayerCache(cfg, B, M, 4 + B * M)


def _share(lc, n, seed, pages_of=None):
    lc.share_prefix(*(dev16(x) for x in _rows(n, seed)), pages_of=pages_of)


def _prefill(lc, seed):
    """Full pages, a tail one short of one, and the step that fills it."""
    import torch
    k, v = _rows(int(OWN.sum()), seed)
    tail = torch.from_numpy(np.stack(_rows(B, seed + 1)).view(np.int16)).cuda().view(2, B, P, Hkv, D).transpose(2, 3)
    lc.prefill(dev16(k), dev16(v), OWN, tail[0].contiguous(), tail[1].contiguous(), np.full(B, 31))
    new = _rows(1, seed + 2)
    lc.append(*(dev16(x[:B]) for x in new), torch.from_numpy(lc.plan_flush()).cuda())


def _stats(lc):
    return () if lc.run_sum is None else (lc.run_sum, lc.run_sumsq, lc.run_count)


def _same(a, c):
    """The same sequences' pages, tails, lengths and statistics, wherever the pages are."""
    import torch
    assert torch.equal(a.num_pages, c.num_pages) and torch.equal(a.tail_len, c.tail_len)
    assert torch.equal(a.num_pages.cpu(), torch.from_numpy(OWN + 1).int())
    pa, pc = (x.pool.view(x.pool_pages, -1) for x in (a, c))
    for b in range(B):
        n = int(a.num_pages[b])
        assert torch.equal(pa[a.block_table[b, :n].long()], pc[c.block_table[b, :n].long()]), b
    assert (a.prefix is None) == (c.prefix is None)
    if a.prefix is not None:
        assert torch.equal(pa[a.prefix.long()], pc[c.prefix.long()])
    for x, y in zip(_stats(a), _stats(c)):
        assert torch.equal(x, y)
    assert int(a.status.item()) == int(c.status.item()) == 0
    assert a.alloc.free_count == c.alloc.free_count and a.kv_tokens() == c.kv_tokens()


@pytest.mark.parametrize("rank", [0, 1, 2], ids=["page", "running", "sequence"])
def test_a_dropped_prefix_leaves_nothing(rank):
    a, c = _cache(rank), _cache(rank)
    _share(a, 4, 1)
    a.drop_prefix()
    _prefill(a, 10)
    _prefill(c, 10)
    _same(a, c)


@pytest.mark.parametrize("rank", [0, 1, 2], ids=["page", "running", "sequence"])
def test_another_prefix_that_some_do_not_see(rank):
    a, c = _cache(rank), _cache(rank)
    _share(a, 4, 1)
    a.drop_prefix()
    for lc in (a, c):
        _share(lc, 3, 2, [3, 0, 0])
        _prefill(lc, 10)
    _same(a, c)


@pytest.mark.parametrize("rank", [0, 1, 2], ids=["page", "running", "sequence"])
def test_the_next_batch_behind_the_same_prefix(rank):
    a, c = _cache(rank), _cache(rank)
    for lc in (a, c):
        _share(lc, 4, 1, [4, 0, 4])
    _prefill(a, 20)
    a.clear()
    for lc in (a, c):
        _prefill(lc, 10)
    _same(a, c)
    # without the prefix
    a.clear()
    a.drop_prefix()
    c = _cache(rank)
    for lc in (a, c):
        _prefill(lc, 30)
    _same(a, c)


@pytest.mark.parametrize("rank", [0, 1, 2], ids=["page", "running", "sequence"])
def test_prefix_pages_and_what_follows_them_against_the_oracle(rank):
    """The prefix ranked as a sequence of its own; the sequences that see it go on from its
    statistics, with one set of channels over their own prompt when the ranking is over sequences."""
    import torch
    lc = _cache(rank)
    sees = np.array([4, 0, 4])
    _share(lc, 4, 1, sees)
    stats = [np.zeros((B, Hkv, D), np.float32), np.zeros((B, Hkv, D), np.float32), np.zeros((B, Hkv), np.int32)]
    one = [np.zeros((1,) + x.shape[1:], x.dtype) for x in stats]
    pool = np.zeros(lc.pool.numel(), np.uint8)
    ids = lc.prefix.cpu().numpy()
    args = (Hkv, 32, rank, DT)
    run = lambda seq, s: dict(seq_of_page=seq, n_seqs=len(s[2]), run_sum=s[0], run_sumsq=s[1], run_count=s[2]) if rank else {}  # noqa: E731
    k, v = _rows(4, 1)
    assert oracle.quantize_pages(*args, k, v, ids, pool, lc.pool_pages, **run(np.zeros(4, np.int32), one)) == 0
    for x, y in zip(stats, one):
        x[sees > 0] = y
    k, v = _rows(int(OWN.sum()), 10)
    own = lc.prefill(dev16(k), dev16(v), OWN)
    seq = np.repeat(np.arange(B), OWN).astype(np.int32)
    assert oracle.quantize_pages(*args, k, v, own.astype(np.int32), pool, lc.pool_pages, **run(seq, stats)) == 0
    assert np.array_equal(lc.pool.cpu().numpy(), pool)
    for x, y in zip(_stats(lc), stats):
        assert np.array_equal(x.cpu().numpy(), y)
    assert int(lc.status.item()) == 0


@pytest.mark.parametrize("prefix", [False, True], ids=["own", "shared"])
def test_a_captured_step_keeps_its_workspace(prefix):
    """Replayed after hints that grew the workspaces, with other tensors allocated since: the
    bytes of the first replay, and the other tensors untouched."""
    import torch
    from mixed_precision_bit_gb300 import kitty
    from mixed_precision_bit_gb300.cache import LayerCache
    cfg = kitty.Config(num_kv_heads=Hkv, num_q_heads=Hq, in_dtype=DT, n_hi=32)
    lc = LayerCache(cfg, B, 400, 20)
    if prefix:
        _share(lc, 4, 1)
    _prefill(lc, 10)
    q = torch.randn(B, Hq, D, device="cuda").bfloat16()
    out = torch.empty(B, Hq, D, device="cuda")
    lc.attend(q, out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lc.attend(q, out)
    g.replay()
    first = out.clone()
    held = (lc.workspace, lc.shared_workspace)
    addresses = [w.data_ptr() for w in held if w is not None]
    del held
    lc.set_plan_hint(1200, 400)
    assert addresses != [w.data_ptr() for w in (lc.workspace, lc.shared_workspace) if w is not None]
    others = [torch.full((n,), 7.0, device="cuda") for n in (1 << 8, 1 << 12, 1 << 14, 1 << 16, 1 << 18) for _ in range(8)]
    for o in others:
        assert not any(o.data_ptr() <= a < o.data_ptr() + 4 * o.numel() for a in addresses)
    for _ in range(3):
        out.zero_()
        g.replay()
        assert torch.equal(out, first)
    assert all(bool((o == 7).all()) for o in others)
