"""Calls on drafted trees that the documentation allows and ordinary use seldom makes: bounded waits that
run out, streams that overlap, pools beyond 32-bit offsets, many sequences, prefixes by both ways."""

import numpy as np
import pytest

from mixed_precision_bit_gb300 import synth
from tests.tree_cases import PackedTree, Plain16Tree, check

pytestmark = pytest.mark.gpu
BF16, F16 = synth.BF16, synth.F16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixed_precision_bit_gb300 import kitty
    kitty.load()


def status0():
    import torch
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def make(kind, pages, counts, **kw):
    """pages[b] full pages and 5 tokens of each sequence."""
    if kind is PackedTree:
        return PackedTree(2, 8, BF16, own=pages, tails=[5] * len(pages), counts=counts, **kw)
    return Plain16Tree(2, 8, BF16, lens=[32 * n + 5 for n in pages], counts=counts, **kw)


@pytest.mark.parametrize("n_prefix", [0, 40])
@pytest.mark.parametrize("kind", [PackedTree, Plain16Tree])
def test_a_wait_that_runs_out_is_reported(kind, n_prefix):
    """One poll of a barrier is too short for a copy from memory: the call ends, says so, and the next
    one gives the same bytes as before."""
    import torch
    from mixed_precision_bit_gb300 import kitty
    c = make(kind, [60, 33], [16, 9], n_prefix=n_prefix, seed=5)
    st = status0()
    before = c.run(status=st)
    assert int(st.item()) == 0
    flush = torch.empty(512 << 20, dtype=torch.uint8, device="cuda")
    flush.fill_(1)
    c.cfg.decode_wait_polls = 1
    c.run(status=st)
    assert int(st.item()) == kitty.ST["TIMEOUT"]
    c.cfg.decode_wait_polls = 0
    st.zero_()
    assert np.array_equal(c.run(status=st), before) and int(st.item()) == 0


@pytest.mark.parametrize("kind", [PackedTree, Plain16Tree])
def test_two_graphs_at_once(kind):
    """Captured calls with a workspace each, replayed on two streams."""
    import torch
    cs = [make(kind, [70, 3, 0], [16, 5, 30], n_prefix=n, seed=7 + n) for n in (0, 6)]
    want = [c.run() for c in cs]
    outs, graphs, keep = [], [], []
    for c in cs:
        ws, pre = c.workspace(), c.prefix_args()
        c.prefix_args = lambda pre=pre: pre
        out = torch.zeros((c.T, 8, 128), dtype=torch.float32, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.call(out, ws=ws)
        outs.append(out), graphs.append(g), keep.append((ws, pre))
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for out, w in zip(outs, want):
        assert np.array_equal(out.cpu().numpy(), w)


@pytest.mark.parametrize("kind", [PackedTree, Plain16Tree])
def test_pages_beyond_32_bit_offsets(kind):
    """The same pages at the end of a pool of more than 4 GB."""
    import torch
    from mixed_precision_bit_gb300 import kitty
    c = make(kind, [9, 4], [7, 16], n_prefix=3, seed=3)
    want = c.run()
    page = (kitty.page_bytes if kind is PackedTree else kitty.f16kv_page_bytes)(c.cfg)[1]
    more = (9 << 29) // page  # 4.5 GB of pages in front
    pool = torch.zeros((more + c.pool_pages) * page, dtype=torch.uint8, device="cuda")
    pool[more * page:] = c.pool.view(torch.uint8).reshape(-1)
    c.pool, c.pool_pages = pool, c.pool_pages + more
    c.bt = np.where(c.bt >= 0, c.bt + more, -1).astype(np.int32)
    c.prefix = (c.prefix + more).astype(np.int32)
    c.c["bt"].copy_(torch.from_numpy(c.bt))
    assert np.array_equal(c.run(), want)


@pytest.mark.parametrize("kind", [PackedTree, Plain16Tree])
def test_many_sequences_of_one_node(kind):
    r = np.random.default_rng(2)
    pages = r.integers(0, 3, 700)
    counts = np.where(r.random(700) < 0.3, 0, 1)
    st = status0()
    check(make(kind, pages, counts, seed=1), status=st)
    assert int(st.item()) == 0


@pytest.mark.parametrize("kind", [PackedTree, Plain16Tree])
@pytest.mark.parametrize("shared", ["all", "some"])
@pytest.mark.parametrize("B,nodes", [(2, 5), (40, 16)])
def test_prefix_in_tiles_and_by_the_prefix_kernel(kind, shared, B, nodes):
    """Few drafted tokens take the prefix as part of each sequence's tiles, many take the prefix
    kernel: both within the bounds (of the first and last sequences), padding rows untouched, rows of NaN
    behind the last sequence without effect."""
    from mixed_precision_bit_gb300 import kitty
    r = np.random.default_rng(B)
    n = 128
    sees = None if shared == "all" else r.integers(0, n + 1, B)
    c = make(kind, r.integers(0, 4, B), r.integers(0, nodes + 1, B), n_prefix=n, shared=sees, pad=3, seed=B)
    # partials of the prefix kernel beside the own ones: more than the splits of few tiles
    apart = c.size(c.cfg, B, c.T, c.max_nodes(), c.max_pages, n) - c.size(c.cfg, B, c.T, c.max_nodes(), c.max_pages, 0)
    assert B == 2 or apart % (c.T * 8 * 528) == c.T * 4
    for name in ("q", "k", "v"):
        c.d[name][c.T - 3:] = 0x7FFF
    st = status0()
    got = c.run(status=st)
    assert int(st.item()) == 0
    for first, last in ((0, 3), (B - 2, B)):
        lo, hi = int(c.start[max(first, 0)]), int(c.start[min(last, B)])
        counts, c.counts = c.counts, [m if first <= b < last else 0 for b, m in enumerate(c.counts)]
        ref, off = c.answer()
        c.counts = counts
        assert (np.abs(got - ref) <= off + 2.0 ** -24 * np.abs(ref))[lo:hi].all()
    if shared == "some":  # a count that is out of range: reported, and none of the prefix is seen
        sees[0] = n + 1
        c.run(status=st)
        assert int(st.item()) == kitty.ST["BAD_LEN"]


def test_strided_rows_behind_a_prefix():
    """Queries, keys and values as columns of one projection, many rows, behind a prefix."""
    for kind in (PackedTree, Plain16Tree):
        c = make(kind, [1] * 24, [12] * 24, n_prefix=6, seed=4)
        assert not c.d["q"].is_contiguous()
        check(c)
