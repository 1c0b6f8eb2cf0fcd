"""Attention of drafted trees over both caches, against 64 bits with a bound derived for each output."""

import numpy as np
import pytest

from mixed_precision_bit_gb300 import synth
from tests.tree_cases import PackedTree, Plain16Tree, check

pytestmark = pytest.mark.gpu
BF16, F16 = synth.BF16, synth.F16
ids = dict(ids=["bf16", "f16"])


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


@pytest.mark.parametrize("dt", [BF16, F16], **ids)
@pytest.mark.parametrize("kind", ["tree", "chain", "any"])
@pytest.mark.parametrize("Hkv,Hq", [(2, 8), (1, 1), (3, 18)])
def test_packed(dt, kind, Hkv, Hq):
    """Ragged trees over nothing, a tail, pages, both; lengths that end inside a tile of pages."""
    c = PackedTree(Hkv, Hq, dt, own=[0, 5, 1, 13, 4, 0], tails=[0, 0, 31, 7, 32, 1], counts=[5, 1, 0, 9, 3, 16],
                   kind=kind, seed=1, pad=2)
    st = status0()
    check(c, status=st)
    empty = kind == "any" and any(int(v) & 31 == 0 for v in c.visible[:5])
    assert int(st.item()) == (1 if empty else 0)


@pytest.mark.parametrize("dt", [BF16, F16], **ids)
@pytest.mark.parametrize("n_hi,lo_bit,v_bit", [(0, 2, 2), (16, 2, 2), (64, 2, 2), (128, 2, 2), (0, 4, 2), (48, 4, 2),
                                               (0, 4, 4), (32, 4, 4), (128, 4, 4)])
def test_formats(dt, n_hi, lo_bit, v_bit):
    c = PackedTree(2, 8, dt, own=[9, 2], tails=[3, 0], counts=[7, 12], n_hi=n_hi, lo_bit=lo_bit, v_bit=v_bit, seed=2)
    st = status0()
    check(c, status=st)
    assert int(st.item()) == 0


@pytest.mark.parametrize("dt", [BF16, F16], **ids)
@pytest.mark.parametrize("kind", ["tree", "chain", "any"])
@pytest.mark.parametrize("Hkv,Hq", [(2, 8), (1, 1), (3, 18)])
def test_plain16(dt, kind, Hkv, Hq):
    c = Plain16Tree(Hkv, Hq, dt, lens=[0, 1, 31, 32, 33, 260, 127, 128, 129], counts=[4, 1, 9, 3, 0, 16, 5, 2, 7],
                    kind=kind, seed=3, pad=3)
    st = status0()
    check(c, status=st)
    empty = kind == "any" and any(int(v) & 15 == 0 for v in c.visible[:4])
    assert int(st.item()) == (1 if empty else 0)


@pytest.mark.parametrize("counts,Hkv,Hq", [([64, 63, 1], 1, 8), ([64], 2, 2), ([33, 64, 17], 1, 5), ([64, 2], 1, 32)])
@pytest.mark.parametrize("kind", ["tree", "any"])
def test_large_trees(counts, Hkv, Hq, kind):
    own = [3, 17, 0][:len(counts)]
    check(PackedTree(Hkv, Hq, BF16, own=own, tails=[4] * len(counts), counts=counts, kind=kind, seed=4))
    check(Plain16Tree(Hkv, Hq, BF16, lens=[32 * x + 4 for x in own], counts=counts, kind=kind, seed=4))


@pytest.mark.parametrize("out_dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dt", [BF16, F16], **ids)
def test_output_types(out_dtype, dt):
    check(PackedTree(2, 6, dt, own=[6, 0], tails=[9, 2], counts=[4, 6], seed=5), out_dtype)
    check(Plain16Tree(2, 6, dt, lens=[200, 2], counts=[4, 6], seed=5), out_dtype)


@pytest.mark.parametrize("dt", [BF16, F16], **ids)
@pytest.mark.parametrize("n_prefix,shared", [(1, None), (7, None), (26, [26, 0, 13, 1])])
def test_behind_a_shared_prefix(dt, n_prefix, shared):
    kw = dict(n_prefix=n_prefix, shared=shared, seed=6, pad=1)
    st = status0()
    check(PackedTree(2, 8, dt, own=[0, 3, 1, 0], tails=[5, 0, 31, 0], counts=[3, 8, 0, 12], **kw), status=st)
    check(Plain16Tree(2, 8, dt, lens=[5, 96, 63, 0], counts=[3, 8, 0, 12], **kw), status=st)
    assert int(st.item()) == 0


@pytest.mark.parametrize("dt", [BF16, F16], **ids)
def test_long_contexts(dt):
    """Many tiles and splits, one sequence alone and beside short ones."""
    check(PackedTree(1, 4, dt, own=[311], tails=[17], counts=[11], seed=7), "f32")
    check(PackedTree(2, 8, dt, own=[150, 2, 0], tails=[0, 30, 3], counts=[6, 20, 1], seed=8))
    check(Plain16Tree(1, 4, dt, lens=[9999], counts=[11], seed=7))
    check(Plain16Tree(2, 8, dt, lens=[4800, 70, 3], counts=[6, 20, 1], seed=8))


@pytest.mark.parametrize("kind", [PackedTree, Plain16Tree])
def test_scores_that_rise(kind):
    """Large queries: maxima far apart, weights from 1 down to nothing, both signs of the scale."""
    kw = dict(own=[40, 3], tails=[5, 31]) if kind is PackedTree else dict(lens=[1285, 127])
    for sm in (kind.sm, -kind.sm):
        c = kind(2, 8, BF16, counts=[9, 4], seed=9, q_scale=8.0, **kw)
        c.sm = sm
        if sm < 0:  # the same as the negated query
            c.rows[:, :8] ^= 0x8000
            ref = c.answer()
            c.rows[:, :8] ^= 0x8000
            c.answer = lambda: ref
        check(c)


@pytest.mark.parametrize("kind", [PackedTree, Plain16Tree])
@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
def test_masked_values_reach_no_one(kind, value):
    """Keys and values that are not finite at a node that only some rows see: the others' outputs are
    the same bytes as with numbers there."""
    kw = dict(own=[3, 0], tails=[5, 1]) if kind is PackedTree else dict(lens=[101, 1])
    c = kind(1, 4, BF16, counts=[7, 3], seed=10, **kw)
    c.visible[:7] = [1, 3, 4 | 1, 8 | 1, 16 | 4 | 1, 32 | 3, 64]
    c.put_rows()
    st = status0()
    base = c.run(status=st)
    assert int(st.item()) == 0
    c.rows[2, 4:] = synth.to_bits(np.full((2, 128), value), BF16)
    c.put_rows()
    with np.errstate(invalid="ignore"):
        got = c.run(status=st)
    assert int(st.item()) == 3  # rows 2 and 4 see it
    rows = [0, 1, 3, 5, 6, 7, 8, 9]
    assert np.array_equal(got[rows], base[rows])
    c.visible[[2, 4]] = 1                                     # now no one does
    c.put_rows()
    st.zero_()
    got = c.run(status=st)
    assert int(st.item()) == 0 and np.array_equal(got[rows], base[rows]) and np.isfinite(got).all()


def test_values_beyond_fp16_on_packed_pages():
    c = PackedTree(1, 2, BF16, own=[2], tails=[3], counts=[3], kind="chain", seed=11)
    st = status0()
    c.rows[2, 2, 5] = synth.to_bits(np.array([1e6]), BF16)[0]   # the last node's key: seen by itself
    c.put_rows()
    base = c.run(status=st)
    assert int(st.item()) == 2
    ref, off = c.answer()
    assert (np.abs(base - ref) <= off + 1e-6)[:2].all()
    c = PackedTree(1, 2, BF16, own=[2], tails=[3], counts=[3], seed=11)
    c.rows[1, 0, 5] = synth.to_bits(np.array([np.nan]), BF16)[0]  # a query
    c.put_rows()
    st.zero_()
    got = c.run(status=st)
    assert int(st.item()) == 3
    ref, off = c.answer()
    ok = np.abs(got - ref) <= off + 1e-6
    ok[1, 0] = True
    assert ok.all()


def test_bad_pages_and_lengths():
    """A page id out of range is left out; a sequence of impossible lengths or starts is skipped."""
    for kind in (PackedTree, Plain16Tree):
        kw = dict(own=[6, 2, 1], tails=[5, 31, 2]) if kind is PackedTree else dict(lens=[197, 95, 34])
        c = kind(2, 4, BF16, counts=[3, 5, 2], seed=12, **kw)
        base = c.run()
        st = status0()
        bt = c.bt.copy()
        c.c["bt"][0, 2] = c.pool_pages
        got = c.run(status=st)
        assert int(st.item()) == 4 and np.array_equal(got[3:], base[3:])
        full = c.cached

        def without(b, h):
            out = full(b, h)
            return tuple(np.delete(x, np.arange(64, 96), 0) for x in out) if b == 0 else out

        c.cached = without
        ref, off = c.answer()
        assert (np.abs(got - ref) <= off + 1e-6).all()
        c.bt[:] = bt
        c.put_cache()
        name = "own" if kind is PackedTree else "lens"
        c.c[name][1] = -1
        st.zero_()
        got = c.run(status=st)
        assert int(st.item()) == 5 and (got[3:8] == 7.0).all()
        assert np.array_equal(got[:3], base[:3]) and np.array_equal(got[8:], base[8:])
        c.put_cache()
        st.zero_()
        got = c.run(status=st, max_nodes=4)                    # the second tree has five nodes
        assert int(st.item()) == 5 and (got[3:8] == 7.0).all() and np.array_equal(got[8:], base[8:])
        c.d["start"][2] = 99
        st.zero_()
        got = c.run(status=st)
        assert int(st.item()) == 9 and np.array_equal(got[:3], base[:3]) and (got[3:] == 7.0).all()


def test_repeats_bit_for_bit():
    import torch
    for c in (PackedTree(2, 8, BF16, own=[150, 2, 0], tails=[0, 30, 3], counts=[6, 20, 1], seed=8),
              Plain16Tree(2, 8, F16, lens=[4800, 70, 3], counts=[6, 20, 1], seed=8, n_prefix=9)):
        first = c.run()
        for _ in range(5):
            assert np.array_equal(c.run(), first)
        # alone, a sequence gives what it gives among the others' rows up to the split of its pages
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        assert np.array_equal(c.run(stream=s), first)


def test_captured_and_replayed():
    """A captured call attends what its tensors hold when it is replayed."""
    import torch
    for kind in (PackedTree, Plain16Tree):
        kw = dict(own=[20, 2], tails=[5, 31]) if kind is PackedTree else dict(lens=[645, 95])
        c = kind(2, 8, BF16, counts=[6, 9], seed=13, n_prefix=4, **kw)
        ws, pre = c.workspace(), c.prefix_args()
        c.prefix_args = lambda: pre
        out = torch.zeros((c.T, 8, 128), dtype=torch.float32, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.call(out, ws=ws)
        name = "own" if kind is PackedTree else "lens"
        for less in (0, 3, 1):
            c.c[name][0] -= less
            (c.own if kind is PackedTree else c.lens)[0] -= less
            g.replay()
            torch.cuda.synchronize()
            ref, off = c.answer()
            assert (np.abs(out.cpu().numpy() - ref) <= off + 1e-6).all()
