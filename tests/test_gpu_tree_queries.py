"""Queries that the tensor cores cannot take are reported however few tiles their sequence has for the
splits of the call."""

import numpy as np
import pytest

from mixed_precision_bit_gb300 import synth
from tests.tree_cases import PackedTree, Plain16Tree

pytestmark = pytest.mark.gpu
BF16, F16 = synth.BF16, synth.F16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixed_precision_bit_gb300 import kitty
    kitty.load()


@pytest.mark.parametrize("kind,dt,value,code", [(PackedTree, BF16, np.nan, 3), (PackedTree, BF16, 1e6, 2),
                                                (PackedTree, F16, np.inf, 3), (Plain16Tree, BF16, -np.inf, 3),
                                                (Plain16Tree, F16, np.nan, 3), (Plain16Tree, BF16, 1e6, 0)])
@pytest.mark.parametrize("nodes", [3, 40])
def test_a_short_sequence_beside_a_long_one(kind, dt, value, code, nodes):
    import torch
    kw = dict(own=[200, 2, 0], tails=[5, 1, 3]) if kind is PackedTree else dict(lens=[6405, 65, 3])
    c = kind(1, 4, dt, counts=[4, nodes, 2], seed=3, **kw)
    splits = c.size(c.cfg, c.B, c.T, c.max_nodes(), c.max_pages, 0) // (c.T * 4 * 528)
    assert splits > 2  # more than the tiles of the short ones
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    base = c.run(status=st)
    assert int(st.item()) == 0
    for row in (4, 3 + nodes, c.T - 1):  # the second sequence's first and last rows, the third's last
        keep = c.rows.copy()
        c.rows[row, 1, 77] = synth.to_bits(np.array([value]), dt)[0]
        c.put_rows()
        got = c.run(status=st)
        assert int(st.item()) == code, row
        other = np.ones((c.T, 4), bool)
        other[row, 1] = False
        assert np.array_equal(got[other], base[other])
        c.rows[:] = keep
        st.zero_()
