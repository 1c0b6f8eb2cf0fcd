"""A captured reservation that is replayed while the host plans the pages: reported, and no page is taken twice."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
P, D = 32, 128


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixed_precision_bit_gb300 import kitty
    kitty.load()


@pytest.mark.parametrize("kind", ["LayerCache", "F16LayerCache"])
def test_replayed_between_hand_overs(kind):
    import torch
    from mixed_precision_bit_gb300 import cache, kitty
    c = getattr(cache, kind)(kitty.Config(num_kv_heads=1, num_q_heads=2, in_dtype=kitty.BF16), 3, 6, 18)
    rows = torch.randn(6 * P, 1, D, device="cuda").bfloat16().view(torch.int16)
    c.prefill(rows, rows, [3, 1, 2])
    c.pages_to_device()
    c.reserve(40)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.reserve(40)
    c.pages_to_host()
    table, free = c.block_table.clone(), c.alloc.free_count
    assert free == 12 and int(c.status.item()) == 0
    graph.replay()
    assert int(c.status.item()) == kitty.ST["BAD_LEN"] and torch.equal(c.block_table, table)
    c.status.zero_()
    c.pages_to_device()
    graph.replay()
    assert int(c.status.item()) == 0
    held = [4, 2, 3] if kind == "LayerCache" else [5, 3, 4]
    assert c.held.cpu().tolist() == held and int(c.free_count.item()) == 18 - sum(held)
    ids = c.block_table.cpu().numpy()
    assert np.unique(ids[ids >= 0]).size == sum(held)
    c.pages_to_host()
    assert c.alloc.free_count == 12 and torch.equal(c.block_table, table)
