"""Pages for tokens that may come: near the end of its row of the block table a sequence gets those that
the row has room for."""

import numpy as np
import pytest

from mixed_precision_bit_gb300 import synth
from tests.kitty_cases import dev32

pytestmark = pytest.mark.gpu
P, D, Hkv, Hq = 32, 128, 1, 2


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


@pytest.mark.parametrize("partial", [True, False])
def test_extra_tokens_end_with_the_row(partial):
    """held + new tokens have to fit, the extra ones need not: [held, new] of rows of 3 pages."""
    from mixed_precision_bit_gb300 import kitty
    import torch
    have, new = np.array([90, 95, 96, 64, 0]), np.array([6, 2, 0, 31, 0])
    fits = have + new <= 3 * P + (0 if partial else P - 1)
    want = np.where(fits, np.minimum((have + new + 20 + (P - 1 if partial else 0)) // P, 3), 0)
    t = dict(held=dev32([0] * 5), block_table=dev32([[-1] * 3] * 5), free_ids=dev32(np.arange(15)),
             free_count=dev32([15]))
    st = status0()
    start = np.concatenate([[0], np.cumsum(new)])
    kitty.page_tables(dev32(have), seq_start=dev32(start), extra=20, partial=partial, status=st, **t)
    assert t["held"].cpu().tolist() == list(want) and int(st.item()) == (0 if fits.all() else 8)
    assert int(t["free_count"].item()) == 15 - want.sum()
    ids = t["block_table"].cpu().numpy()
    assert [int((row >= 0).sum()) for row in ids] == list(want) and np.unique(ids[ids >= 0]).size == want.sum()
    # and back again
    kitty.page_tables(dev32(have), seq_start=dev32(start), partial=partial, shrink=True, status=st, **t)
    small = np.where(fits, (have + new + (P - 1 if partial else 0)) // P, 0)
    assert t["held"].cpu().tolist() == list(small)
    assert torch.equal(t["free_ids"][:15 - int(small.sum())], dev32(np.arange(15 - small.sum())))


@pytest.mark.parametrize("kind", ["LayerCache", "F16LayerCache"])
def test_the_last_paths_of_a_full_row(kind):
    """Rows of 2 pages near their end: short paths still go in though room for 8 was asked; then one that
    is too long is refused, the others go on."""
    from mixed_precision_bit_gb300 import cache, kitty
    import torch
    cfg = kitty.Config(num_kv_heads=Hkv, num_q_heads=Hq, in_dtype=synth.BF16)
    packed = kind == "LayerCache"  # 2 full pages and a tail of up to 31 tokens; else 64 tokens
    pages, tails, first, most = ([2, 2, 1], [27, 28, 0], [3, 3, 8], 95) if packed else ([1, 1, 1], [28, 28, 0], [3, 4, 8], 64)
    c = getattr(cache, kind)(cfg, 3, 2, 6)
    rows = torch.randn(sum(pages) * P, Hkv, D, device="cuda").bfloat16().view(torch.int16)
    tail = [torch.randn(3, Hkv, P, D, device="cuda").bfloat16().view(torch.int16) for _ in range(2)]
    c.prefill(rows, rows, pages, *tail, tails)
    c.pages_to_device()

    def step(lens):
        k = torch.randn(24, Hkv, D, device="cuda").bfloat16()
        n = dev32(lens)
        c.reserve(8)
        c.commit_tree(k, k, dev32([0, 8, 16, 24]), dev32([list(range(8))] * 3), n)
        return n

    total = lambda: (c.num_pages * P + c.tail_len if packed else c.ctx_len).cpu().tolist()  # noqa: E731
    for lens, after in ((first, [most - 1, most, 40]), ([1, 0, 8], [most, most, 48]), ([0, 0, 8], [most, most, 56])):
        step(lens)
        assert int(c.status.item()) == 0 and total() == after
    step([1, 0, 8])
    assert int(c.status.item()) == kitty.ST["TABLE_FULL"] and total() == [most, most, 64]
    c.pages_to_host()
    assert c.alloc.free_count == 0


def test_a_step_without_new_tokens():
    """Slot maps without an entry: pages as without them."""
    from mixed_precision_bit_gb300 import kitty
    import torch
    for empty in (dict(slots=torch.zeros(0, dtype=torch.int64, device="cuda")), dict(new_page_ids=dev32([]))):
        t = dict(held=dev32([0, 0]), block_table=dev32([[-1] * 3] * 2), free_ids=dev32(np.arange(5)), free_count=dev32([5]))
        st = status0()
        kitty.page_tables(dev32([33, 0]), seq_start=dev32([0, 0, 0]), status=st, **empty, **t)
        assert int(st.item()) == 0 and t["held"].cpu().tolist() == [2, 0] and t["block_table"].cpu().tolist()[0] == [4, 3, -1]
        kitty.page_tables(dev32([33, 0]), seq_start=dev32([0, 0, 1]), status=st, **empty, **t)  # a token without an entry
        assert int(st.item()) == kitty.ST["BAD_SEQ"]
