"""More pages in the rows of a block table than 32-bit sums with the stack's height hold."""

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixed_precision_bit_gb300 import kitty
    kitty.load()


def test_rows_that_hold_the_same_page_over_and_over():
    """1024 rows of 2097151 times page 0, which are to go back on a stack of 2048 with 1024 pages on it: 2^31
    entries, refused as a whole."""
    import torch
    from mixed_precision_bit_gb300 import kitty
    rows, width = 1024, 2097151
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("a block table of 9 GB")
    i32 = lambda *s, v=0: torch.full(s, v, dtype=torch.int32, device="cuda")  # noqa: E731
    table, held, ids, count, st = i32(rows, width), i32(rows, v=width), i32(2048, v=5), i32(1, v=1024), i32(1)
    kitty.page_tables(i32(rows), held, table, ids, count, shrink=True, status=st)
    assert int(st.item()) == kitty.ST["BAD_PAGE"] and int(count.item()) == 1024
    assert bool((held == width).all()) and bool((ids == 5).all()) and not bool(table.any())
