"""Slot maps without an entry: a step that brings no new tokens."""

import types

import pytest


@pytest.fixture
def call(monkeypatch):
    """kitty.page_tables on host tensors; what the library is given."""
    import torch
    from mixed_precision_bit_gb300 import kitty
    given = []
    monkeypatch.setattr(kitty, "_device", lambda: -1)
    monkeypatch.setattr(kitty, "_dense", lambda t, dev: None if t is None else t.data_ptr())
    monkeypatch.setattr(kitty, "load", lambda: types.SimpleNamespace(kitty_page_tables=lambda *a: given.append(a) or 0))
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731

    def run(**kw):
        kitty.page_tables(i32(3), i32(3), i32(3, 4), i32(12), i32(1), stream=0, **kw)
        return given[-1]

    return run


@pytest.mark.parametrize("slots,ids", [(0, 0), (0, None), (None, 0)])
def test_no_entries(call, slots, ids):
    import torch
    a = call(seq_start=torch.zeros(4, dtype=torch.int32),
             slots=None if slots is None else torch.zeros(slots, dtype=torch.int64),
             new_page_ids=None if ids is None else torch.zeros(ids, dtype=torch.int32))
    assert a[3] == 0 and not a[13] and not a[14]


def test_entries_are_counted(call):
    import torch
    start = torch.zeros(4, dtype=torch.int32)
    assert call(seq_start=start)[3] == 0x7FFFFFFF  # no map is written: any starts will do
    assert call()[3] == 0
    a = call(seq_start=start, slots=torch.zeros(7, dtype=torch.int64), new_page_ids=torch.zeros(7, dtype=torch.int32))
    assert a[3] == 7 and a[13] and a[14]
    for n, m in ((7, 6), (7, 0), (0, 7)):
        with pytest.raises(ValueError, match="new_page_ids|slots"):
            call(seq_start=start, slots=torch.zeros(n, dtype=torch.int64), new_page_ids=torch.zeros(m, dtype=torch.int32))
