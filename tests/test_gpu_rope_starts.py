"""Starts out of order in a ragged append: reported, and no sequence is advanced by tokens that
were not appended to it."""

import numpy as np
import pytest

from mixed_precision_bit_gb300 import synth
from tests import test_gpu_rope as rope_cases
from tests.kitty_cases import dev32

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixed_precision_bit_gb300 import kitty
    kitty.load()


@pytest.mark.parametrize("start,n", [([0, 5, 3, 8], 8), ([0, 3, 8, 5], 8), ([0, 2, 2, 9], 8), ([2, 5, 5, 8], 8),
                                     ([0, 8, 0, 8], 8), ([-1, 3, 5, 8], 8), ([0, 3, -4, 8], 8),
                                     ([0, 3, 5, 8], 8), ([0] + [40, 33] * 40, 48),
                                     (list(range(71)) + [60, 72], 72)])
def test_lengths_advance_by_whole_runs_alone(start, n):
    """Token t belongs to the sequence whose index is the number of ends at or before it; a
    sequence is advanced when all of its tokens are its own."""
    import torch
    from mixed_precision_bit_gb300 import kitty
    Hkv, Hq, dt = 1, 2, synth.BF16
    B, ends = len(start) - 1, np.array(start[1:])
    lens = np.arange(B) % 7
    cfg, pool, pool_pages, bt, free = rope_cases._cache16(B, Hkv, Hq, dt, 3, lens, 5)
    owner = (ends[None] <= np.arange(n)[:, None]).sum(1)
    want, bad = lens.copy(), False
    ids = np.full(n, -1, np.int32)
    want_bt = bt.copy()
    for t in range(n):
        b = owner[t]
        if b < B and start[b] <= t and (lens[b] + t - start[b]) % 32 == 0:
            ids[t] = free.pop()
    for b in range(B):
        lo, hi = start[b], start[b + 1]
        if lo == hi:
            continue
        if 0 <= lo < hi <= n and (owner[lo:hi] == b).all():
            want[b] += hi - lo
            for t in range(lo, hi):
                if ids[t] >= 0:
                    want_bt[b, (lens[b] + t - lo) // 32] = ids[t]
        else:
            bad = True
    bad = bad or start[0] > 0
    rope, _ = rope_cases._rope(32, 0, dt, "")
    x = rope_cases._rows(n, Hq + 2 * Hkv, dt, 6)
    qo = torch.full((n, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    d_ln, d_bt = dev32(lens), dev32(bt)
    kitty.f16kv_append_rope(cfg, rope, x[:, :Hq], x[:, Hq:Hq + 1], x[:, Hq + 1:], qo, pool, pool_pages, d_bt,
                            d_ln, dev32(ids), seq_start=dev32(start), status=st)
    assert int(st.item()) == (kitty.ST["BAD_SEQ"] if bad else 0)
    assert d_ln.tolist() == want.tolist()
    assert np.array_equal(d_bt.cpu().numpy(), want_bt)
    # rows that are no sequence's keep what they held
    own = [b < B and 0 <= start[b] <= t < start[b + 1] <= n for t, b in enumerate(owner)]
    assert ((qo != 7).any(-1).any(-1).cpu().numpy() == np.array(own)).all()
