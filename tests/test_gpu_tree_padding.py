"""Batches without a drafted token: only rows of padding, or only sequences that are skipped."""

import numpy as np
import pytest

from mixed_precision_bit_gb300 import synth
from tests.tree_cases import PackedTree, Plain16Tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixed_precision_bit_gb300 import kitty
    kitty.load()


@pytest.mark.parametrize("skipped", [False, True], ids=["padding", "skipped"])
@pytest.mark.parametrize("shared", [None, 100], ids=["all", "some"])
@pytest.mark.parametrize("kind", [PackedTree, Plain16Tree])
def test_a_call_behind_one_without_tokens(kind, shared, skipped):
    """Behind a prefix long enough for the prefix kernel, which attends the rows of padding too: the call
    ends with it, so that the next one may use the workspace."""
    import torch
    B, nodes, n = 40, 16, 128
    kw = dict(own=[1] * B, tails=[5] * B) if kind is PackedTree else dict(lens=[37] * B)
    c = kind(2, 8, synth.BF16, counts=[nodes] * B, n_prefix=n, shared=None if shared is None else [shared] * B, seed=1, **kw)
    apart = c.size(c.cfg, B, c.T, nodes, c.max_pages, n) - c.size(c.cfg, B, c.T, nodes, c.max_pages, 0)
    assert apart > c.T * 8 * 528  # the prefix kernel's partials
    ws, pre, start = c.workspace(), c.prefix_args(), c.d["start"].clone()
    c.prefix_args = lambda: pre
    want = c.run(ws=ws)
    none = torch.zeros_like(start)
    if skipped:
        none[:] = torch.arange(B, -1, -1, device="cuda")
    out = torch.full((c.T, 8, 128), 7.0, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(20):
        c.d["start"].copy_(none)
        c.call(out, status=st, ws=ws)
        c.d["start"].copy_(start)
        got = torch.full((c.T, 8, 128), 7.0, device="cuda")
        c.call(got, ws=ws)
        ws.fill_(float("nan"))  # nothing may write here any more
        assert bool(torch.isnan(ws).all())
        assert np.array_equal(got.cpu().numpy(), want)
    assert bool((out == 7.0).all()) and int(st.item()) == (9 if skipped else 0)
