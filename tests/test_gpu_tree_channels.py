"""Elements of a drafted node's key or value on 16-bit pages that are not numbers: each counts as 0, its
neighbours as what they are."""

import numpy as np
import pytest

from mixed_precision_bit_gb300 import synth
from tests.tree_cases import Plain16Tree, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixed_precision_bit_gb300 import kitty
    kitty.load()


@pytest.mark.parametrize("dt", [synth.BF16, synth.F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("row", ["key", "value"])
def test_one_channel_that_is_not_a_number(dt, value, row):
    import torch
    c = Plain16Tree(1, 4, dt, lens=[101, 1], counts=[40, 3], kind="chain", seed=10)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    check(c, status=st)
    assert int(st.item()) == 0
    for node, channel in ((0, 0), (2, 77), (35, 126), (40, 9)):
        c.rows[node, 4 if row == "key" else 5, channel] = synth.to_bits(np.array([value]), dt)[0]
    c.put_rows()
    check(c, status=st)
    assert int(st.item()) == 3
