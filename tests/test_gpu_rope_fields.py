"""A Rope whose fields change between calls: each call takes what they are then."""

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


def test_calls_take_the_fields_as_they_are():
    import torch
    from mixed_precision_bit_gb300 import kitty
    n, Hkv, Hq, dt = 9, 2, 6, synth.BF16
    cfg, f = rope_cases._cfg(Hkv, Hq, dt), kitty.rope_frequencies(128)[0]
    w = [(1 + 0.2 * torch.randn(D, device="cuda")).bfloat16() for _ in range(4)]
    q, k, pos = rope_cases._rows(n, Hq, dt, 1), rope_cases._rows(n, Hkv, dt, 2), dev32(range(50, 50 + n))

    def turned(rope):
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        kitty.norm_rope(cfg, rope, q, k, pos, qo, ko)
        return qo, ko

    same = lambda a, b: all(torch.equal(x, y) for x, y in zip(a, b))  # noqa: E731
    rope = kitty.Rope(f, q_weight=w[0], k_weight=w[1])
    turned(rope)
    rope.q_weight, rope.k_weight = w[2], w[3]              # the old ones are still alive: nothing stale is read
    assert same(turned(rope), turned(kitty.Rope(f, q_weight=w[2], k_weight=w[3])))
    rope.k_weight = None
    assert same(turned(rope), turned(kitty.Rope(f, q_weight=w[2])))
    rope.layout, rope.amplitude, rope.eps = kitty.ROPE_INTERLEAVED, 0.5, 0.125
    assert same(turned(rope), turned(kitty.Rope(f, kitty.ROPE_INTERLEAVED, 0.5, q_weight=w[2], eps=0.125)))
    keep = w[2].data
    rope.q_weight.data = w[0].clone()                      # the same tensor, other memory
    assert same(turned(rope), turned(kitty.Rope(f, kitty.ROPE_INTERLEAVED, 0.5, q_weight=w[0], eps=0.125)))
    del keep
