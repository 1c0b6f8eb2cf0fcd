"""How large and how small Keys and Values may be for the fp16 operands of packed pages: the limits that
kitty.h states, from both sides, and the rounding of what is near fp16's smallest numbers."""

import numpy as np
import pytest

from mixed_precision_bit_gb300 import synth
from tests.kitty_cases import dev16, dev32
from tests.tree_cases import D, P, PackedTree, check

pytestmark = pytest.mark.gpu
F16 = synth.F16


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


def refill(c, k, v):
    """The pages of c, all with the Keys and Values k, v [32, 128]."""
    from mixed_precision_bit_gb300 import kitty
    ids = np.concatenate([c.prefix, c.bt[c.bt >= 0]])
    x = [dev16(synth.to_bits(np.broadcast_to(y[None, :, None], (ids.size, P, c.Hkv, D)).reshape(-1, c.Hkv, D), F16)) for y in (k, v)]
    st = status0()
    kitty.quantize_pages(c.cfg, *x, dev32(ids), c.pool, c.pool_pages, status=st)
    assert int(st.item()) == 0


def spread(most, tokens):
    """+-most by turns, along the tokens (a channel's range) or the channels (a group's)."""
    t, ch = np.arange(P)[:, None], np.arange(D)[None]
    return np.where((t if tokens else ch) % 2 == 0, most, -most) + 0.0 * (t + ch)


# a step is rounded up to seven bits: 4064 is the largest below 4096, 8128 below 8192
LIMITS = [("key", 0, 2, 2, 6092, 6100), ("key", 128, 2, 2, 7616, 7624), ("key", 0, 4, 2, 30464, 30496),
          ("key", 128, 4, 4, 32368, 32400), ("value", 16, 2, 2, 12184, 12200), ("value", 0, 4, 4, 60928, 61024)]


@pytest.mark.parametrize("what,n_hi,lo_bit,v_bit,most,more", LIMITS)
def test_steps_at_the_limit(what, n_hi, lo_bit, v_bit, most, more):
    r = np.random.default_rng(1)
    c = PackedTree(2, 8, F16, own=[3, 1], tails=[5, 0], counts=[7, 12], n_hi=n_hi, lo_bit=lo_bit, v_bit=v_bit, seed=2,
                   q_scale=1e-3)
    for value, code in ((most, 0), (more, 2)):
        x, y = spread(value, what == "key"), r.standard_normal((P, D))
        refill(c, *((x, y) if what == "key" else (y, x)))
        st = status0()
        if code == 0:
            c.__dict__.pop("_pages", None)
            check(c, status=st)
        else:
            c.run(status=st)
        assert int(st.item()) == code, value


# (2-bit Keys of 6100 to 16376 * 3 / 2, 4-bit Values above 4094 * 15 / 2): tiles, prefix kernel
@pytest.mark.parametrize("what,lo_bit,v_bit,value,tiles,kernel", [("key", 2, 2, 6100, 2, 0), ("value", 4, 4, 40000, 0, 2),
                                                                  ("key", 2, 2, 6092, 0, 0), ("value", 4, 4, 30400, 0, 0)])
def test_a_prefix_is_held_to_either_limit(what, lo_bit, v_bit, value, tiles, kernel):
    r = np.random.default_rng(1)
    for B, nodes, code in ((2, 5, tiles), (40, 16, kernel)):
        c = PackedTree(2, 8, F16, own=[0] * B, tails=[5] * B, counts=[nodes] * B, n_prefix=128, n_hi=0, lo_bit=lo_bit,
                       v_bit=v_bit, seed=2, q_scale=1e-3)
        x, y = spread(value, what == "key"), r.standard_normal((P, D))
        refill(c, *((x, y) if what == "key" else (y, x)))
        st = status0()
        c.run(status=st)
        assert int(st.item()) == code, B


@pytest.mark.parametrize("lo_bit,v_bit", [(2, 2), (4, 4)])
@pytest.mark.parametrize("scale", [2.0 ** -11, 2.0 ** -15, 2.0 ** -19])
def test_small_values(scale, lo_bit, v_bit):
    """Each off by 2^-21 at most, as the bound has it."""
    r = np.random.default_rng(3)
    c = PackedTree(2, 8, F16, own=[3, 1], tails=[5, 31], counts=[7, 12], n_hi=16, lo_bit=lo_bit, v_bit=v_bit, seed=2)
    refill(c, r.standard_normal((P, D)), scale * r.standard_normal((P, D)))
    c.tail_v = synth.to_bits(scale * synth.from_bits(c.tail_v, F16), F16)
    c.put_cache()
    c.rows[:, 10:] = synth.to_bits(scale * synth.from_bits(c.rows[:, 10:], F16), F16)
    c.put_rows()
    st = status0()
    check(c, status=st)
    assert int(st.item()) == 0


@pytest.mark.parametrize("n_hi,lo_bit,v_bit", [(0, 2, 2), (16, 2, 2), (0, 4, 2), (16, 4, 4)])
@pytest.mark.parametrize("scale", [2.0 ** -10, 2.0 ** -14, 2.0 ** -18])
def test_small_keys(scale, n_hi, lo_bit, v_bit):
    """A page's Key elements off by 2^-21 at most, with 8-bit boosted ones by 2^-19 (a sixteenth of a step, times a
    low code, and two sums, each rounded at 2^-25 under 2^4): a score by that times the sum of |q|, which is as much
    as 1/4 or 1 more in the magnitudes that the bound takes 2^-19 of."""
    r = np.random.default_rng(3)
    c = PackedTree(2, 8, F16, own=[3, 1], tails=[0, 0], counts=[7, 12], n_hi=n_hi, lo_bit=lo_bit, v_bit=v_bit, seed=2,
                   q_scale=min(0.5 / scale, 2.0 ** 12))
    refill(c, scale * r.standard_normal((P, D)), r.standard_normal((P, D)))
    c.rows[:, 8:10] = synth.to_bits(scale * synth.from_bits(c.rows[:, 8:10], F16), F16)
    c.put_rows()
    held, more = c.cached, 1.0 if lo_bit == 4 and n_hi else 0.25

    def cached(b, h):
        k, v, part, size, most = held(b, h)
        return k, v, part, size + more, most

    c.cached = cached
    st = status0()
    check(c, status=st)
    assert int(st.item()) == 0
