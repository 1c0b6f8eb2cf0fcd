"""Decode attention behind a shared prefix, on the GPU, against the fp64 oracle's decode over
each sequence's prefix pages followed by its own: within the decode's 2e-3 of the output RMS
(+ half an output ulp).  Where that comes from here: a probability is rounded to fp16 once, by
at most 2^-11 of it, and the sum of the softmax is that of the rounded ones: an output is off
by sum p d (v - out) with |d| <= 2^-11 and random signs, 2^-11 / sqrt(3) = 2.8e-4 of the output
RMS (which is that of sum p v with random v): 7 deviations.  16-bit pages keep p in two parts
(2^-17 or less).  Key steps times codes, Key minima and Value steps times centered codes are
exact in fp16 for 2- and 4-bit codes; a Value group's middle is rounded once, by 2^-11 of it,
again with random signs over the tokens and no larger than v itself: sqrt(2) of the above at
most, 5 deviations."""

import numpy as np
import pytest

from mixed_precision_bit_gb300 import synth
from tests.kitty_cases import attn_error, dev32
from tests.shared_cases import D, Packed, Plain16, SM

pytestmark = pytest.mark.gpu
BF16, F16 = synth.BF16, synth.F16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixed_precision_bit_gb300 import kitty
    kitty.load()


def _status():
    import torch
    return torch.zeros(1, dtype=torch.int32, device="cuda")


PACKED = {
    "one": dict(Hkv=1, Hq=1, dt=F16, n_prefix=1, shared=None, own=[0], tails=[0]),
    "one_token": dict(Hkv=1, Hq=2, dt=BF16, n_prefix=2, shared=[0], own=[0], tails=[1]),
    "small": dict(Hkv=2, Hq=8, dt=BF16, n_prefix=5, shared=[5, 0, 3, 4], own=[0, 1, 0, 2], tails=[0, 7, 31, 5]),
    "odd": dict(Hkv=3, Hq=9, dt=F16, n_prefix=37, shared=None, own=[1, 0, 2, 0, 4], tails=[3, 1, 0, 0, 31]),
    "rows129": dict(Hkv=1, Hq=3, dt=BF16, n_prefix=7, shared=None, own=[0] * 43, tails=[1] * 43),
    "rows128": dict(Hkv=2, Hq=8, dt=BF16, n_prefix=9, shared=None, own=[0] * 32, tails=list(range(32))),
    "rows260": dict(Hkv=1, Hq=4, dt=F16, n_prefix=13, shared=[i % 14 for i in range(65)], own=[i % 2 for i in range(65)],
                    tails=[i % 32 for i in range(65)]),
    "group8": dict(Hkv=2, Hq=16, dt=BF16, n_prefix=40, shared=None, own=[2, 0, 1] * 6, tails=[9, 0, 31] * 6),
    "group32": dict(Hkv=1, Hq=32, dt=F16, n_prefix=11, shared=[11, 2], own=[1, 0], tails=[0, 3]),
    "group7": dict(Hkv=2, Hq=14, dt=BF16, n_prefix=12, shared=[12, 6, 1], own=[0, 0, 0], tails=[0, 0, 0]),
    "plain2": dict(Hkv=2, Hq=4, dt=BF16, n_prefix=20, shared=[20, 19, 18], own=[1, 1, 0], tails=[0, 0, 2], n_hi=0),
    "all_hi": dict(Hkv=2, Hq=4, dt=F16, n_prefix=20, shared=None, own=[1, 1, 0], tails=[0, 0, 2], n_hi=128),
    "k4": dict(Hkv=2, Hq=8, dt=BF16, n_prefix=14, shared=[14, 3], own=[1, 0], tails=[5, 0], n_hi=0, lo_bit=4),
    "kv4": dict(Hkv=2, Hq=8, dt=F16, n_prefix=14, shared=None, own=[1, 0], tails=[5, 0], n_hi=0, lo_bit=4, v_bit=4),
    "wide": dict(Hkv=8, Hq=32, dt=BF16, n_prefix=96, shared=None, own=[3] * 20, tails=[17] * 20),
}


@pytest.mark.parametrize("name", list(PACKED))
@pytest.mark.parametrize("out_dtype", ["f32", "bf16", "f16"])
def test_packed_matches_oracle(name, out_dtype):
    c = Packed(seed=7, **PACKED[name])
    st = _status()
    got = c.run(out_dtype, st)
    ref, ost = c.oracle()
    assert int(st.item()) == ost
    excess, rel = attn_error(got, ref, out_dtype)
    assert excess <= 0, "max err %.3e of RMS" % rel


@pytest.mark.parametrize("n_hi,v_bit", [(32, 2), (128, 2), (48, 4)])
def test_packed_84_matches_oracle(n_hi, v_bit):
    """8-bit boosted channels: a step of 7 bits times a code of 8 may take 15, and is rounded to
    fp16's 11: up to 2^-12 of each boosted Key, so a score is off by sm * 2^-12 * sum |q_c k_c|
    at most, and every probability and with it the output by that share of sum p |v|."""
    c = Packed(2, 8, BF16, 21, [21, 20, 1], [1, 0, 2], [4, 0, 31], seed=8, n_hi=n_hi, lo_bit=4, v_bit=v_bit)
    st = _status()
    got = c.run("f32", st)
    ref, ost = c.oracle()
    assert int(st.item()) == ost == 0
    q = np.abs(synth.from_bits(c.q, c.dt).astype(np.float64)).reshape(c.B, c.Hkv, -1, D)
    k = np.abs(synth.from_bits(c.k, c.dt).astype(np.float64))
    # every Key as if boosted, the largest over the tokens; two sides of the softmax's ratio
    shift = 2 * SM * 2.0 ** -12 * np.einsum("bhgd,thd->bhgt", q, k).max(-1).reshape(c.B, c.Hq, 1)
    vmax = np.abs(synth.from_bits(c.v, c.dt)).max()
    rms = np.sqrt((ref ** 2).mean())
    assert (np.abs(got - ref) <= 2e-3 * rms + np.expm1(shift) * vmax).all()
    assert np.sqrt(((got - ref) ** 2).mean()) <= 2e-3 * rms


PLAIN = {
    "one": dict(Hkv=1, Hq=1, dt=F16, n_prefix=1, shared=None, lens=[0]),
    "own_only": dict(Hkv=1, Hq=2, dt=BF16, n_prefix=2, shared=[0], lens=[1]),
    "small": dict(Hkv=2, Hq=8, dt=BF16, n_prefix=5, shared=[5, 0, 3, 4], lens=[0, 7, 33, 64]),
    "odd": dict(Hkv=3, Hq=9, dt=F16, n_prefix=37, shared=None, lens=[1, 0, 70, 0, 200]),
    "rows129": dict(Hkv=1, Hq=3, dt=BF16, n_prefix=7, shared=None, lens=[1] * 43),
    "rows260": dict(Hkv=1, Hq=4, dt=F16, n_prefix=13, shared=[i % 14 for i in range(65)], lens=[i % 40 for i in range(65)]),
    "wide": dict(Hkv=8, Hq=32, dt=BF16, n_prefix=96, shared=None, lens=[77] * 20),
}


@pytest.mark.parametrize("name", list(PLAIN))
@pytest.mark.parametrize("out_dtype", ["f32", "bf16", "f16"])
def test_16_bit_matches_oracle(name, out_dtype):
    c = Plain16(seed=9, **PLAIN[name])
    st = _status()
    got = c.run(out_dtype, st)
    ref, ost = c.oracle()
    assert int(st.item()) == ost
    excess, rel = attn_error(got, ref, out_dtype)
    assert excess <= 0, "max err %.3e of RMS" % rel


@pytest.mark.parametrize("kind", [Packed, Plain16])
def test_peaked_scores(kind):
    """Scores hundreds apart: one token takes all of the softmax, its maximum rises late in the
    prefix, and most probabilities are exactly 0."""
    own = dict(own=[1, 0, 0], tails=[3, 0, 9]) if kind is Packed else dict(lens=[35, 0, 9])
    c = kind(Hkv=2, Hq=8, dt=F16, n_prefix=50, shared=[50, 49, 2], seed=10, q_scale=30.0, **own)
    ref, _ = c.oracle()
    got = c.run("f32")
    # scores of magnitude s are formed in fp32 from products of that size: 2^-22 s each
    s = 30 * np.sqrt(D) * 60 * SM
    assert np.abs(got - ref).max() <= 2e-3 * np.sqrt((ref ** 2).mean()) + s * 2.0 ** -22 * 128 * 4


def test_empty_prefix_is_the_plain_decode():
    import torch
    c = Packed(2, 8, BF16, 0, None, [3, 0, 1], [5, 0, 0], seed=11)
    st = _status()
    got = c.run("f32", st)
    ref, ost = c.oracle()
    assert int(st.item()) == ost == 1                  # EMPTY: a sequence without a token
    assert attn_error(got, ref)[0] <= 0 and (got[1] == 0).all()
    c = Plain16(2, 8, BF16, 0, None, [70, 0, 1], seed=11)
    st = _status()
    got = c.run("f32", st)
    assert attn_error(got, c.oracle()[0])[0] <= 0 and int(st.item()) == 1


@pytest.mark.parametrize("kind", [Packed, Plain16])
def test_pages_that_a_sequence_does_not_share_do_not_touch_it(kind):
    """Infinities and NaN in the last pages of the prefix: the sequences that forked off before
    them give the bytes that they gave without."""
    import torch
    own = dict(own=[0, 1, 0, 0], tails=[3, 0, 9, 0]) if kind is Packed else dict(lens=[3, 32, 9, 0])
    c = kind(Hkv=2, Hq=8, dt=F16, n_prefix=11, shared=[5, 9, 11, 0], seed=12, **own)
    before = c.run("f32")
    pool = c.pool.view(c.pool_pages, -1).view(torch.uint8)
    for at in (9, 10):
        pool[int(c.prefix[at])] = 0x7C                 # 16-bit words 7cff (NaN) and 7c00 (infinity)
        pool[int(c.prefix[at]), ::2] = 0xFF if at == 9 else 0x00
    after = c.run("f32")
    for b in (0, 1, 3):
        assert np.array_equal(before[b], after[b]), b
    assert np.isfinite(before).all()


@pytest.mark.parametrize("kind", [Packed, Plain16])
def test_bad_ids_and_lengths_are_reported(kind):
    import torch
    own = dict(own=[1, 0, 2], tails=[3, 1, 9]) if kind is Packed else dict(lens=[35, 1, 70])
    c = kind(Hkv=2, Hq=4, dt=BF16, n_prefix=9, shared=[9, 4, 8], seed=13, **own)
    full = c.run("f32")
    # a page id out of range: its 32 tokens are left out
    for bad in (-1, c.pool_pages):
        st = _status()
        c.dev["prefix"][6] = bad
        got = c.run("f32", st)
        assert int(st.item()) == 4
        assert np.array_equal(got[1], full[1])         # does not share page 6
        keep = c.prefix.copy()
        c2p, c2s = np.delete(keep, 6), np.array([8, 4, 7])
        c.prefix, old = c2p, c.shared
        c.shared = c2s
        ref, _ = c.oracle()
        c.prefix, c.shared = keep, old
        assert attn_error(got, ref)[0] <= 0
    c.dev["prefix"][6] = int(c.prefix[6])
    # a prefix length outside [0, n_prefix] counts as 0
    for bad in (-3, 10):
        st = _status()
        c.dev["shared"][0] = bad
        got = c.run("f32", st)
        assert int(st.item()) == 5
        c.shared = np.array([0, 4, 8])
        assert attn_error(got, c.oracle()[0])[0] <= 0
        assert np.array_equal(got[1:], full[1:])
        c.shared = np.array([9, 4, 8])


def test_steps_beyond_fp16_products_are_reported():
    """A Key channel that spans the whole input range: its step times a code leaves fp16."""
    import torch
    from mixed_precision_bit_gb300 import kitty
    c = Packed(1, 2, F16, 4, [4, 2], [0, 0], [1, 1], seed=14, n_hi=0)
    ok = c.run("f32")
    k = c.k.copy()
    k[3 * 32:4 * 32, 0, 5] = np.where(np.arange(32) % 2, 0x7BFF, 0xFBFF)  # +-65504 in page 3
    from tests.kitty_cases import dev16
    kitty.quantize_pages(c.cfg, dev16(k), dev16(c.v), dev32(c.ids), c.pool, c.pool_pages)
    st = _status()
    got = c.run("f32", st)
    assert int(st.item()) == 2
    assert np.array_equal(got[1], ok[1])               # shares pages 0 and 1 only


def test_offsets_beyond_32_bits():
    """Prefix and own pages more than 4 GiB into the pool."""
    import torch
    if torch.cuda.get_device_properties(0).total_memory < 16 << 30:
        pytest.skip("needs 16 GiB")
    c = Packed(8, 32, BF16, 6, [6, 3], [1, 0], [2, 5], seed=15, spare=200000)
    assert int(c.prefix.min()) * 8 * 3360 > 1 << 32
    ref, _ = Packed.oracle(c)
    assert attn_error(c.run("f32"), ref)[0] <= 0


@pytest.mark.parametrize("kind", [Packed, Plain16])
def test_same_call_twice_gives_the_same_bytes_and_graphs_replay(kind):
    """Captured as a first call, two graphs on one workspace replayed in turn, and direct calls
    on a side stream: the same bytes, however often."""
    import torch
    own = dict(own=[1, 0, 2] * 8, tails=[3, 1, 9] * 8) if kind is Packed else dict(lens=[35, 1, 70] * 8)
    a = kind(Hkv=2, Hq=8, dt=BF16, n_prefix=33, shared=None, seed=16, **own)
    b = kind(Hkv=2, Hq=8, dt=BF16, n_prefix=33, shared=[33, 12, 5] * 8, seed=17, **own)
    ws = a.workspace()
    outs, graphs = [], []
    for c in (a, b):
        out = torch.zeros(c.B, c.Hq, D, dtype=torch.bfloat16, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.call(out, ws=ws)
        outs.append(out)
        graphs.append(g)
    first = None
    for _ in range(3):
        for g in graphs:
            g.replay()
        now = [o.clone() for o in outs]
        assert first is None or all(torch.equal(x, y) for x, y in zip(first, now))
        first = first or now
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for c, o in zip((a, b), outs):
            o.zero_()
            c.call(o, ws=ws, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(first, outs))
    for c, o in zip((a, b), outs):
        assert attn_error(o.float().cpu().numpy().astype(np.float64), c.oracle()[0], "bf16")[0] <= 0


def test_next_calls_in_the_stream_see_the_outputs():
    """Three launches that may overlap: what follows them in the stream reads finished outputs,
    and a call that reuses the workspace at once does not disturb the one before."""
    import torch
    c = Packed(4, 16, BF16, 64, None, [4] * 16, [11] * 16, seed=18)
    ref = c.run("f32")
    ws = c.workspace()
    outs = [torch.zeros(c.B, c.Hq, D, device="cuda") for _ in range(20)]
    copies = []
    for o in outs:
        c.call(o, ws=ws)
        copies.append(o.clone())
    torch.cuda.synchronize()
    for o in copies:
        assert np.array_equal(o.cpu().numpy().astype(np.float64), ref)
