"""Shared-prefix decode against bounds derived for each output: maxima that rise by more than the
kernel lets pass without a rescale, and the rounding of 8-bit boosted Keys."""

import numpy as np
import pytest

import oracle
from mixed_precision_bit_gb300 import synth
from tests.kitty_cases import attn_error, dev16, dev32
from tests.shared_cases import D, P, Packed, Plain16, SM

pytestmark = pytest.mark.gpu
BF16, F16 = synth.BF16, synth.F16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixed_precision_bit_gb300 import kitty
    kitty.load()


def _staircase(n, stairs, u, r):
    """Keys [n * 32, Hkv, 128] along +-1 vectors u [Hkv, 128]: small ones, and at each stair
    (page, token) a score 20 log2 units above the stair before; the last two as high."""
    c = 0.02 * r.standard_normal((n * P, u.shape[0]))
    level = 0.0
    for i, (page, token) in enumerate(stairs):
        if i < len(stairs) - 1:
            level += 20.0 / (D * SM * np.log2(np.e))
        c[page * P + token] = level
    return c[:, :, None] * u


@pytest.mark.parametrize("dt", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("kind", [Packed, Plain16])
@pytest.mark.parametrize("Hq,B", [(2, 1), (8, 3), (8, 70)])
def test_maxima_that_rise_through_the_prefix(kind, dt, Hq, B):
    """Five stairs of 20 log2 units (more than the 15 that the reference may be passed by), two in
    one tile, the last two equal and tiles apart: the output is the mix of the last ones that a
    sequence sees, and what came before must vanish in a rescale.  The scores' errors do not
    matter: at most 120 log2 units, formed in fp32 by 8 sums of 16 exact products and a few
    more, each rounded by 2^-23 of it at most: 16 * 2^-23 * 120 * ln 2 = 1.6e-4 of a weight, so the
    2e-3 of the output RMS stand as they are."""
    n, Hkv = 50, 2
    r = np.random.default_rng(60)
    own = dict(own=[i % 2 for i in range(B)], tails=[1 + i % 31 for i in range(B)]) if kind is Packed else \
        dict(lens=[1 + 7 * i % 40 for i in range(B)])
    shared = None if B == 1 else [(50, 45, 23)[i % 3] for i in range(B)]
    c = kind(Hkv=Hkv, Hq=Hq, dt=dt, n_prefix=n, shared=shared, seed=61, **own)
    c.cfg.decode_total_pages = 1 << 20                     # on few blocks: many tiles each
    u = r.choice([-1.0, 1.0], (Hkv, D))
    k = synth.to_bits(_staircase(n, [(2, 3), (3, 0), (20, 31), (22, 8), (40, 5), (48, 17)], u, r), dt)
    scale = np.array([1.0, 1.25, 0.875, 1.5])[np.arange(Hq) % (Hq // Hkv)]
    q = u[np.arange(Hq) // (Hq // Hkv)] * scale[:, None]
    c.q = synth.to_bits(np.broadcast_to(q, (B, Hq, D)), dt)
    c.dev["q"].copy_(dev16(c.q))
    if kind is Packed:
        from mixed_precision_bit_gb300 import kitty
        kitty.quantize_pages(c.cfg, dev16(k), dev16(c.v[:n * P]), dev32(c.ids[:n]), c.pool, c.pool_pages)
    else:
        c.host[c.prefix, :, 0] = k.reshape(n, P, Hkv, D).transpose(0, 2, 1, 3)
        c.pool.copy_(dev16(c.host))
    ref, _ = c.oracle()
    got = c.run("f32")
    excess, rel = attn_error(got, ref)
    assert excess <= 0, "max err %.3e of RMS" % rel
    # the oracle without the last stair is far off: the token before it carries weight, too
    sees, c.shared = c.shared, np.minimum(c.shared, 48)
    less, _ = c.oracle()
    rows = sees == 50
    assert (np.abs(less - ref)[rows].max(-1) > 0.1 * np.sqrt((ref ** 2).mean())).all()


@pytest.mark.parametrize("n_hi,v_bit", [(32, 2), (128, 2), (48, 4), (16, 4)])
@pytest.mark.parametrize("q_scale", [1.0, 3.0])
def test_boosted_84_keys_within_their_rounding(n_hi, v_bit, q_scale):
    """A step of 7 bits times a code of 8 has 15, rounded to the 11 of fp16: off by at most half a
    step of it, 2^-11 of step * code.  So token t's score is off by at most
      e_t = sm * 2^-11 * sum over the page's boosted channels of |q_c| (k_tc - M_c),
    and since sum p (v - out) = 0,
      |out' - out| = |sum p (exp(d) - 1) (v - out)| / sum p exp(d), |d_t| <= e_t
                  <= exp(max e) * sum p expm1(e_t) |v_t - out|,
    beside the 2e-3 of the output RMS of all else."""
    Hkv, Hq, g = 2, 8, 4
    c = Packed(Hkv, Hq, BF16, 37, [37, 36, 1], [1, 0, 2], [4, 0, 31], seed=62, n_hi=n_hi, lo_bit=4, v_bit=v_bit,
               q_scale=q_scale)
    got = c.run("f32")
    ref, ost = c.oracle()
    assert ost == 0
    blobs = c.pool.cpu().numpy().reshape(c.pool_pages, Hkv, -1)
    q = synth.from_bits(c.q, c.dt).astype(np.float64)
    tk, tv = (synth.from_bits(x, c.dt).astype(np.float64) for x in (c.tail_k, c.tail_v))
    rms = np.sqrt((ref ** 2).mean())
    sharp = []
    for b in range(c.B):
        ids = np.concatenate([c.prefix[:c.shared[b]], c.bt[b, :c.own[b]]])
        for h in range(Hkv):
            ks, vs, parts = [], [], []
            for i, pid in enumerate(ids):
                kd, vd, _ = oracle.dequant_page(blobs[pid, h], n_hi, 4, v_bit)
                part = np.zeros((P, D))
                if i < c.shared[b]:
                    ch = np.asarray(oracle.page_channels(blobs[pid, h], n_hi, 4), int)
                    part[:, ch] = (kd - kd.min(0))[:, ch]  # the token of the minimum has code 0
                ks.append(kd)
                vs.append(vd)
                parts.append(part)
            n = c.tails[b]
            ks, vs = np.concatenate(ks + [tk[b, h, :n]]), np.concatenate(vs + [tv[b, h, :n]])
            parts = np.concatenate(parts + [np.zeros((n, D))])
            for j in range(g):
                row = q[b, h * g + j]
                s = SM * (ks @ row)
                p = np.exp(s - s.max())
                p /= p.sum()
                out = p @ vs
                assert np.abs(out - ref[b, h * g + j]).max() <= 1e-6 * rms  # the same softmax as the oracle's
                e = SM * 2.0 ** -11 * (parts @ np.abs(row))
                bound = np.exp(e.max()) * (p * np.expm1(e)) @ np.abs(vs - out)
                off = np.abs(got[b, h * g + j] - out)
                assert (off <= 2e-3 * rms + bound).all(), (b, h, j, (off - bound).max() / rms)
                sharp.append(bound.max() / rms)
    assert max(sharp) < 0.2                                # a bound that says something
