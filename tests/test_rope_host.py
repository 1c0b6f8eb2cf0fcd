"""Frequencies and rotation tables (host) against their formulas, and the refusals of
the calls that norm and rotate: all checked before anything is launched."""

import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest

from mixed_precision_bit_gb300 import kitty as K

# 2 pi to 40 digits
TWO_PI = Fraction(6283185307179586476925286766559005768394, 10 ** 39)


@pytest.fixture(scope="module")
def lib():
    return K.load()


@pytest.mark.parametrize("rot", [2, 16, 96, 128])
def test_plain_and_linear_frequencies(lib, rot):
    f, amp = K.rope_frequencies(rot, 10000.0)
    ref = [10000.0 ** (-2.0 * j / rot) for j in range(rot // 2)]
    assert amp == 1.0 and np.allclose(f, ref, rtol=1e-14, atol=0)
    g, amp = K.rope_frequencies(rot, 10000.0, K.ROPE_LINEAR, factor=8.0)
    assert amp == 1.0 and np.allclose(g, f / 8, rtol=1e-15, atol=0)


def test_ntk_keeps_the_first_pair_and_stretches_the_last(lib):
    f, _ = K.rope_frequencies(128, 10000.0)
    g, amp = K.rope_frequencies(128, 10000.0, K.ROPE_NTK, factor=4.0)
    assert amp == 1.0 and g[0] == 1.0
    assert math.isclose(g[-1], f[-1] / 4, rel_tol=1e-12)  # base' = base * s^(d / (d - 2))
    assert (np.diff(g) < 0).all()


def test_yarn_ramp(lib):
    f, _ = K.rope_frequencies(128, 10000.0)
    g, amp = K.rope_frequencies(128, 10000.0, K.ROPE_YARN, factor=16.0, trained=4096)
    assert math.isclose(amp, 0.1 * math.log(16.0) + 1.0)
    lo = math.floor(128 * math.log(4096 / (2 * math.pi * 32)) / (2 * math.log(10000.0)))
    hi = math.ceil(128 * math.log(4096 / (2 * math.pi * 1)) / (2 * math.log(10000.0)))
    for j in range(64):
        u = min(max((j - lo) / (hi - lo), 0.0), 1.0)
        assert math.isclose(g[j], f[j] * (1 - u) + f[j] / 16 * u, rel_tol=1e-13), j
    assert (g[:lo + 1] == f[:lo + 1]).all() and np.allclose(g[hi:], f[hi:] / 16, rtol=1e-15)


def test_bands(lib):
    f, _ = K.rope_frequencies(128, 500000.0)
    g, amp = K.rope_frequencies(128, 500000.0, K.ROPE_BANDS, factor=8.0, trained=8192, fast=4.0, slow=1.0)
    assert amp == 1.0
    for j in range(64):
        wave = 2 * math.pi / f[j]
        if wave < 8192 / 4.0:
            ref = f[j]
        elif wave > 8192 / 1.0:
            ref = f[j] / 8.0
        else:
            u = (8192 / wave - 1.0) / (4.0 - 1.0)
            ref = (1 - u) * f[j] / 8.0 + u * f[j]
        assert math.isclose(g[j], ref, rel_tol=1e-13), j


def test_factor_one_changes_nothing(lib):
    f, _ = K.rope_frequencies(64, 10000.0)
    for kind in (K.ROPE_LINEAR, K.ROPE_NTK, K.ROPE_YARN, K.ROPE_BANDS):
        g, amp = K.rope_frequencies(64, 10000.0, kind, factor=1.0, trained=2048)
        assert amp == 1.0 and np.allclose(g, f, rtol=1e-14, atol=0)


def test_turns_are_fractions_of_a_turn(lib):
    """turns = f / 2 pi modulo 1, times 2^64: from the double quotient, whose error is
    2^-53 relative, and the last of its own 64 bits."""
    f = np.array([1.0, 1e-3, 1e-7, 6.5, -1.0, 0.0, 123456.789, 2.0 ** -70])
    t = np.zeros(f.size, np.uint64)
    assert lib.kitty_rope_turns(f.ctypes.data, f.size, t.ctypes.data) == 0
    for x, got in zip(f, t):
        q = Fraction(float(x)) / TWO_PI
        err = abs(Fraction(int(got)) - (q % 1) * 2 ** 64)
        err = min(err, 2 ** 64 - err)  # around a whole turn
        assert err <= abs(q) * 2 ** (64 - 52) + 1, x


def test_frequency_refusals(lib):
    for args in ((0, 1e4), (130, 1e4), (15, 1e4), (64, 1.0), (64, math.inf), (64, math.nan)):
        with pytest.raises(K.KittyError) as e:
            K.rope_frequencies(*args)
        assert e.value.code == -1
    for kw in (dict(kind=5), dict(kind=-1), dict(kind=K.ROPE_LINEAR, factor=0.5),
               dict(kind=K.ROPE_LINEAR, factor=math.nan), dict(kind=K.ROPE_YARN, factor=2.0, trained=0),
               dict(kind=K.ROPE_BANDS, factor=2.0, trained=8192, fast=1.0, slow=1.0),
               dict(kind=K.ROPE_BANDS, factor=2.0, trained=8192, fast=4.0, slow=0.0)):
        with pytest.raises(K.KittyError):
            K.rope_frequencies(64, 1e4, **kw)
    t = np.zeros(1, np.uint64)
    bad = np.array([math.inf])
    assert lib.kitty_rope_turns(bad.ctypes.data, 1, t.ctypes.data) == -1
    assert lib.kitty_rope_turns(None, 1, t.ctypes.data) == -1
    assert lib.kitty_rope_turns(None, 0, None) == 0


# Device addresses that are never used: every call below is refused or empty.
A = 1 << 20


def _rope(**kw):
    d = dict(rot_dim=128, layout=0, amplitude=1.0, eps=1e-6, turns=A, q_weight=None, k_weight=None)
    d.update(kw)
    return K._Rope(*[d[n] for n, _ in K._Rope._fields_])


def _cfg(**kw):
    return K.Config(**{**dict(num_kv_heads=2, num_q_heads=8), **kw}).c()


def _norm(lib, cfg=None, rope=None, q=A, qs=1024, k=A, ks=256, pos=A, n=4, qo=A, qos=1024, ko=A, kos=256):
    return lib.kitty_norm_rope(ctypes.byref(cfg or _cfg()), ctypes.byref(rope or _rope()), q, qs, k, ks,
                               pos, n, qo, qos, ko, kos, None)


def test_norm_rope_refusals(lib):
    assert _norm(lib, n=0) == 0                        # empty: nothing to do
    assert _norm(lib, n=-1) == -1
    assert _norm(lib, cfg=_cfg(head_dim=64)) == -2
    for kw in (dict(pos=None), dict(q=None, k=None), dict(qo=None), dict(ko=None), dict(q=A + 2),
               dict(qo=A + 8), dict(ks=255), dict(ks=260), dict(qs=1016), dict(kos=128), dict(qs=-1024)):
        assert _norm(lib, **kw) == -1, kw
    for kw in (dict(rot_dim=-16), dict(rot_dim=144), dict(layout=2), dict(amplitude=math.inf),
               dict(eps=-1e-6), dict(eps=math.nan), dict(turns=None), dict(turns=A + 4)):
        assert _norm(lib, rope=_rope(**kw)) == -1, kw
    for rot in (8, 20, 120):
        assert _norm(lib, rope=_rope(rot_dim=rot)) == -2, rot


def _append(lib, cfg=None, rope=None, **kw):
    a = dict(q=A, qs=1024, k=A, ks=256, v=A, vs=256, qo=A, qos=1024, tk=A, tv=A, tl=A, rs=None, rq=None,
             rc=None, fl=A, bt=A, mp=4, np=A, pool=A, pp=4, base=None, counted=0, B=2, st=None, stream=None)
    a.update(kw)
    return lib.kitty_append_rope(ctypes.byref(cfg or _cfg()), ctypes.byref(rope or _rope()), *a.values())


def test_append_rope_refusals(lib):
    assert _append(lib, B=0) == 0
    for kw in (dict(B=-1), dict(mp=-1), dict(pp=-1), dict(k=None), dict(v=None), dict(qo=None), dict(tk=None),
               dict(tv=A + 4), dict(tl=None), dict(fl=None), dict(bt=None), dict(np=None), dict(pool=None),
               dict(vs=136), dict(ks=252), dict(q=A + 6)):
        assert _append(lib, **kw) == -1, kw
    assert _append(lib, rope=_rope(rot_dim=24)) == -2
    assert _append(lib, cfg=_cfg(rank_mode=K.RANK_RUNNING)) == -1       # no running statistics
    assert _append(lib, cfg=_cfg(v_bit=4)) == -2


def _append16(lib, cfg=None, rope=None, **kw):
    a = dict(q=A, qs=1024, k=A, ks=256, v=A, vs=256, n=2, qo=A, qos=1024, pool=A, pp=4, bt=A, mp=4, ln=A,
             ids=A, start=None, base=None, counted=0, B=2, st=None, stream=None)
    a.update(kw)
    return lib.kitty_f16kv_append_rope(ctypes.byref(cfg or _cfg()), ctypes.byref(rope or _rope()), *a.values())


def test_f16kv_append_rope_refusals(lib):
    assert _append16(lib, B=0, n=0) == 0
    assert _append16(lib, n=0, start=A) == 0
    for kw in (dict(n=3), dict(n=-1, start=A), dict(B=-1), dict(pool=None), dict(pool=A + 8), dict(bt=None),
               dict(ln=None), dict(ids=None), dict(k=None), dict(v=None), dict(qo=None), dict(qs=8),
               dict(vs=264 + 4)):
        assert _append16(lib, **kw) == -1, kw
    assert _append16(lib, rope=_rope(rot_dim=40)) == -2


class _OnDevice:
    """A host tensor that claims to be on a device: the checks read shapes and strides only."""

    def __init__(self, t, dev=0):
        self._t, self._dev = t, dev

    def __getattr__(self, name):
        return getattr(self._t, name)

    is_cuda = True

    def get_device(self):
        return self._dev

    @property
    def device(self):
        return "cuda:%d" % self._dev


def test_rows_of_the_binding_are_checked():
    import torch
    x = torch.zeros(3, 20, 128, dtype=torch.int16)
    rows = lambda t, n, h, dev=0: K._rows(_OnDevice(t), n, h, dev)  # noqa: E731
    assert rows(x, 3, 20)[1] == 20 * 128
    assert rows(x[:, 4:6], 3, 2)[1] == 20 * 128           # a slice of a joint projection
    assert rows(x[:1, 4:6], 1, 2)[1] == 2 * 128
    assert K._rows(None, 3, 2, 0) == (None, 0)
    for bad in (x[:, ::2], x.float()[:, :10], x[0], x.transpose(1, 2), x[:, :3], x[:2, :10]):
        with pytest.raises(ValueError):
            rows(bad, 3, 10)
    with pytest.raises(ValueError):
        rows(x, 3, 20, 1)                                 # another device than the current one
    with pytest.raises(ValueError):
        K._rows(x, 3, 20, 0)                              # host memory
    for bad, n in ((torch.zeros(3, dtype=torch.int64), 3), (torch.zeros(3), 3), (torch.zeros(2, dtype=torch.int32), 3)):
        with pytest.raises(ValueError):
            K._ints("positions", _OnDevice(bad), n, 0)
    with pytest.raises(ValueError):
        K._dense(_OnDevice(x[:, 4:6]), 0)


def test_config_reference_follows_its_fields():
    cfg = K.Config(num_kv_heads=2, num_q_heads=8)
    first = cfg.ref()
    assert cfg.ref() is first
    cfg.n_hi = 16
    assert cfg.ref() is not first and cfg.ref()._obj.n_hi == 16


def test_rope_reference_follows_its_fields():
    """A weight that is replaced, or whose memory moves, is the one that calls get."""
    import torch
    weights = [_OnDevice(torch.ones(128, dtype=torch.bfloat16) * i) for i in range(3)]
    rope = K.Rope(K.rope_frequencies(64)[0], q_weight=weights[0], device="cpu")
    rope.turns = _OnDevice(rope.turns)
    first = rope.ref(0)
    assert rope.ref(0) is first and first._obj.q_weight == weights[0].data_ptr() and first._obj.k_weight is None
    rope.q_weight = weights[1]
    assert rope.ref(0)._obj.q_weight == weights[1].data_ptr()
    rope.k_weight = weights[0]
    assert rope.ref(0)._obj.k_weight == weights[0].data_ptr()
    weights[1]._t.data = torch.zeros(128, dtype=torch.bfloat16)
    assert rope.ref(0)._obj.q_weight == weights[1].data_ptr()
    rope.amplitude, rope.eps, rope.layout, rope.rot_dim = 0.5, 0.25, K.ROPE_INTERLEAVED, 32
    c = rope.ref(0)._obj
    assert (c.amplitude, c.eps, c.layout, c.rot_dim) == (0.5, 0.25, 1, 32)
    rope.q_weight = None
    assert rope.ref(0)._obj.q_weight is None
    # what a later assignment may not be
    for name, bad in (("q_weight", _OnDevice(torch.zeros(64, dtype=torch.int16))), ("k_weight", _OnDevice(torch.zeros(128))),
                      ("q_weight", torch.zeros(128, dtype=torch.int16)), ("rot_dim", 66),
                      ("q_weight", _OnDevice(torch.zeros(256, dtype=torch.int16)[::2])),
                      ("k_weight", _OnDevice(torch.zeros(128, dtype=torch.int16), 1))):
        keep = getattr(rope, name)
        setattr(rope, name, bad)
        with pytest.raises(ValueError):
            rope.ref(0)
        setattr(rope, name, keep)
    rope.ref(0)
    with pytest.raises(ValueError):
        rope.ref(1)                                       # another device is current
    # one table kept alive by the structure's owner: no reference into a freed object
    import copy
    again = copy.copy(rope)
    again.eps = 0.5
    assert rope.ref(0)._obj.eps == 0.25 and again.ref(0)._obj.eps == 0.5


def test_rows_of_the_other_16_bit_type_are_refused():
    import torch
    bf, h, raw = (torch.zeros(3, 2, 128, dtype=t) for t in (torch.bfloat16, torch.float16, torch.int16))
    for own, other, dt in ((bf, h, K.BF16), (h, bf, K.F16)):
        K._rows(_OnDevice(own), 3, 2, 0, dt)
        K._rows(_OnDevice(raw), 3, 2, 0, dt)              # the bits, as the caches hold them
        cfg = K.Config(num_kv_heads=1, num_q_heads=2, in_dtype=dt)
        out = _OnDevice(torch.zeros(3, 2, 128))
        K._attended(cfg, _OnDevice(own), out, 3, 0)
        with pytest.raises(ValueError, match="configuration has"):
            K._rows(_OnDevice(other), 3, 2, 0, dt)
        with pytest.raises(ValueError, match="configuration has"):
            K._attended(cfg, _OnDevice(other), out, 3, 0)
        rope = K.Rope(K.rope_frequencies(64)[0], q_weight=_OnDevice(own[0, 0]), device="cpu")
        rope.turns = _OnDevice(rope.turns)
        rope.ref(0, dt)
        with pytest.raises(ValueError, match="configuration has"):
            rope.ref(0, K.F16 + K.BF16 - dt)              # the same weights under the other configuration
        rope.k_weight = _OnDevice(other[0, 0])
        with pytest.raises(ValueError, match="configuration has"):
            rope.ref(0, dt)


def test_calls_pass_their_configuration_s_type():
    """Every binding of rows refuses the other type before it launches (the other arguments are
    on the device that is asked for)."""
    import torch
    from unittest import mock
    z = lambda *s, t=torch.int32: _OnDevice(torch.zeros(s, dtype=t))  # noqa: E731
    rows = lambda h, t=torch.bfloat16: _OnDevice(torch.zeros(3, h, 128, dtype=t))  # noqa: E731
    cfg = K.Config(num_kv_heads=1, num_q_heads=2, in_dtype=K.BF16)
    rope = K.Rope(K.rope_frequencies(64)[0], device="cpu")
    rope.turns = z(32, t=torch.int64)
    tail = lambda B=3, t=torch.int16: z(B, 1, 32, 128, t=t)  # noqa: E731
    good = dict(q=rows(2), k=rows(1), v=rows(1), qo=rows(2), ko=rows(1), qw=None)

    class Lib:
        def __getattr__(self, name):
            return lambda *a: 0

    def calls(q, k, v, qo, ko, qw):
        rope.q_weight = qw
        yield lambda: K.norm_rope(cfg, rope, q, k, z(3), qo, ko, stream=0)
        yield lambda: K.append_rope(cfg, rope, q, k, v, qo, tail(), tail(), z(3), None, None, None, z(3), z(3, 2), z(3),
                                    z(8), 1, stream=0)
        yield lambda: K.f16kv_append_rope(cfg, rope, q, k, v, qo, z(8), 1, z(3, 2), z(3), z(3), stream=0)

    with mock.patch.object(K, "_device", lambda: 0), mock.patch.object(K, "load", Lib):
        for call in calls(**good):
            call()
        for name in good:
            bad = _OnDevice(torch.zeros(128, dtype=torch.float16)) if name == "qw" else \
                rows(2 if name in ("q", "qo") else 1, torch.float16)
            for i, call in enumerate(calls(**{**good, name: bad})):
                if (name, i) in (("v", 0), ("ko", 1), ("ko", 2)):
                    continue                              # not an argument of that call
                with pytest.raises(ValueError, match="configuration has"):
                    call()
        for bad in (tail(2), tail(t=torch.float16), tail(t=torch.int32)):
            for tails in ((bad, tail()), (tail(), bad)):
                rope.q_weight = None
                with pytest.raises(ValueError):
                    K.append_rope(cfg, rope, None, good["k"], good["v"], None, *tails, z(3), None, None, None, z(3),
                                  z(3, 2), z(3), z(8), 1, stream=0)
                with pytest.raises(ValueError):
                    K.decode_attention_shared(cfg, good["q"], z(8), 1, z(1), None, z(3, 2), z(3), *tails, z(3), 1.0,
                                              rows(2), stream=0)
