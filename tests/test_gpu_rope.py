"""Norm and rotation of queries and keys, alone and on the way into both caches, on the
GPU against a plain evaluation in 64 bits.

Tolerance of a computed element, from the roundings: one to the 16-bit output (eps / 2 of
the value, or half of the smallest subnormal), and the fp32 evaluation: the norm's 128-term
sum and its root, the sine and cosine (2 ulp and an angle to 2^-32 of a turn) and two
products, under 16 roundings of 2^-24 on terms no larger than the pair's: 2^-20 of
amplitude * (|a| + |b|), a and b the normed pair."""

import dataclasses

import numpy as np
import pytest

from mixed_precision_bit_gb300 import synth
from tests.kitty_cases import dev32

pytestmark = pytest.mark.gpu
P, D = 32, 128
BF16, F16 = synth.BF16, synth.F16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixed_precision_bit_gb300 import kitty
    kitty.load()


def _dt(dt):
    import torch
    return torch.bfloat16 if dt == BF16 else torch.float16


def _cfg(Hkv, Hq, dt, **kw):
    from mixed_precision_bit_gb300 import kitty
    return kitty.Config(num_kv_heads=Hkv, num_q_heads=Hq, in_dtype=dt, **kw)


def _rows(n, H, dt, seed, gap=0):
    """[n, H, 128] rows as a slice of wider rows (gap more heads a token)."""
    import torch
    x = torch.from_numpy(np.random.default_rng(seed).standard_normal((n, H + gap, D)) * 2).to(_dt(dt)).cuda()
    return x[:, gap // 2:gap // 2 + H]


def _rope(rot, layout, dt, norms, seed=3, amplitude=1.0, base=10000.0):
    import torch
    from mixed_precision_bit_gb300 import kitty
    r = np.random.default_rng(seed)
    w = [torch.from_numpy(1 + 0.2 * r.standard_normal(D)).to(_dt(dt)).cuda() if c in norms else None for c in "qk"]
    f = kitty.rope_frequencies(rot, base)[0] if rot else np.zeros(0)
    return kitty.Rope(f, layout=layout, amplitude=amplitude, q_weight=w[0], k_weight=w[1], eps=1e-5), f


def _turned(x, f, pos, layout, amplitude, weight, eps=1e-5):
    """(y, tolerance before the output's rounding) in 64 bits; x [n, H, 128] float64."""
    n, H, _ = x.shape
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    y, tol = x.copy(), 2.0 ** -20 * np.abs(x)
    h = f.size
    if h:
        ang = np.fmod(pos.astype(np.longdouble)[:, None] * f.astype(np.longdouble),
                      2 * np.arccos(np.longdouble(-1))).astype(np.float64)
        c, s = amplitude * np.cos(ang)[:, None], amplitude * np.sin(ang)[:, None]
        ia, ib = (np.arange(h), np.arange(h) + h) if layout == 0 else (2 * np.arange(h), 2 * np.arange(h) + 1)
        a, b = x[..., ia], x[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        # the table's own last bit: 2^-53 of the quotient f / 2 pi, times the position
        m = amplitude * (np.abs(a) + np.abs(b)) * (2.0 ** -20 + (np.abs(pos)[:, None] * f * 2.0 ** -52)[:, None])
        tol[..., ia], tol[..., ib] = m, m
    return y, tol


def _check(got, ref, tol, dt):
    import torch
    fi = torch.finfo(_dt(dt))
    g = got.double().cpu().numpy()
    bound = tol + np.maximum(fi.eps / 2 * (np.abs(ref) + tol), fi.smallest_normal * fi.eps / 2)
    bad = ~(np.abs(g - ref) <= bound)
    assert not bad.any(), "%d of %d off, worst %.3g of its bound" % (
        bad.sum(), bad.size, np.nanmax(np.abs(g - ref) / bound))


POS = np.array([0, 1, -1, 7, 31, 32, 4095, 8192, 131071, 1 << 24, -(1 << 20), 2 ** 31 - 1, -2 ** 31, 5, 9, 77, 1000])
CASES = [  # Hkv, Hq, rot, layout, norms, amplitude, gap
    (2, 8, 128, 0, "qk", 1.0, 0),
    (8, 32, 128, 0, "qk", 1.0, 16),
    (1, 1, 64, 1, "", 1.0, 0),
    (5, 5, 32, 0, "q", 1.25, 2),
    (3, 6, 96, 1, "k", 0.75, 1),
    (1, 7, 16, 0, "qk", 1.0, 3),
    (8, 64, 128, 1, "", 1.0, 8),
    (2, 4, 0, 0, "qk", 1.0, 0),       # norms alone
]


@pytest.mark.parametrize("dt", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("case", CASES, ids=["c%d" % i for i in range(len(CASES))])
@pytest.mark.parametrize("n", [1, 17])
def test_norm_rope_matches_64_bits(case, dt, n):
    import torch
    from mixed_precision_bit_gb300 import kitty
    Hkv, Hq, rot, layout, norms, amp, gap = case
    rope, f = _rope(rot, layout, dt, norms, amplitude=amp)
    q, k = _rows(n, Hq, dt, 1, gap), _rows(n, Hkv, dt, 2, gap)
    pos = POS[-n:] if n == 1 else POS[:n]
    qo, ko = (torch.full((n, H, D), float("nan"), dtype=_dt(dt), device="cuda") for H in (Hq, Hkv))
    kitty.norm_rope(_cfg(Hkv, Hq, dt), rope, q, k, dev32(pos), qo, ko)
    for x, y, w in ((q, qo, rope.q_weight), (k, ko, rope.k_weight)):
        wn = None if w is None else w.double().cpu().numpy()
        _check(y, *_turned(x.double().cpu().numpy(), f, pos, layout, amp, wn), dt)
    # only queries, only keys: the same rows
    q1, k1 = torch.empty_like(qo), torch.empty_like(ko)
    kitty.norm_rope(_cfg(Hkv, Hq, dt), rope, q, None, dev32(pos), q1, None)
    kitty.norm_rope(_cfg(Hkv, Hq, dt), rope, None, k, dev32(pos), None, k1)
    assert torch.equal(q1.view(torch.int16), qo.view(torch.int16))
    assert torch.equal(k1.view(torch.int16), ko.view(torch.int16))
    # in place
    kitty.norm_rope(_cfg(Hkv, Hq, dt), rope, q, k, dev32(pos), q, k)
    assert torch.equal(q.contiguous().view(torch.int16), qo.view(torch.int16))
    assert torch.equal(k.contiguous().view(torch.int16), ko.view(torch.int16))


def test_norm_rope_many_tokens_and_neighbours_untouched():
    """More tokens than any block count of a small grid, in place in the middle of joint rows."""
    import torch
    from mixed_precision_bit_gb300 import kitty
    n, Hkv, Hq = 4099, 1, 2
    x = torch.randn(n, 6, D, device="cuda").to(torch.bfloat16)
    ref = x.clone()
    rope, f = _rope(128, 0, BF16, "qk")
    pos = np.arange(n) * 31 % 5003
    kitty.norm_rope(_cfg(Hkv, Hq, BF16), rope, x[:, 1:3], x[:, 4:5], dev32(pos), x[:, 1:3], x[:, 4:5])
    for i in (0, 3, 5):
        assert torch.equal(x[:, i].view(torch.int16), ref[:, i].view(torch.int16))
    for sl, w in ((slice(1, 3), rope.q_weight), (slice(4, 5), rope.k_weight)):
        _check(x[:, sl], *_turned(ref[:, sl].double().cpu().numpy(), f, pos, 0, 1.0, w.double().cpu().numpy()), BF16)


def test_non_finite_rows_stay_in_their_rows():
    import torch
    from mixed_precision_bit_gb300 import kitty
    q, k = _rows(3, 4, F16, 5), _rows(3, 2, F16, 6)
    q[1, 2, 3], q[0, 1, 100], k[2, 0, 5] = float("nan"), float("inf"), float("-inf")
    rope, f = _rope(64, 0, F16, "")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    kitty.norm_rope(_cfg(2, 4, F16), rope, q, k, dev32([3, 4, 5]), qo, ko)
    bad = ~torch.isfinite(qo)
    assert bad.sum() == 3 and bad[1, 2, 3] and bad[1, 2, 35]
    assert qo[0, 1, 100] == float("inf")               # past the rotated channels: passed through
    assert torch.equal(~torch.isfinite(ko), torch.zeros_like(ko, dtype=torch.bool).index_put_(
        (torch.tensor([2, 2]), torch.tensor([0, 0]), torch.tensor([5, 37])), torch.tensor(True)))


# ------------------------------------------------------------------ 16-bit cache
def _cache16(B, Hkv, Hq, dt, max_pages, lens, seed):
    """An empty pool, block table and lengths of a cache that already holds `lens` tokens."""
    import torch
    from mixed_precision_bit_gb300 import kitty
    cfg = _cfg(Hkv, Hq, dt)
    pool_pages = B * max_pages + 1
    ids = np.random.default_rng(seed).permutation(pool_pages).astype(np.int32)
    bt = np.full((B, max_pages), -1, np.int32)
    used = 0
    for b, L in enumerate(lens):
        n = (L + P - 1) // P
        bt[b, :n] = ids[used:used + n]
        used += n
    pool = torch.randint(-2000, 2000, (pool_pages, Hkv, 2, P, D), dtype=torch.int16, device="cuda")
    assert kitty.f16kv_page_bytes(cfg)[1] == pool[0].numel() * 2
    return cfg, pool, pool_pages, bt, list(ids[used:])


def test_f16kv_append_rope_one_token_equals_separate_calls():
    """Step by step: the pool, table and lengths of norm_rope then f16kv_append, bit for bit."""
    import torch
    from mixed_precision_bit_gb300 import kitty
    lens, Hkv, Hq, dt = [30, 0, 64, 5, 31], 2, 8, BF16
    B = len(lens)
    cfg, pool, pool_pages, bt, free = _cache16(B, Hkv, Hq, dt, 4, lens, 1)
    rope, _ = _rope(128, 0, dt, "qk")
    base = dev32([0, 100, 7, 0, 64])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    a = dict(pool=pool.clone(), bt=dev32(bt), ln=dev32(lens))
    c = dict(pool=pool.clone(), bt=dev32(bt), ln=dev32(lens))
    h = np.array(lens)
    for step in range(40):
        x = _rows(B, Hq + 2 * Hkv, dt, 100 + step)
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        new = dev32([free.pop() if n % P == 0 else -1 for n in h])
        q1, q2, k2 = torch.empty_like(q.contiguous()), torch.empty_like(q.contiguous()), torch.empty_like(k.contiguous())
        pos = a["ln"] + base
        kitty.f16kv_append_rope(cfg, rope, q, k, v, q1, c["pool"], pool_pages, c["bt"], c["ln"], new,
                                pos_base=base, status=st)
        kitty.norm_rope(cfg, rope, q, k, pos, q2, k2)
        kitty.f16kv_append(cfg, k2, v.contiguous(), a["pool"], pool_pages, a["bt"], a["ln"], new, status=st)
        assert torch.equal(q1.view(torch.int16), q2.view(torch.int16)), step
        # layers that share the lengths: counted, into a pool of their own, nothing advanced
        other, before = pool.clone(), (c["bt"].clone(), c["ln"].clone())
        kitty.f16kv_append_rope(cfg, rope, None, k, v, None, other, pool_pages, c["bt"], c["ln"], None,
                                pos_base=base, counted=True, status=st)
        assert torch.equal(before[0], c["bt"]) and torch.equal(before[1], c["ln"])
        for b in range(B):
            pid, slot = int(c["bt"][b, h[b] // P]), h[b] % P
            assert torch.equal(other[pid, :, :, slot], c["pool"][pid, :, :, slot])
        h += 1
        for n in ("pool", "bt", "ln"):
            assert torch.equal(a[n], c[n]), (step, n)
    assert int(st.item()) == 0


@pytest.mark.parametrize("dt", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("new", [[5, 0, 70, 1, 33], [1, 1, 1, 1, 1], [0, 0, 0, 0, 96], [32, 64, 2, 31, 40]],
                         ids=["ragged", "ones", "last", "pages"])
@pytest.mark.parametrize("pad", [0, 3])
def test_f16kv_append_rope_ragged(new, pad, dt):
    import torch
    from mixed_precision_bit_gb300 import kitty
    lens, Hkv, Hq = [30, 0, 33, 64, 0], 2, 6
    B, n = len(lens), sum(new) + pad
    cfg, pool, pool_pages, bt, free = _cache16(B, Hkv, Hq, dt, 5, lens, 2)
    rope, f = _rope(64, 1, dt, "k")
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    ids = np.full(n, -7, np.int32)                      # entries of other tokens are ignored
    pos, where, want_bt = np.zeros(n, np.int64), {}, bt.copy()
    for b in range(B):
        for i in range(new[b]):
            t, p = start[b] + i, lens[b] + i
            if p % P == 0:
                ids[t] = want_bt[b, p // P] = free.pop()
            pos[t] = p
            where[t] = (int(want_bt[b, p // P]), p % P)
    q, k, v = _rows(n, Hq, dt, 3, 2), _rows(n, Hkv, dt, 4, 3), _rows(n, Hkv, dt, 5)
    qo = torch.full((n, Hq, D), 7.0, dtype=_dt(dt), device="cuda")
    q2, k2 = torch.empty_like(qo), torch.empty_like(v.contiguous())
    kitty.norm_rope(cfg, rope, q, k, dev32(pos), q2, k2)
    want = pool.clone()
    for t, (pid, slot) in where.items():
        want[pid, :, 0, slot], want[pid, :, 1, slot] = k2[t].view(torch.int16), v[t].view(torch.int16)
    q2[sum(new):] = 7.0
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    d_bt, d_ln = dev32(bt), dev32(lens)
    args = (cfg, rope, q, k, v, qo, pool, pool_pages, d_bt, d_ln, dev32(ids))
    kitty.f16kv_append_rope(*args, seq_start=dev32(start), status=st)
    assert int(st.item()) == 0
    assert torch.equal(pool, want)
    assert torch.equal(qo.view(torch.int16), q2.view(torch.int16))
    assert np.array_equal(d_bt.cpu().numpy(), want_bt)
    assert np.array_equal(d_ln.cpu().numpy(), np.array(lens) + new)
    # again, counted: the same places
    pool.zero_()
    kitty.f16kv_append_rope(*args, seq_start=dev32(start), counted=True, status=st)
    for t, (pid, slot) in where.items():
        assert torch.equal(pool[pid, :, :, slot], want[pid, :, :, slot])
    assert np.array_equal(d_ln.cpu().numpy(), np.array(lens) + new) and int(st.item()) == 0


def test_f16kv_append_rope_refused_sequences():
    """A sequence without room, a bad length, a bad page: reported and not advanced; the others
    are appended."""
    import torch
    from mixed_precision_bit_gb300 import kitty
    Hkv, Hq, dt, B = 1, 2, BF16, 4
    rope, _ = _rope(32, 0, dt, "")
    for lens, new, bad_at, code in (([0, 60, 3, 3], [2, 5, 2, 2], None, 8),     # TABLE_FULL
                                    ([0, -1, 3, 3], [2, 5, 2, 2], None, 5),     # BAD_LEN
                                    ([0, 65, 3, 3], [2, 5, 2, 2], None, 5),
                                    ([0, 0, 3, 3], [2, 40, 2, 2], 2 + 32, 4)):  # BAD_PAGE in its second page
        cfg, pool, pool_pages, bt, free = _cache16(B, Hkv, Hq, dt, 2, [max(min(x, 64), 0) for x in lens], 5)
        start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        n = int(start[-1])
        ids = np.full(n, -1, np.int32)
        for b in range(B):
            for i in range(new[b]):
                if (lens[b] + i) % P == 0 and lens[b] >= 0:
                    ids[start[b] + i] = free.pop() if free else -1
        if bad_at is not None:
            ids[bad_at] = pool_pages
        x = _rows(n, Hq + 2 * Hkv, dt, 6)
        qo = torch.zeros(n, Hq, D, dtype=torch.bfloat16, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        d_ln = dev32(lens)
        kitty.f16kv_append_rope(cfg, rope, x[:, :Hq], x[:, Hq:Hq + 1], x[:, Hq + 1:], qo, pool, pool_pages,
                                dev32(bt), d_ln, dev32(ids), seq_start=dev32(start), status=st)
        assert int(st.item()) == code
        assert d_ln.tolist() == [2, lens[1], 5, 5]
        if bad_at is None:
            assert (qo[start[1]:start[2]] == 0).all()
        assert (qo[start[2]:] != 0).any(-1).all()
    # starts out of order: every access stays inside, the code says so
    cfg, pool, pool_pages, bt, free = _cache16(B, Hkv, Hq, dt, 2, [0] * B, 5)
    st.zero_()
    d_ln = dev32([0] * B)
    x = _rows(8, Hq + 2 * Hkv, dt, 6)
    kitty.f16kv_append_rope(cfg, rope, x[:, :Hq], x[:, Hq:Hq + 1], x[:, Hq + 1:], qo[:8].contiguous(), pool, pool_pages,
                            dev32(bt), d_ln, dev32([-1] * 8), seq_start=dev32([0, 6, 4, 9, 20]), status=st)
    assert int(st.item()) in (4, 9)


# ------------------------------------------------------------------ packed cache
def _packed(B, Hkv, Hq, dt, max_pages, seed, rank, **kw):
    import torch
    from mixed_precision_bit_gb300 import kitty
    cfg = _cfg(Hkv, Hq, dt, rank_mode=rank, **kw)
    pool_pages = B * max_pages
    r = np.random.default_rng(seed)
    tail = torch.from_numpy(r.standard_normal((2, B, Hkv, P, D))).to(_dt(dt)).cuda()
    s = dict(tail_k=tail[0].clone(), tail_v=tail[1].clone(), run_sum=torch.zeros(B, Hkv, D, device="cuda"),
             run_sumsq=torch.zeros(B, Hkv, D, device="cuda"),
             run_count=torch.zeros(B, Hkv, dtype=torch.int32, device="cuda"),
             pool=torch.zeros(pool_pages * kitty.page_bytes(cfg)[1], dtype=torch.uint8, device="cuda"))
    return cfg, pool_pages, s


FORMATS = [dict(n_hi=32), dict(n_hi=0), dict(n_hi=48, hi_bit=8, lo_bit=4), dict(n_hi=16, hi_bit=8, lo_bit=4, v_bit=4)]


@pytest.mark.parametrize("fmt", FORMATS, ids=["42", "2", "84", "84v4"])
@pytest.mark.parametrize("dt", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("rank", [0, 1], ids=["page", "running"])
def test_append_rope_equals_separate_calls(fmt, dt, rank):
    """Through two flushes of every sequence: tails, lengths, tables, statistics and pages of
    norm_rope then append_token, bit for bit; and of a counted append that follows it."""
    import torch
    from mixed_precision_bit_gb300 import kitty
    B, Hkv, Hq, max_pages = 3, 2, 6, 4
    cfg, pool_pages, s0 = _packed(B, Hkv, Hq, dt, max_pages, 11, rank, **fmt)
    rope, _ = _rope(96, 0, dt, "qk", amplitude=1.1)
    tl, npg = np.array([0, 30, 17]), np.array([0, 1, 0])
    new = lambda: {n: x.clone() for n, x in s0.items()}  # noqa: E731
    lens = lambda: dict(tail_len=dev32(tl), num_pages=dev32(npg), block_table=dev32(np.full((B, max_pages), -1)))  # noqa: E731
    a, c, o = dict(new(), **lens()), dict(new(), **lens()), new()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    base = dev32([0, 5, 1000])
    h_t, h_p, next_id = tl.copy(), npg.copy(), 0
    run = lambda s: (s["run_sum"], s["run_sumsq"], s["run_count"]) if rank else (None, None, None)  # noqa: E731
    for step in range(66):
        x = _rows(B, Hq + 2 * Hkv, dt, 200 + step)
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        fl = np.full(B, -1)
        for b in range(B):
            if h_t[b] == 31 and h_p[b] < max_pages:
                fl[b], next_id = next_id, next_id + 1
        flush = dev32(fl)
        q1, q2, k2 = (torch.empty(B, H, D, dtype=x.dtype, device="cuda") for H in (Hq, Hq, Hkv))
        kitty.norm_rope(cfg, rope, q, k, base + 32 * a["num_pages"] + a["tail_len"], q2, k2)
        kitty.append_token(cfg, k2, v.contiguous(), a["tail_k"], a["tail_v"], a["tail_len"], *run(a), flush,
                           a["block_table"], a["num_pages"], a["pool"], pool_pages, status=st)
        kitty.append_rope(cfg, rope, q, k, v, q1, c["tail_k"], c["tail_v"], c["tail_len"], *run(c), flush,
                          c["block_table"], c["num_pages"], c["pool"], pool_pages, pos_base=base, status=st)
        kept = [c[n].clone() for n in ("tail_len", "num_pages", "block_table")]
        kitty.append_rope(cfg, rope, None, k, v, None, o["tail_k"], o["tail_v"], c["tail_len"], *run(o), flush,
                          c["block_table"], c["num_pages"], o["pool"], pool_pages, pos_base=base, counted=True,
                          status=st)
        assert all(torch.equal(x, c[n]) for x, n in zip(kept, ("tail_len", "num_pages", "block_table")))
        assert torch.equal(q1.view(torch.int16), q2.view(torch.int16)), step
        for n in a:
            assert torch.equal(a[n].view(torch.uint8), c[n].view(torch.uint8)), (step, n)
            if n in o:
                assert torch.equal(a[n].view(torch.uint8), o[n].view(torch.uint8)), (step, n, "counted")
        for b in range(B):
            h_t[b] += 1
            if fl[b] >= 0:
                h_t[b], h_p[b] = 0, h_p[b] + 1
    assert int(st.item()) == 0 and next_id >= 6


def test_append_rope_refused_sequences():
    import torch
    from mixed_precision_bit_gb300 import kitty
    B, Hkv, Hq, dt, max_pages = 3, 1, 2, BF16, 2
    rope, _ = _rope(128, 0, dt, "")
    for tl, npg, fl, code, after in (((3, 32, 1), (0, 0, 0), (-1, -1, -1), 6, (4, 32, 2)),   # TAIL_FULL
                                     ((3, 33, 1), (0, 0, 0), (-1, -1, -1), 5, (4, 33, 2)),   # BAD_LEN
                                     ((3, 4, 1), (0, 3, 0), (-1, -1, -1), 5, (4, 4, 2)),     # num_pages past the table
                                     ((3, 4, 1), (0, -1, 0), (-1, -1, -1), 5, (4, 4, 2)),
                                     ((3, 4, 1), (0, 0, 0), (-1, 1, -1), 7, (4, 5, 2)),      # BAD_FLUSH
                                     ((3, 31, 1), (0, 2, 0), (-1, 1, -1), 8, (4, 32, 2)),    # TABLE_FULL
                                     ((3, 31, 1), (0, 0, 0), (-1, 99, -1), 4, (4, 32, 2))):  # BAD_PAGE
        cfg, pool_pages, s = _packed(B, Hkv, Hq, dt, max_pages, 12, 0)
        x = _rows(B, Hq + 2 * Hkv, dt, 8)
        qo = torch.zeros(B, Hq, D, dtype=torch.bfloat16, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        d_tl, d_np, bt = dev32(tl), dev32(npg), dev32(np.full((B, max_pages), -1))
        kitty.append_rope(cfg, rope, x[:, :Hq], x[:, Hq:Hq + 1], x[:, Hq + 1:], qo, s["tail_k"], s["tail_v"],
                          d_tl, None, None, None, dev32(fl), bt, d_np, s["pool"], pool_pages, status=st)
        assert int(st.item()) == code and tuple(d_tl.tolist()) == after and tuple(d_np.tolist()) == npg
        assert (qo[0] != 0).any() and (qo[2] != 0).any()
        if code in (5, 6):
            assert (qo[1] == 0).all()
        assert (s["pool"] == 0).all() and (bt == -1).all()


def test_capture_replay_and_side_stream():
    """The three calls in one graph, replayed on new contents, equal direct calls; a call on a
    side stream is ordered there."""
    import torch
    from mixed_precision_bit_gb300 import kitty
    B, Hkv, Hq, dt, max_pages = 4, 2, 8, BF16, 3
    rope, _ = _rope(128, 0, dt, "qk")
    cfg, pool_pages, s = _packed(B, Hkv, Hq, dt, max_pages, 13, 1)
    x = _rows(B, Hq + 2 * Hkv, dt, 20).contiguous()
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    qo = torch.empty(B, Hq, D, dtype=x.dtype, device="cuda")
    fl = dev32([-1] * B)
    state = dict(s, tail_len=dev32([28, 0, 31, 5]), num_pages=dev32([0, 0, 1, 0]),
                 block_table=dev32(np.full((B, max_pages), -1)))

    def call(stream=None):
        kitty.append_rope(cfg, rope, q, k, v, qo, state["tail_k"], state["tail_v"], state["tail_len"],
                          state["run_sum"], state["run_sumsq"], state["run_count"], fl, state["block_table"],
                          state["num_pages"], state["pool"], pool_pages, stream=stream)
    start = {n: t.clone() for n, t in state.items()}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    assert all(torch.equal(state[n], start[n]) for n in state)  # capturing runs nothing
    inputs = [_rows(B, Hq + 2 * Hkv, dt, 30 + i).contiguous() for i in range(5)]
    flushes = [[-1, -1, 0, -1], [-1] * 4, [-1] * 4, [1, -1, -1, -1], [-1] * 4]
    outs = []
    for y, f in zip(inputs, flushes):
        x.copy_(y)
        fl.copy_(dev32(f))
        g.replay()
        outs.append(qo.clone())
    end = {n: t.clone() for n, t in state.items()}
    for n, t in start.items():
        state[n].copy_(t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for y, f, o in zip(inputs, flushes, outs):
            x.copy_(y)
            fl.copy_(dev32(f))
            call(side)
            assert torch.equal(qo.view(torch.int16), o.view(torch.int16))
    torch.cuda.synchronize()
    for n in state:
        assert torch.equal(state[n].view(torch.uint8), end[n].view(torch.uint8)), n
