"""Edges of the shared-prefix calls and of the calls with norms and rotation, on the GPU, that
the cases by size do not reach.  Tolerances as in test_gpu_shared.py and test_gpu_rope.py."""

import numpy as np
import pytest

from mixed_precision_bit_gb300 import synth
from tests import test_gpu_rope as rope_cases
from tests.kitty_cases import attn_error, dev32
from tests.shared_cases import D, Packed, Plain16

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


def _own(kind, n):
    """n sequences' own tokens."""
    if kind is Packed:
        return dict(own=[i % 3 for i in range(n)], tails=[(7 * i + 1) % 32 for i in range(n)])
    return dict(lens=[(29 * i + 1) % 90 for i in range(n)])


@pytest.mark.parametrize("kind", [Packed, Plain16])
@pytest.mark.parametrize("sm", [-0.05, 0.0, 0.3])
def test_scales(kind, sm):
    """A negative scale (the smallest products win), none (the mean of the Values), a large one:
    scores of up to |s| are formed in fp32, 2^-22 |s| off, which shifts a probability by that."""
    c = kind(Hkv=2, Hq=8, dt=BF16, n_prefix=30, shared=[30, 29, 7, 0], seed=30, **_own(kind, 4))
    c.sm = sm
    st = _status()
    got = c.run("f32", st)
    ref, ost = c.oracle()
    assert int(st.item()) == ost == 0
    assert attn_error(got, ref)[0] <= 0


@pytest.mark.parametrize("kind", [Packed, Plain16])
@pytest.mark.parametrize("n,Hkv,Hq,B", [(997, 1, 1, 1), (1021, 1, 4, 3), (514, 2, 2, 150), (401, 4, 128, 3),
                                         (401, 4, 16, 3)])
def test_long_prefixes_over_many_splits(kind, n, Hkv, Hq, B):
    """One row to several blocks of them, splits of uneven lengths."""
    r = np.random.default_rng(n)
    shared = None if B == 1 else r.integers(0, n + 1, B)
    c = kind(Hkv=Hkv, Hq=Hq, dt=F16, n_prefix=n, shared=shared, seed=31, **_own(kind, B))
    st = _status()
    if kind is Plain16 and Hq // Hkv > 4:              # as kitty_f16kv_decode: groups up to 4
        from mixed_precision_bit_gb300 import kitty
        with pytest.raises(kitty.KittyError, match="UNSUPPORTED"):
            c.run("bf16", st)
        return
    got = c.run("bf16", st)
    ref, ost = c.oracle()
    assert int(st.item()) == ost == 0
    assert attn_error(got, ref, "bf16")[0] <= 0


@pytest.mark.parametrize("kind", [Packed, Plain16])
def test_a_page_twice_in_the_table(kind):
    c = kind(Hkv=2, Hq=8, dt=F16, n_prefix=9, shared=[9, 8], seed=32, **_own(kind, 2))
    c.prefix[:] = c.prefix[[0, 0, 1, 2, 1, 5, 5, 5, 0]]
    c.dev["prefix"].copy_(dev32(c.prefix))
    assert attn_error(c.run("f32"), c.oracle()[0])[0] <= 0


@pytest.mark.parametrize("kind", [Packed, Plain16])
@pytest.mark.parametrize("t", ["float32", "bfloat16"])
def test_outputs_that_are_not_aligned(kind, t):
    import torch
    c = kind(Hkv=1, Hq=3, dt=BF16, n_prefix=7, shared=None, seed=33, **_own(kind, 5))
    n = c.B * c.Hq * D
    whole = torch.full((n + 2,), 7.0, dtype=getattr(torch, t), device="cuda")
    out = whole[1:-1].view(c.B, c.Hq, D)
    assert out.data_ptr() % 16
    c.call(out)
    ref = torch.zeros(c.B, c.Hq, D, dtype=out.dtype, device="cuda")
    c.call(ref)
    assert torch.equal(out, ref) and whole[0] == 7 and whole[-1] == 7


def test_queries_beyond_fp16_are_reported():
    """As by the plain decode: also where a sequence has the prefix alone."""
    import torch
    c = Packed(1, 2, BF16, 5, None, [0, 0], [0, 0], seed=34)
    c.dev["q"].view(torch.bfloat16)[1, 0, 3] = 1e5
    st = _status()
    got = c.run("f32", st)
    assert int(st.item()) == 2
    assert attn_error(got[:1], c.oracle()[0][:1])[0] <= 0


@pytest.mark.parametrize("kind", [Packed, Plain16])
def test_two_calls_at_once(kind):
    """On two streams, a workspace each: the bytes of one after the other."""
    import torch
    cs = [kind(Hkv=2, Hq=8, dt=BF16, n_prefix=200, shared=None, seed=40 + i, **_own(kind, 12)) for i in range(2)]
    want = [torch.empty(c.B, c.Hq, D, device="cuda") for c in cs]
    ws = [c.workspace() for c in cs]
    for c, o, w in zip(cs, want, ws):
        c.call(o, ws=w)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(10):
        outs = [torch.zeros_like(o) for o in want]
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        for c, o, w, s in zip(cs, outs, ws, streams):
            c.call(o, ws=w, stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outs, want))


@pytest.mark.parametrize("gap", [17, 19, 21])
@pytest.mark.parametrize("dt", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("kind", [Packed, Plain16])
def test_one_large_score_before_many_small_ones(kind, dt, gap):
    """The first token's score is `gap` log2 units above 30000 others: each weighs 2^-gap of it,
    together up to a quarter.  On one block (a hint of many own pages), within the 2e-3."""
    from tests.kitty_cases import dev16
    n = 960
    own = dict(own=[0], tails=[1]) if kind is Packed else dict(lens=[1])
    c = kind(Hkv=1, Hq=1, dt=dt, n_prefix=n, shared=None, seed=46, **own)
    c.cfg.decode_total_pages = 1 << 20
    q = synth.from_bits(c.q, dt).astype(np.float64).reshape(D)
    k = np.random.default_rng(1).standard_normal((n * 32, 1, D)) * 1e-3
    k[0, 0] = q * gap / ((q * q).sum() * c.sm * np.log2(np.e))
    k = synth.to_bits(k, dt)
    if kind is Packed:
        from mixed_precision_bit_gb300 import kitty
        kitty.quantize_pages(c.cfg, dev16(k), dev16(c.v[:n * 32]), dev32(c.ids[:n]), c.pool, c.pool_pages)
    else:
        c.host[c.prefix, 0, 0] = k.reshape(n, 32, D)
        c.pool.copy_(dev16(c.host))
    ref, _ = c.oracle()
    assert attn_error(c.run("f32"), ref)[0] <= 0


@pytest.mark.parametrize("kind", [Packed, Plain16])
def test_the_merge_waits_for_a_prefix_that_ends_last(kind):
    """Hardly any own tokens: their kernel has long ended when the prefix's does, in a graph and
    in direct calls, with a workspace that holds NaN before each."""
    import torch
    own = dict(own=[0] * 3, tails=[1, 0, 2]) if kind is Packed else dict(lens=[1, 0, 2])
    c = kind(Hkv=1, Hq=4, dt=BF16, n_prefix=6000, shared=None, seed=45, **own)
    c.cfg.decode_total_pages = 1 << 20   # a hint far too high: the prefix on few blocks
    ws = c.workspace()
    out = torch.zeros(c.B, c.Hq, D, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call(out, ws=ws)
    ref, _ = c.oracle()
    for step in range(6):
        ws.fill_(float("nan"))
        out.zero_()
        g.replay() if step % 2 else c.call(out, ws=ws)
        torch.cuda.synchronize()
        assert attn_error(out.cpu().numpy().astype(np.float64), ref)[0] <= 0, step


def test_16_bit_offsets_beyond_32_bits():
    """Prefix and own pages more than 4 GiB into the pool."""
    import torch
    if torch.cuda.get_device_properties(0).total_memory < 16 << 30:
        pytest.skip("needs 16 GiB")
    c = Plain16(8, 32, BF16, 6, [6, 3], [33, 5], seed=35)
    ref, _ = c.oracle()
    spare = (4 << 30) // (c.pool[0].numel() * 2) + 1000
    pool = torch.zeros((spare + c.pool_pages,) + tuple(c.pool.shape[1:]), dtype=c.pool.dtype, device="cuda")
    pool[spare:] = c.pool
    c.pool, c.pool_pages = pool, c.pool_pages + spare
    c.dev["prefix"] += spare
    c.dev["bt"] += spare
    assert attn_error(c.run("f32"), ref)[0] <= 0


@pytest.mark.parametrize("kind", [Packed, Plain16])
def test_wait_timeout_reports_and_returns(kind):
    """A wait bounded to one poll of its barrier runs out on ordinary copies (the pool is
    evicted from L2 first): reported, the call completes, and the next one with the library's
    bound gives the same bytes as before."""
    import torch
    own = dict(own=[0] * 40, tails=[1] * 40) if kind is Packed else dict(lens=[1] * 40)
    c = kind(Hkv=8, Hq=32, dt=BF16, n_prefix=300, shared=None, seed=36, **own)
    before = c.run("f32")
    flush = torch.empty(512 << 20, dtype=torch.uint8, device="cuda")   # > 3x L2
    flush.fill_(1)
    from mixed_precision_bit_gb300 import kitty
    st = _status()
    c.cfg.decode_wait_polls = 1
    c.run("f32", st)
    assert int(st.item()) == kitty.ST["TIMEOUT"]
    c.cfg.decode_wait_polls = 0
    st.zero_()
    after = c.run("f32", st)
    assert int(st.item()) == 0 and np.array_equal(before, after)


# ------------------------------------------------------------------ norms and rotation
@pytest.mark.parametrize("dt", [BF16, F16], ids=["bf16", "f16"])
def test_weights_and_tables_that_are_not_aligned(dt):
    """Norm weights at any 2-byte address."""
    import torch
    from mixed_precision_bit_gb300 import kitty
    n, Hkv, Hq = 5, 2, 6
    t = rope_cases._dt(dt)
    w = (1 + 0.2 * torch.randn(2 * D + 3, device="cuda")).to(t)
    qw, kw = w[1:1 + D], w[D + 2:2 * D + 2]
    f = kitty.rope_frequencies(128, 10000.0)[0]
    rope = kitty.Rope(f, q_weight=qw, k_weight=kw, eps=1e-5)
    q, k = rope_cases._rows(n, Hq, dt, 1, 1), rope_cases._rows(n, Hkv, dt, 2, 1)
    qo, ko = torch.empty(n, Hq, D, dtype=t, device="cuda"), torch.empty(n, Hkv, D, dtype=t, device="cuda")
    pos = np.arange(n) * 100
    kitty.norm_rope(rope_cases._cfg(Hkv, Hq, dt), rope, q, k, dev32(pos), qo, ko)
    for x, y, wn in ((q, qo, qw), (k, ko, kw)):
        rope_cases._check(y, *rope_cases._turned(x.double().cpu().numpy(), f, pos, 0, 1.0, wn.double().cpu().numpy()), dt)


@pytest.mark.parametrize("B,each", [(300, 2), (70, 9), (513, 1), (2, 700)])
def test_append_of_many_sequences_and_tokens(B, each):
    """The search over seq_start at batches of several of its rounds, token counts past the
    launch rule's threshold, sequences without tokens between: pages, queries and lengths of
    norm_rope and plain copies."""
    import torch
    from mixed_precision_bit_gb300 import kitty
    r = np.random.default_rng(B)
    Hkv, Hq, dt = 1, 2, BF16
    new = np.full(B, each)
    new[r.integers(0, B, B // 3)] = 0
    new[-1] = each
    lens = r.integers(0, 40, B)
    n, max_pages = int(new.sum()), (40 + each) // 32 + 1
    cfg = rope_cases._cfg(Hkv, Hq, dt)
    bt = r.permutation(B * max_pages).reshape(B, max_pages).astype(np.int32)
    pool = torch.zeros(B * max_pages, Hkv, 2, 32, D, dtype=torch.int16, device="cuda")
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    seq = np.repeat(np.arange(B), new)
    pos = lens[seq] + np.arange(n) - start[seq]
    ids = bt[seq, pos // 32]
    rope, _ = rope_cases._rope(128, 0, dt, "qk")
    x = rope_cases._rows(n, Hq + 2 * Hkv, dt, 3)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    qo, q2 = (torch.empty(n, Hq, D, dtype=x.dtype, device="cuda") for _ in range(2))
    k2 = torch.empty(n, Hkv, D, dtype=x.dtype, device="cuda")
    kitty.norm_rope(cfg, rope, q, k, dev32(pos), q2, k2)
    want = torch.zeros_like(pool)
    at = (torch.from_numpy(ids.astype(np.int64)).cuda(), slice(None), slice(None), torch.from_numpy(pos % 32).cuda())
    want[at] = torch.stack([k2.view(torch.int16), v.contiguous().view(torch.int16)], 2)
    d_ln, st = dev32(lens), _status()
    kitty.f16kv_append_rope(cfg, rope, q, k, v, qo, pool, B * max_pages, dev32(bt), d_ln, dev32(ids),
                            seq_start=dev32(start), status=st)
    assert int(st.item()) == 0
    assert torch.equal(pool, want) and torch.equal(qo.view(torch.int16), q2.view(torch.int16))
    assert np.array_equal(d_ln.cpu().numpy(), lens + new)


def test_calls_without_tokens():
    import torch
    from mixed_precision_bit_gb300 import kitty
    cfg = rope_cases._cfg(1, 2, BF16)
    rope, _ = rope_cases._rope(128, 0, BF16, "qk")
    e = lambda h: torch.empty(0, h, D, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    kitty.norm_rope(cfg, rope, e(2), e(1), z(0), e(2), e(1))
    pool = torch.zeros(4, 1, 2, 32, D, dtype=torch.int16, device="cuda")
    ln = dev32([3, 4])
    kitty.f16kv_append_rope(cfg, rope, e(2), e(1), e(1), e(2), pool, 4, z(2, 2), ln, z(0), seq_start=z(3))
    assert ln.tolist() == [3, 4] and (pool == 0).all()
