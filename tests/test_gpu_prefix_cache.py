"""The operators together, as a server uses them: a prompt from the projections (norm and
rotation, prefill) behind a shared prefix, then decode steps (rotated append, shared attention)
through flushes, against caches of the same kind that hold every sequence's whole context by
itself.  Both sides' outputs are within 2e-3 of the output RMS of the exact value, so they
agree within 4e-3; pages, tails and lengths that both hold are the same bytes."""

import numpy as np
import pytest

from mixed_precision_bit_gb300 import synth

pytestmark = pytest.mark.gpu
P, D = 32, 128
B, Hkv, Hq, NP = 5, 2, 8, 6            # NP shared pages
OWN = np.array([0, 40, 64, 31, 7])     # own prompt tokens


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixed_precision_bit_gb300 import kitty
    kitty.load()


def _rope(dt):
    import torch
    from mixed_precision_bit_gb300 import kitty
    t = torch.bfloat16 if dt == synth.BF16 else torch.float16
    w = [(1 + 0.1 * torch.randn(D, device="cuda")).to(t) for _ in range(2)]
    return kitty.Rope(kitty.rope_frequencies(128, 10000.0)[0], q_weight=w[0], k_weight=w[1]), t


def _rows(n, t, seed):
    import torch
    x = torch.randn(n, Hq + 2 * Hkv, D, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)).to(t)
    return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]


def _close(a, b):
    d = (a.float() - b.float()).abs().max().item()
    assert d <= 4e-3 * b.float().square().mean().sqrt().item(), d


def _whole(k, v, starts):
    """Each sequence's prefix tokens followed by its own."""
    import torch
    pk, pv, ok, ov = k[0], v[0], k[1], v[1]
    ks = [torch.cat([pk, ok[starts[b]:starts[b + 1]]]) for b in range(B)]
    vs = [torch.cat([pv, ov[starts[b]:starts[b + 1]]]) for b in range(B)]
    return torch.cat(ks), torch.cat(vs)


@pytest.mark.parametrize("rank", [0, 1], ids=["page", "running"])
@pytest.mark.parametrize("fmt", [dict(n_hi=32), dict(n_hi=16, hi_bit=8, lo_bit=4, v_bit=4)], ids=["42", "84v4"])
def test_packed_cache_behind_a_shared_prefix(rank, fmt):
    import torch
    from mixed_precision_bit_gb300 import kitty
    from mixed_precision_bit_gb300.cache import LayerCache
    torch.manual_seed(5)
    rope, t = _rope(synth.BF16)
    cfg = kitty.Config(num_kv_heads=Hkv, num_q_heads=Hq, in_dtype=synth.BF16, rank_mode=rank, **fmt)
    max_pages = 5
    a = LayerCache(cfg, B, max_pages, NP + B * max_pages)
    c = LayerCache(cfg, B, NP + max_pages, B * (NP + max_pages))
    starts = np.concatenate([[0], np.cumsum(OWN)])
    _, pk, pv = _rows(NP * P, t, 1)
    q, ok, ov = _rows(int(OWN.sum()), t, 2)
    # the shared cache: the prefix's keys rotated once, then the sequences' own prompts
    pos = torch.arange(NP * P, dtype=torch.int32, device="cuda")
    pk_rot = torch.empty(NP * P, Hkv, D, dtype=t, device="cuda")
    kitty.norm_rope(cfg, rope, None, pk, pos, None, pk_rot)
    a.share_prefix(pk_rot, pv.contiguous())
    qa = torch.empty(q.shape, dtype=t, device="cuda")
    a.prefill_rope(rope, q, ok, ov, OWN, qa)
    # the whole contexts
    wk, wv = _whole((pk, ok), (pv, ov), starts)
    wq = torch.randn(wk.shape[0], Hq, D, device="cuda").to(t)
    c.prefill_rope(rope, wq, wk, wv, NP * P + OWN, torch.empty_like(wq))
    assert torch.equal(a.tail_len, c.tail_len) and torch.equal(a.num_pages + NP, c.num_pages)
    assert a.kv_tokens() == c.kv_tokens()
    outs = [torch.empty(B, Hq, D, device="cuda") for _ in range(2)]
    qr = [torch.empty(B, Hq, D, dtype=t, device="cuda") for _ in range(2)]
    for step in range(40):
        q, k, v = _rows(B, t, 100 + step)
        for lc, o, r in ((a, outs[0], qr[0]), (c, outs[1], qr[1])):
            fl = torch.from_numpy(lc.plan_flush()).cuda()
            lc.step_rope(rope, q, k, v, fl, r, o)
        assert torch.equal(qr[0].view(torch.int16), qr[1].view(torch.int16))
        assert torch.equal(a.tail_len, c.tail_len) and torch.equal(a.num_pages + NP, c.num_pages)
        _close(*outs)
    # the pages that both hold: the prefix's, and each sequence's own
    pools = [lc.pool.view(lc.pool_pages, -1) for lc in (a, c)]
    for b in range(B):
        n = int(a.num_pages[b])
        ids = (torch.cat([a.prefix, a.block_table[b, :n]]).long(), c.block_table[b, :NP + n].long())
        assert torch.equal(pools[0][ids[0]], pools[1][ids[1]]), b
        m = int(a.tail_len[b])
        for x, y in ((a.tail_k, c.tail_k), (a.tail_v, c.tail_v)):
            assert torch.equal(x[b, :, :m], y[b, :, :m])
    if rank:
        assert torch.equal(a.run_sum, c.run_sum) and torch.equal(a.run_count, c.run_count)
    assert int(a.status.item()) == int(c.status.item()) == 0
    free = a.alloc.free_count
    a.drop_prefix()
    assert a.alloc.free_count == free + NP and a.prefix is None


def test_16_bit_cache_behind_a_forked_prefix():
    import torch
    from mixed_precision_bit_gb300 import kitty
    from mixed_precision_bit_gb300.cache import F16LayerCache
    torch.manual_seed(6)
    rope, t = _rope(synth.F16)
    cfg = kitty.Config(num_kv_heads=Hkv, num_q_heads=Hq, in_dtype=synth.F16)
    max_pages = 5
    sees = np.array([6, 0, 3, 6, 5])
    a = F16LayerCache(cfg, B, max_pages, NP + B * max_pages)
    c = F16LayerCache(cfg, B, NP + max_pages, B * (NP + max_pages))
    _, pk, pv = _rows(NP * P, t, 1)
    pos = torch.arange(NP * P, dtype=torch.int32, device="cuda")
    pk_rot = torch.empty(NP * P, Hkv, D, dtype=t, device="cuda")
    kitty.norm_rope(cfg, rope, None, pk, pos, None, pk_rot)
    a.share_prefix(pk_rot, pv.contiguous(), pages_of=sees)
    starts = np.concatenate([[0], np.cumsum(OWN)])
    q, ok, ov = _rows(int(OWN.sum()), t, 2)
    a.extend_rope(rope, q, ok, ov, OWN, torch.empty(q.shape, dtype=t, device="cuda"))
    ks = torch.cat([torch.cat([pk[:sees[b] * P], ok[starts[b]:starts[b + 1]]]) for b in range(B)])
    vs = torch.cat([torch.cat([pv[:sees[b] * P], ov[starts[b]:starts[b + 1]]]) for b in range(B)])
    wq = torch.randn(ks.shape[0], Hq, D, device="cuda").to(t)
    # the whole contexts, in two runs of uneven lengths
    whole = sees * P + OWN
    first = whole // 3
    s = np.concatenate([[0], np.cumsum(whole)])
    for lo, hi in ((np.zeros(B, int), first), (first, whole)):
        sel = torch.from_numpy(np.concatenate([np.arange(s[b] + lo[b], s[b] + hi[b]) for b in range(B)])).cuda()
        c.extend_rope(rope, wq[sel], ks[sel], vs[sel], hi - lo, torch.empty(sel.numel(), Hq, D, dtype=t, device="cuda"))
    assert a.kv_tokens() == c.kv_tokens()
    outs = [torch.empty(B, Hq, D, device="cuda") for _ in range(2)]
    qr = [torch.empty(B, Hq, D, dtype=t, device="cuda") for _ in range(2)]
    for step in range(34):
        q, k, v = _rows(B, t, 200 + step)
        for lc, o, r in ((a, outs[0], qr[0]), (c, outs[1], qr[1])):
            lc.step_rope(rope, q, k, v, torch.from_numpy(lc.plan_flush()).cuda(), r, o)
        assert torch.equal(qr[0].view(torch.int16), qr[1].view(torch.int16))
        _close(*outs)
    assert int(a.status.item()) == int(c.status.item()) == 0
    assert np.array_equal(a.ctx_len.cpu().numpy(), a.h_len)


def test_serving_step_behind_a_shared_prefix():
    """ServingStep's graphs call the shared attention of layers that have a prefix: the bytes of
    direct calls."""
    import torch
    from mixed_precision_bit_gb300 import kitty
    from mixed_precision_bit_gb300.cache import LayerCache, ServingStep
    cfg = kitty.Config(num_kv_heads=Hkv, num_q_heads=Hq, in_dtype=synth.BF16, n_hi=32)
    t, layers = torch.bfloat16, []
    for copy in range(2):
        for l in range(2):
            lc = LayerCache(cfg, B, 5, NP + 5 * B)
            _, k, v = _rows(NP * P, t, 10 + l)
            lc.share_prefix(k.contiguous(), v.contiguous())
            _, k, v = _rows(B * P, t, 20 + l)
            lc.prefill(k.contiguous(), v.contiguous(), np.ones(B, int))
            layers.append(lc)
    srv = ServingStep(layers[:2])
    out = torch.empty(B, Hq, D, dtype=t, device="cuda")
    for step in range(34):
        rows = [[x.contiguous() for x in _rows(B, t, 300 + 2 * step + l)] for l in range(2)]
        for l in range(2):
            for dst, x in zip((srv.q[l], srv.k_new[l], srv.v_new[l]), rows[l]):
                dst.copy_(x.view(torch.int16).cpu())
        got = srv.run().clone()
        for l in range(2):
            lc = layers[2 + l]
            lc.step(rows[l][1], rows[l][2], torch.from_numpy(lc.plan_flush()).cuda(), rows[l][0], out)
            assert torch.equal(got[l].view(torch.int16), out.cpu().view(torch.int16)), (step, l)


@pytest.mark.parametrize("packed", [True, False], ids=["packed", "16-bit"])
def test_captured_steps_behind_a_prefix(packed):
    """One graph of step_rope (rotated append, shared attention), replayed on new rows and flush
    plans: outputs and cache of direct calls."""
    import torch
    from mixed_precision_bit_gb300 import kitty
    from mixed_precision_bit_gb300.cache import F16LayerCache, LayerCache
    torch.manual_seed(7)
    rope, t = _rope(synth.BF16)
    cfg = kitty.Config(num_kv_heads=Hkv, num_q_heads=Hq, in_dtype=synth.BF16)
    caches = []
    _, pk, pv = _rows(NP * P, t, 1)
    _, ok, ov = _rows(int(OWN.sum()), t, 2)
    for _ in range(2):
        lc = (LayerCache if packed else F16LayerCache)(cfg, B, 5, NP + B * 5)
        lc.share_prefix(pk.contiguous(), pv.contiguous(), pages_of=[6, 2, 6, 0, 5])
        (lc.prefill_rope if packed else lc.extend_rope)(rope, None, ok, ov, OWN, None)
        caches.append(lc)
    q, k, v = _rows(B, t, 3)
    fl = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    r, out = torch.empty(B, Hq, D, dtype=t, device="cuda"), torch.zeros(B, Hq, D, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        caches[0].step_rope(rope, q, k, v, fl, r, out)
    r2, out2 = torch.empty_like(r), torch.zeros_like(out)
    for step in range(34):
        y = _rows(B, t, 400 + step)
        for dst, x in zip((q, k, v), y):
            dst.copy_(x)
        plans = [lc.plan_flush() for lc in caches]
        assert np.array_equal(*plans)
        fl.copy_(torch.from_numpy(plans[0]))
        g.replay()
        caches[1].step_rope(rope, *y, torch.from_numpy(plans[1]).cuda(), r2, out2)
        assert torch.equal(out, out2) and torch.equal(r, r2), step
    assert torch.equal(caches[0].pool, caches[1].pool)
    assert all(int(lc.status.item()) == 0 for lc in caches)


@pytest.mark.parametrize("change", ["share", "drop", "clear"])
def test_serving_step_refuses_layers_that_it_was_not_captured_with(change):
    """A step's graphs attend the prefix that the layers had when it was made: without it, or with
    another, they would go on without a word.  Direct calls follow the layers."""
    import torch
    from mixed_precision_bit_gb300 import kitty
    from mixed_precision_bit_gb300.cache import LayerCache, ServingStep
    cfg = kitty.Config(num_kv_heads=Hkv, num_q_heads=Hq, in_dtype=synth.BF16, n_hi=32)
    t = torch.bfloat16
    pre, own = [[x.contiguous() for x in _rows(n * P, t, s)[1:]] for n, s in ((NP, 10), (B, 20))]
    x = [[r.contiguous() for r in _rows(B, t, s)] for s in (30, 31)]

    def layer(prefix):
        lc = LayerCache(cfg, B, 5, NP + 5 * B)
        if prefix:
            lc.share_prefix(*pre)
        return lc

    layers = {g: [layer(change != "share") for _ in range(2)] for g in (True, False)}
    srv = {g: ServingStep(layers[g], graphs=g) for g in (True, False)}
    for g, lcs in layers.items():
        for lc in lcs:
            if change == "share":
                lc.share_prefix(*pre)
            elif change == "drop":
                lc.drop_prefix()
            else:
                lc.clear()
            lc.prefill(*own, np.ones(B, int))
        for l in range(2):
            for dst, r in zip((srv[g].q[l], srv[g].k_new[l], srv[g].v_new[l]), x[l]):
                dst.copy_(r.view(torch.int16).cpu())
    tails = [lc.tail_len.clone() for lc in layers[True]]
    with pytest.raises(ValueError, match="new ServingStep"):
        srv[True].run()
    for lc, n in zip(layers[True], tails):                 # refused before anything was planned or run
        assert torch.equal(lc.tail_len, n) and (lc.h_tail == 0).all()
    got = {False: srv[False].run().clone()}
    again = ServingStep(layers[True])
    for l in range(2):
        for dst, r in zip((again.q[l], again.k_new[l], again.v_new[l]), x[l]):
            dst.copy_(r.view(torch.int16).cpu())
    got[True] = again.run().clone()
    assert torch.equal(got[True].view(torch.int16), got[False].view(torch.int16))
    out = torch.empty(B, Hq, D, dtype=t, device="cuda")
    for l in range(2):
        lc = layer(change != "drop")
        lc.prefill(*own, np.ones(B, int))
        lc.step(x[l][1], x[l][2], torch.from_numpy(lc.plan_flush()).cuda(), x[l][0], out)
        assert torch.equal(got[True][l].view(torch.int16), out.cpu().view(torch.int16)), l
