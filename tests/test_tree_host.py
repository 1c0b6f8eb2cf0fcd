"""Refusals of the calls on drafted trees: argument errors come back before anything is launched."""

import ctypes

import pytest


@pytest.fixture(scope="module")
def K():
    from mixed_precision_bit_gb300 import kitty
    kitty.load()
    return kitty


X = 256  # a device address that is never read: every call below is refused, or has nothing to do


def test_plan(K):
    f = K.load().kitty_tree_plan
    ok = [X, X, 4, None, X, None, X, X, 2, None, None]
    for i, bad, code in ((0, None, -1), (1, None, -1), (2, -1, -1), (4, None, -1), (6, 257, -1), (8, -1, -1)):
        a = list(ok)
        a[i] = bad
        assert f(*a) == code, i
    assert f(X, X, 4, None, X, None, None, None, 2, None, None) == -1      # nothing to write
    assert f(None, None, 0, None, None, None, None, None, 0, None, None) == 0
    assert f(None, None, 0, None, None, None, None, None, 7, None, None) == 0


def test_page_tables(K):
    f = K.load().kitty_page_tables
    #     pages lens start  n extra part shr held  bt  M  ids count pool slots new  B  st stream
    ok = [None, X, X, 4, 0, 1, 0, X, X, 8, X, X, 64, X, X, 2, None, None]
    for i, bad, code in ((1, None, -1), (3, -1, -1), (7, None, -1), (8, None, -1), (9, -1, -1), (10, None, -1),
                         (11, None, -1), (12, -1, -1), (13, 260, -1), (15, -1, -1), (2, None, -1), (9, 1 << 30, -2)):
        a = list(ok)
        a[i] = bad
        assert f(*a) == code, i
    a = list(ok)
    a[15] = 0
    assert f(*a) == 0


def _attention(K, cfg, f16, **change):
    #        q  stride k  stride v  stride n  start vis nodes pool pages ptab np ppre  bt  M
    a = dict(q=X, qs=1024, k=X, ks=256, v=X, vs=256, n=4, start=X, vis=X, nodes=3, pool=X, pages=8, ptab=None,
             np=0, ppre=None, bt=X, M=4, lens=X, tk=X, tv=X, tl=X, sm=0.1, out=X, dt=2, ws=X, wsb=1 << 40, B=2,
             st=None, s=None)
    a.update(change)
    if f16:
        for x in ("tk", "tv", "tl"):
            del a[x]
    c = cfg.c()
    return getattr(K.load(), "kitty_f16kv_tree_attention" if f16 else "kitty_tree_attention")(ctypes.byref(c), *a.values())


@pytest.mark.parametrize("f16", [False, True])
def test_attention(K, f16):
    cfg = K.Config(num_kv_heads=2, num_q_heads=8)
    for change, code in ((dict(q=None), -1), (dict(q=264), -1), (dict(qs=1016), -1), (dict(qs=1028), -1), (dict(k=None), -1),
                         (dict(ks=128), -1), (dict(v=8), -1), (dict(vs=260), -1), (dict(n=-1), -1), (dict(start=None), -1),
                         (dict(vis=260), -1), (dict(nodes=0), -1), (dict(nodes=65), -2), (dict(pool=None), -1),
                         (dict(pool=264), -1), (dict(pages=-1), -1), (dict(np=1), -1), (dict(np=-1), -1),
                         (dict(bt=None), -1), (dict(M=-1), -1), (dict(lens=None), -1), (dict(sm=float("nan")), -1),
                         (dict(out=None), -1), (dict(out=264), -1), (dict(dt=3), -1), (dict(B=-1), -1)):
        assert _attention(K, cfg, f16, **change) == code, change
    if not f16:
        for change in (dict(tk=None), dict(tv=None), dict(tl=None), dict(tk=264), dict(tv=24)):
            assert _attention(K, cfg, f16, **change) == -1, change
    assert _attention(K, cfg, f16, B=0) == 0 and _attention(K, cfg, f16, n=0) == 0
    assert _attention(K, K.Config(num_kv_heads=1, num_q_heads=33), f16) == -2
    assert _attention(K, K.Config(num_kv_heads=2, num_q_heads=8, n_hi=8), f16) == -2


def test_workspace(K):
    cfg = K.Config(num_kv_heads=2, num_q_heads=8)
    for size in (K.tree_workspace_bytes, K.f16kv_tree_workspace_bytes):
        assert size(cfg, 0, 0, 1, 0) == 0
        assert size(cfg, 4, 20, 5, 300) >= 0
        for bad in ((-1, 4, 5, 3), (4, -1, 5, 3), (4, 4, 0, 3), (4, 4, 5, -1), (4, 4, 65, 3)):
            with pytest.raises(K.KittyError):
                size(cfg, *bad)
        with pytest.raises(K.KittyError):
            size(cfg, 4, 4, 5, 3, -1)


def test_commit(K):
    L, cfg = K.load(), K.Config(num_kv_heads=2, num_q_heads=8)
    c = ctypes.byref(cfg.c())
    #         k  ks   v  vs   n start path w len  tk tv tl run run run bt M np pool pages counted B st s
    packed = [X, 256, X, 256, 4, X, X, 8, X, X, X, X, None, None, None, X, 4, X, X, 8, 0, 2, None, None]
    for i, bad, code in ((0, None, -1), (1, 128, -1), (2, 264, -1), (3, 252, -1), (4, -1, -1), (5, None, -1), (6, None, -1),
                         (7, -1, -1), (7, 65, -2), (8, None, -1), (9, None, -1), (10, 264, -1), (11, None, -1),
                         (15, None, -1), (16, -1, -1), (17, None, -1), (18, 264, -1), (19, -1, -1), (21, -1, -1)):
        a = list(packed)
        a[i] = bad
        assert L.kitty_tree_commit(c, *a) == code, i
    for i in (4, 7, 21):
        a = list(packed)
        a[i] = 0
        assert L.kitty_tree_commit(c, *a) == 0
    run = ctypes.byref(K.Config(num_kv_heads=2, num_q_heads=8, rank_mode=1).c())
    assert L.kitty_tree_commit(run, *packed) == -1
    #        k  ks   v  vs   n start path w len pool pages bt M lens counted B st s
    plain = [X, 256, X, 256, 4, X, X, 8, X, X, 8, X, 4, X, 0, 2, None, None]
    for i, bad, code in ((0, 264, -1), (1, 260, -1), (4, -1, -1), (5, None, -1), (6, None, -1), (7, 65, -2), (8, None, -1),
                         (9, None, -1), (10, -1, -1), (11, None, -1), (12, -1, -1), (13, None, -1), (15, -1, -1)):
        a = list(plain)
        a[i] = bad
        assert L.kitty_f16kv_tree_commit(c, *a) == code, i


def test_tensors_are_checked(K, monkeypatch):
    """Shapes, types and devices of tensors, before the library is called."""
    import torch
    monkeypatch.setattr(K, "_device", lambda: 0)
    cfg = K.Config(num_kv_heads=2, num_q_heads=8)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    rows = lambda h, dt=torch.bfloat16: torch.zeros((4, h, 128), dtype=dt)  # noqa: E731
    with pytest.raises(ValueError, match="device"):
        K.tree_plan(i32(4), i32(3), i32(2), torch.zeros(4, dtype=torch.int64), i32(4))
    with pytest.raises(ValueError, match="64-bit"):
        K._longs("visible", i32(4), 4, -1)
    with pytest.raises(ValueError, match="64-bit"):
        K._longs("visible", torch.zeros(3, dtype=torch.int64), 4, -1)
    with pytest.raises(ValueError, match="out must be"):
        K.tree_attention(cfg, rows(8), rows(2), rows(2), i32(3), None, 4, None, 0, i32(2, 3), i32(2), None, None,
                         i32(2), 0.1, rows(7))
    with pytest.raises(ValueError, match="16-bit rows|float16"):
        K.tree_attention(cfg, rows(8, torch.float16), rows(2), rows(2), i32(3), None, 4, None, 0, i32(2, 3), i32(2), None,
                         None, i32(2), 0.1, rows(8))
    with pytest.raises(ValueError, match="paths"):
        K._path(i32(1, 8), i32(2), 2, -1)
    with pytest.raises(ValueError, match="path_len"):
        K._path(i32(2, 8), i32(1), 2, -1)


@pytest.mark.parametrize("kind", ["LayerCache", "F16LayerCache"])
def test_pages_are_planned_in_one_place(K, kind):
    """While the device plans the pages, what the host plans is refused, and the other way round."""
    import numpy as np
    import torch
    from mixed_precision_bit_gb300 import cache
    c = getattr(cache, kind)(K.Config(num_kv_heads=2, num_q_heads=4), 3, 4, 11, device="cpu")
    with pytest.raises(ValueError, match="on the host"):
        c.reserve(1)
    with pytest.raises(ValueError, match="on the host"):
        c.commit_tree(None, None, None, None, None)
    with pytest.raises(ValueError, match="on the host"):
        c.pages_to_host()
    mine = c.alloc.alloc(2)
    c.pages_to_device()
    assert c.free_count.tolist() == [9] and c.held.tolist() == [0, 0, 0] and c.alloc.free_count == 0
    ids = c.free_ids.tolist()
    assert sorted(ids[:9] + list(mine)) == list(range(11)) and ids[9:] == [-1, -1]
    for call in (c.plan_flush, c.clear, c.drop_prefix, c.kv_tokens, c.algorithmic_bytes, c.pages_to_device,
                 lambda: c.prefill(None, None, np.zeros(3)), lambda: c.share_prefix(torch.zeros(32, 2, 128), None)):
        with pytest.raises(ValueError, match="on the device"):
            call()
    if kind == "F16LayerCache":
        with pytest.raises(ValueError, match="on the device"):
            c.plan_extend([1, 1, 1])
    # an append that was planned and not made: its page is in no table yet
    c = getattr(cache, kind)(K.Config(num_kv_heads=2, num_q_heads=4), 3, 4, 11, device="cpu")
    c.plan_flush()
    with pytest.raises(ValueError, match="has not been made"):
        c.pages_to_device()


@pytest.mark.parametrize("name", ["kitty_tree_workspace_bytes", "kitty_f16kv_tree_workspace_bytes"])
def test_rows_are_counted_in_32_bits(K, name):
    cfg, n = K.Config(num_kv_heads=2, num_q_heads=4), ctypes.c_size_t()
    f = getattr(K.load(), name)
    assert f(cfg.ref(), 65535, (1 << 29) - 1, 64, 300, 8, ctypes.byref(n)) == 0
    assert f(cfg.ref(), 65535, 1 << 29, 64, 300, 8, ctypes.byref(n)) == -2
